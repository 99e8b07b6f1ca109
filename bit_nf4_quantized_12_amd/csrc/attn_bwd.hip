// Backward pass of the sliding-window attention with visible first tokens.
//
// With p_ij = exp(s_ij - lse_i) over the pairs that query i sees (attn.hpp):
//   delta_i = sum_d do_id o_id
//   ds_ij = scale p_ij (do_i . v_j - delta_i)
//   dq_i = sum_j ds_ij k_j,  dk_j = sum_i ds_ij q_i,  dv_j = sum_i p_ij do_i
// where j's sums run over all query heads that share its key head.
//
// Up to five kernels, none with atomics, so gradients do not change from run to run:
//   dq      128 queries per workgroup, as the forward pass; also writes delta
//           and lse in base 2
//   sink    the first tokens are seen by every later query: their dK and dV
//           from the queries past the window of key block 0, cut into ranges
//           of rows, float32 shares (only with sinks)
//   join    adds those shares in order
//   dkdv    64 keys per workgroup, loops over the queries (and the heads) that
//           can see them; key block 0 adds the joined shares. With few key
//           blocks each one's loop is cut into parts, and a last kernel adds
//           their float32 shares in order
// Scores are computed twice (7 products in all instead of 5): the alternative,
// dq added up across workgroups, needs float32 atomics in memory.
//
// At 16 x 512 tokens, 64 heads of 128, window 256: 508 to 520 us for calls in a row;
// under a kernel trace, which lengthens each launch by 5 to 10 %, dq takes 263 and
// dkdv 305. Neither the matrix pipe (busy 17 and 19 %), vector issue (21 and 26 %)
// nor HBM (2 to 3 TB/s) is full: walks of 1 to 8 tiles do not hide the way to their
// first one. 6143 uneven tokens, 32 heads of 64 on 8 key heads, window 1000: 242 to
// 262 us, by the lengths; under the trace dq 88 (matrix 28 %, vector 39 %), sink and
// join 22, dkdv 162 (19 and 34 %): its longest walks, 17 tiles for each of 4 heads,
// end last. Long walks (8192 tokens, 32 heads of 128, window 4096): 1661 us, dq with
// the matrix pipe busy 44 %, dkdv 38 %.
#include "attn.hpp"

namespace qlora {
namespace {

constexpr int kRows = 128;  // queries of a workgroup (dq)

// ---------------------------------------------------------------------------
// dq
// ---------------------------------------------------------------------------
template <int DP>
struct DqState {
  bf16x8 q[DP / 16], g[DP / 16];  // q and do of the lane's query
  f32x16 dq[DP / 32];
  float lse2, delta;              // base 2
};

template <int DP>
__device__ __forceinline__ void dq_tile(const uint16_t* __restrict__ kt, const uint16_t* __restrict__ vt,
                                        DqState<DP>& st, int j0, int pos, bool edge, int window, int sinks, float c,
                                        const LaneOffsets& lofs, int l) {
  constexpr int KS = DP / 16, G = DP / 32, NR = KS / G;  // groups of a row product: 2
  constexpr int N = 2 * NR + 2;                          // groups of 32 keys: k rows, v rows, k columns
  bf16x8 f[3][G];
  // group g of the tile, fragments read two groups ahead of their products
  auto read = [&](int g) {
    const int b = g / N, h = g % N;
#pragma unroll
    for (int i = 0; i < G; ++i) {
      if (h < 2 * NR) f[g % 3][i] = row_frag<DP>(h < NR ? kt : vt, 32 * b, h % NR * G + i, lofs);
      else f[g % 3][i] = col_frag<DP>(kt, 32 * b + 16 * (h - 2 * NR), i, lofs);
    }
  };
  read(0);
  read(1);
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    f32x16 s = zero16(), dp = zero16();
#pragma unroll
    for (int h = 0; h < 2 * NR; ++h) {
      const int g = b * N + h;
      __builtin_amdgcn_sched_barrier(0);
      read(g + 2);
#pragma unroll
      for (int i = 0; i < G; ++i) {
        if (h < NR) s = mfma32(f[g % 3][i], st.q[h * G + i], s);
        else dp = mfma32(f[g % 3][i], st.g[(h - NR) * G + i], dp);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int r = 0; r < 16; ++r) s[r] = fast_exp2(__builtin_fmaf(s[r], c, -st.lse2)) * (dp[r] - st.delta);
    if (edge) hide_keys(s, 0.f, j0 + 32 * b, pos, window, sinks, l);
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      const int g = b * N + 2 * NR + kb;
      __builtin_amdgcn_sched_barrier(0);
      if (g + 2 < 2 * N) read(g + 2);
      const bf16x8 ds = pack_frag(s, kb);
#pragma unroll
      for (int d = 0; d < G; ++d) st.dq[d] = mfma32(f[g % 3][d], ds, st.dq[d]);
    }
  }
}

template <int DP>
__global__ __launch_bounds__(256, 2) void attn_dq_kernel(AttnArgs a, int nq, UnitGrid ug) {
  extern __shared__ __align__(16) uint16_t lds[];
  constexpr int kTile = 64 * DP;
  const UnitItem ui = unit_item(ug);
  if (ui.item < 0) return;
  const int tid = threadIdx.x, l = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int group = a.H / a.Hkv;
  const int b = ui.unit / a.Hkv, hk = ui.unit % a.Hkv, hq = hk * group + ui.item % group, x = ui.item / group;
  const SeqView sv = seq_view(a, b);
  const uint16_t* kp = static_cast<const uint16_t*>(a.k.p) + sv.k0 * a.k.st + hk * a.k.sh;
  const uint16_t* vp = static_cast<const uint16_t*>(a.v.p) + sv.k0 * a.v.st + hk * a.v.sh;
  const float c = a.scale * kAttnLog2e;
  const int shift = sv.Lk - sv.Lq;
  const LaneOffsets lofs = lane_offsets<DP>(l);
  const TileLoad<DP, 4> load_k(a.k.st, a.D, w, l), load_v(a.v.st, a.D, w, l);
  const int blocks = (sv.Lq + kRows - 1) / kRows;
  for (int y = blocks - 1 - x; y >= 0; y -= nq) {
    const int i0 = y * kRows, i1 = min(i0 + kRows, sv.Lq) - 1;
    const int wi0 = i0 + 32 * w, wi1 = min(wi0 + 31, sv.Lq - 1);
    const int iq = wi0 + (l & 31);
    const bool have = iq < sv.Lq;
    const int pos = min(iq + shift, sv.Lk - 1);
    const int64_t row = sv.q0 + (have ? iq : 0);
    const uint16_t* qp = static_cast<const uint16_t*>(a.q.p) + row * a.q.st + hq * a.q.sh;
    const uint16_t* gp = static_cast<const uint16_t*>(a.d_o.p) + row * a.d_o.st + hq * a.d_o.sh;
    const uint16_t* op = static_cast<const uint16_t*>(a.o.p) + row * a.o.st + hq * a.o.sh;
    DqState<DP> st;
    float dot = 0.f;
#pragma unroll
    for (int ks = 0; ks < DP / 16; ++ks) {
      st.q[ks] = global_frag(qp, have, a.D, ks, l);
      st.g[ks] = global_frag(gp, have, a.D, ks, l);
      const bf16x8 ov = global_frag(op, have, a.D, ks, l);
#pragma unroll
      for (int e = 0; e < 8; ++e) dot = __builtin_fmaf((float)st.g[ks][e], (float)ov[e], dot);
    }
    st.delta = half_sum(dot);
    const int64_t at = (int64_t)hq * a.Tq + row;
    st.lse2 = have ? a.lse[at] * kAttnLog2e : 0.f;
    if (have && l < 32) {
      a.delta[at] = st.delta;
      a.lse2[at] = st.lse2 == -__builtin_inff() ? 0.f : st.lse2;  // sees nothing: p is masked
    }
#pragma unroll
    for (int d = 0; d < DP / 32; ++d) st.dq[d] = zero16();

    const TileWalk walk(i0 + shift, i1 + shift, wi0 + shift, wi1 + shift, sv.Lk, a.window, a.sinks);
    TileSource src_k(kp, a.k.st, walk), src_v(vp, a.v.st, walk);
    int last = sv.Lk - 1 - 64 * walk.tile(0);  // of the tile asked for next
    auto issue = [&](int i) {
      uint16_t* dst = lds + (i & 1) * 2 * kTile;
      load_k(src_k.p, last, dst, w);
      load_v(src_v.p, last, dst + kTile, w);
      src_k.next(i, walk);
      src_v.next(i, walk);
      last -= i + 1 == walk.first ? walk.jump : 64;
    };
    if (walk.n > 0) issue(0);
    for (int t0 = 0; t0 < walk.n; t0 += 2) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int i = t0 + u;
        if (i >= walk.n) break;
        wait_vm<0>();
        __builtin_amdgcn_s_barrier();
        if (i + 1 < walk.n) issue(i + 1);
        const int t = walk.tile(i);
        if (walk.hidden(t)) continue;
        const uint16_t* kt = lds + u * 2 * kTile;
        dq_tile<DP>(kt, kt + kTile, st, 64 * t, pos, walk.edge(t), a.window, a.sinks, c, lofs, l);
      }
    }
    __builtin_amdgcn_s_barrier();
    if (have) {
      uint16_t* dst = static_cast<uint16_t*>(a.dq.p) + row * a.dq.st + hq * a.dq.sh;
#pragma unroll
      for (int d = 0; d < DP / 32; ++d)
#pragma unroll
        for (int r = 0; r < 16; r += 4) {
          const int col = 32 * d + block_row(r, l >> 5);
          if (col < a.D)
            *reinterpret_cast<uint2*>(dst + col) =
                make_uint2(pack_bf16(st.dq[d][r] * a.scale, st.dq[d][r + 1] * a.scale),
                           pack_bf16(st.dq[d][r + 2] * a.scale, st.dq[d][r + 3] * a.scale));
        }
    }
  }
  if (b == a.B - 1) zero_rows(a.dq, hq, sv.q0 + sv.Lq, a.Tq, a.D, x, nq);
}

// ---------------------------------------------------------------------------
// dk and dv
// ---------------------------------------------------------------------------
// A wave takes 16 keys, in 16 x 16 x 32 products: with 32 keys and heads of 128 its
// two 32 x D accumulators and its keys and values fill 192 registers, one wave fits a SIMD
// and the compiler moves half of them in and out of the accumulation file for
// every tile (477 us where this form takes 300, at 16 x 512 tokens and 64 heads
// of 128). The price is twice the LDS reads for a product, 100 of the 222 bytes
// a clock that a compute unit's LDS was measured to give. Heads of 64, which would
// have the room for 32 keys, use the same form: theirs was not built.
// Four waves, 64 keys, a workgroup: two workgroups share a compute unit without
// waiting for each other's barriers (506 us; one workgroup of 128 keys and three
// stages 534 us).
constexpr int kKeyWaves = 4;
constexpr int kKeys = 16 * kKeyWaves;  // of a workgroup
constexpr int kSinkWaves = 8;
template <int DP>
struct DkvState {
  bf16x8 k[DP / 32], v[DP / 32];  // of the lane's key
  f32x4 dk[DP / 16], dv[DP / 16];
};

// 64 query rows (positions p0 .. + 63, the first `rows` of them exist) against
// the wave's 16 keys: the scores of 4 blocks of 16 rows, then the products of
// the two halves; the exponentials of a block run between later products, and
// fragments are read two groups of products ahead. qt, gt: tiles of q and do;
// ls, dl: their lse (base 2) and delta.
template <int DP>
__device__ __forceinline__ void dkv_tile(const uint16_t* __restrict__ qt, const uint16_t* __restrict__ gt,
                                         const float* __restrict__ ls, const float* __restrict__ dl,
                                         DkvState<DP>& st, int p0, int rows, int key, int window, int sinks, float c,
                                         const LaneOffsets& lofs, int l) {
  constexpr int G = DP / 32;  // G products make a group, 16 groups a tile
  // A row at distance d behind the lane's key sees it when 0 <= d < window (any
  // d for a first token) and the row exists: one unsigned comparison, made for
  // every tile (two forms of this loop cost more in copies of the accumulators
  // than the comparisons do beside the products).
  const uint32_t behind = (uint32_t)(p0 + 4 * (l >> 4) - key);
  const uint32_t reach = (uint32_t)max(0, min(key < sinks ? INT32_MAX : window, p0 + rows - key));
  bf16x8 f[3][G];
  f32x4 s[4], dp[4], l2[2], de[2];
  // groups 0 - 7: scores of block g / 2 (q, then do); 8 - 11 and 12 - 15: the
  // products of a half (dv, dv, dk, dk)
  auto read = [&](int g) {
#pragma unroll
    for (int i = 0; i < G; ++i) {
      if (g < 8) f[g % 3][i] = row_frag16<DP>(g % 2 == 0 ? qt : gt, 16 * (g / 2), i, lofs);
      else f[g % 3][i] = col_frag16<DP>(g % 4 < 2 ? gt : qt, 32 * ((g - 8) / 4), g % 2 * G + i, lofs);
    }
  };
  auto read_stats = [&](int b) {
    l2[b % 2] = *reinterpret_cast<const f32x4*>(ls + 16 * b + 4 * (l >> 4));
    de[b % 2] = *reinterpret_cast<const f32x4*>(dl + 16 * b + 4 * (l >> 4));
  };
  auto gradients = [&](int b, int r) {
    const float p = fast_exp2(__builtin_fmaf(s[b][r], c, -l2[b % 2][r]));
    const float d = p * (dp[b][r] - de[b % 2][r]);
    const bool see = behind + (uint32_t)(16 * b + r) < reach;
    float ps = see ? p : 0.f, ds = see ? d : 0.f;
    asm("" : "+v"(ps), "+v"(ds));  // (rounded in pairs, not one by one before the choice)
    s[b][r] = ps;
    dp[b][r] = ds;
  };
  read(0);
  read(1);
#pragma unroll
  for (int g = 0; g < 16; ++g) {
    __builtin_amdgcn_sched_barrier(0);
    if (g + 2 < 16) read(g + 2);
    if (g % 2 == 1 && g < 8) read_stats(g / 2);
    if (g < 8) {
      const int b = g / 2;
      if (g % 2 == 0) s[b] = dp[b] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < G; ++i) {
        if (g % 2 == 0) s[b] = mfma16(f[g % 3][i], st.k[i], s[b]);
        else dp[b] = mfma16(f[g % 3][i], st.v[i], dp[b]);
      }
    } else {
      const int h = (g - 8) / 4;
      const f32x4 &x = g % 4 < 2 ? s[2 * h] : dp[2 * h], &y = g % 4 < 2 ? s[2 * h + 1] : dp[2 * h + 1];
      const bf16x8 w = __builtin_bit_cast(bf16x8, make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]),
                                                             pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3])));
#pragma unroll
      for (int i = 0; i < G; ++i) {
        const int d = g % 2 * G + i;
        if (g % 4 < 2) st.dv[d] = mfma16(f[g % 3][i], w, st.dv[d]);
        else st.dk[d] = mfma16(f[g % 3][i], w, st.dk[d]);
      }
    }
    if (g >= 2 && g < 10) {
      gradients(g / 2 - 1, g % 2 * 2);
      gradients(g / 2 - 1, g % 2 * 2 + 1);
    }
  }
  __builtin_amdgcn_sched_barrier(0);
}

template <int DP>
__device__ __forceinline__ void load_keys(const AttnArgs& a, const SeqView& sv, int hk, int key, DkvState<DP>& st,
                                          int l) {
  const bool have = key < sv.Lk;
  const int64_t row = sv.k0 + (have ? key : 0);
  const uint16_t* kp = static_cast<const uint16_t*>(a.k.p) + row * a.k.st + hk * a.k.sh;
  const uint16_t* vp = static_cast<const uint16_t*>(a.v.p) + row * a.v.st + hk * a.v.sh;
#pragma unroll
  for (int ks = 0; ks < DP / 32; ++ks) {
    const int col = 32 * ks + 8 * (l >> 4);
    const bool ok = have && col < a.D;
    const bf16x8 zero = __builtin_bit_cast(bf16x8, make_uint4(0, 0, 0, 0));
    st.k[ks] = ok ? *reinterpret_cast<const bf16x8*>(kp + col) : zero;
    st.v[ks] = ok ? *reinterpret_cast<const bf16x8*>(vp + col) : zero;
  }
#pragma unroll
  for (int d = 0; d < DP / 16; ++d) st.dk[d] = st.dv[d] = f32x4{0.f, 0.f, 0.f, 0.f};
}

// 64 query rows from row i0 of head hq into a stage: q, do, lse, delta.
template <int DP, int NW>
__device__ __forceinline__ void load_queries(const AttnArgs& a, const SeqView& sv, const TileLoad<DP, NW>& load_q,
                                             const TileLoad<DP, NW>& load_g, int hq, int i0, uint16_t* dst, int w,
                                             int l) {
  const int last = sv.Lq - 1 - i0;
  const int64_t row = sv.q0 + i0;
  load_q(static_cast<const uint16_t*>(a.q.p) + row * a.q.st + hq * a.q.sh, last, dst, w);
  load_g(static_cast<const uint16_t*>(a.d_o.p) + row * a.d_o.st + hq * a.d_o.sh, last, dst + 64 * DP, w);
  // lse and delta of the rows: waves 0 and 1 (the others repeat them, so that
  // every wave has the same number of loads in flight)
  const float* src = (w & 1 ? a.delta : a.lse2) + (int64_t)hq * a.Tq + row + min(l, last);
  __builtin_amdgcn_global_load_lds((gbl_void_t*)src, (lds_void_t*)(dst + 128 * DP + w * 128), 4, 0, 0);
}
template <int DP, int NW>
constexpr int kStage = 128 * DP + 128 * NW;  // elements: q, do, then 64 float32 of each wave
constexpr int kDkvStages = 2;  // of query tiles

// Rows of queries that see only key block 0's sinks: from `far` on.
__device__ __forceinline__ int far_row(const SeqView& sv, int window) {
  // positions past the last one at which any of the sinks' keys is in the window
  const int64_t p = (int64_t)kKeys - 1 + window;
  const int64_t i = p - (sv.Lk - sv.Lq);
  return i < 0 ? 0 : i > sv.Lq ? sv.Lq : (int)i;
}

// NS streams: the workgroup's waves are NS times kKeyWaves, each set takes its
// own range of the (head, query tile) steps with its own stages in LDS, and
// the first set adds the others' sums at the end. CUT: a.parts workgroups share
// a key block's steps likewise and leave float32 shares, which
// attn_dkv_join_kernel adds. (Forms of their own: the bookkeeping in the plain
// one costs 2 % at 16 x 512 tokens and 64 heads.)
template <int DP, int NS, bool CUT>
__global__ __launch_bounds__(64 * kKeyWaves * NS, 2) void attn_dkv_kernel(AttnArgs a, int nk, const float* sink, UnitGrid ug) {
  extern __shared__ __align__(16) uint16_t all_lds[];
  const UnitItem ui = unit_item(ug);
  if (ui.item < 0) return;
  const int tid = threadIdx.x, l = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int w = wave % kKeyWaves, stream = wave / kKeyWaves;
  uint16_t* lds = all_lds + stream * kDkvStages * kStage<DP, kKeyWaves>;
  const int b = ui.unit / a.Hkv, hk = ui.unit % a.Hkv, x = CUT ? ui.item / a.parts : ui.item, part = CUT ? ui.item % a.parts : 0;
  const SeqView sv = seq_view(a, b);
  const int group = a.H / a.Hkv;
  const float c = a.scale * kAttnLog2e;
  const int shift = sv.Lk - sv.Lq;
  const LaneOffsets lofs = lane_offsets16<DP>(l);
  const TileLoad<DP, kKeyWaves> load_q(a.q.st, a.D, w, l), load_g(a.d_o.st, a.D, w, l);
  for (int y = x; (int64_t)y * kKeys < sv.Lk; y += nk) {
    const int j0 = y * kKeys, j1 = min(j0 + kKeys, sv.Lk) - 1;
    const int wj0 = j0 + 16 * w, wj1 = min(wj0 + 15, sv.Lk - 1);
    const int key = wj0 + (l & 15);
    // query rows that have one of these keys in their window
    const int lo = max(0, j0 - shift);
    // (and, without the sink kernel, those that have one as a first token)
    int64_t up = min((int64_t)sv.Lq - 1, (int64_t)j1 + a.window - 1 - shift);
    if (y == 0 && a.sinks > 0 && sink == nullptr) up = sv.Lq - 1;
    const int tiles = sv.Lq > 0 && up >= lo ? (int)((up - lo) / 64 + 1) : 0;
    // steps of a stream; the last have fewer
    constexpr bool kWhole = NS == 1 && !CUT;
    const int ranges = CUT ? NS * a.parts : NS;
    const int steps = kWhole ? tiles * group : (tiles * group + ranges - 1) / ranges;
    const int beg = (part * NS + stream) * steps, n = kWhole ? steps : min(steps, tiles * group - beg);
    const int limit = (int)min((int64_t)sv.Lq, up + 1);
    int nh = 0, nt = 0;  // head and tile asked for next
    if (!kWhole && n > 0) nh = beg / tiles, nt = beg % tiles;
    int tile = nt, stage = 0;
    auto issue = [&](int stage) {
      load_queries<DP, kKeyWaves>(a, sv, load_q, load_g, hk * group + nh, lo + 64 * nt,
                                  lds + stage * kStage<DP, kKeyWaves>, w, l);
      if (++nt == tiles) nt = 0, ++nh;
    };
    constexpr int PER = 2 * TileLoad<DP, kKeyWaves>::NI + 1;
#pragma unroll
    for (int i = 0; i < kDkvStages - 1; ++i)
      if (i < n) issue(i);
    DkvState<DP> st;
    load_keys<DP>(a, sv, hk, key, st, l);
    // Everything so far has to be there: otherwise the compiler, which cannot
    // tell the keys' loads from the tiles' in flight, waits for all of them in
    // every pass of the loop.
    wait_vm<0>();
    for (int i = 0; i < steps; ++i) {
      wait_tile<PER, kDkvStages - 2>(i, n);
      __builtin_amdgcn_s_barrier();
      if (!kWhole && i >= n) continue;
      if (i + kDkvStages - 1 < n) issue(stage == 0 ? kDkvStages - 1 : stage - 1);
      const int i0 = lo + 64 * tile, p0 = i0 + shift;
      if (++tile == tiles) tile = 0;
      const uint16_t* t = lds + stage * kStage<DP, kKeyWaves>;
      if (++stage == kDkvStages) stage = 0;
      if (wj1 < wj0 || p0 + 63 < wj0 || (p0 - wj1 >= a.window && wj0 >= a.sinks)) continue;
      const int rows = min(64, limit - i0);
      const float* ls = reinterpret_cast<const float*>(t + 128 * DP);
      dkv_tile<DP>(t, t + 64 * DP, ls, ls + 64, st, p0, rows, key, a.window, a.sinks, c, lofs.fresh(), l);
    }
    __builtin_amdgcn_s_barrier();
    if constexpr (NS > 1) {
      // each later stream leaves its sums in its own stages
      if (stream > 0) {
        f32x4* f = reinterpret_cast<f32x4*>(lds) + w * 64 + l;
#pragma unroll
        for (int d = 0; d < DP / 16; ++d) {
          f[2 * d * 64 * kKeyWaves] = st.dk[d];
          f[(2 * d + 1) * 64 * kKeyWaves] = st.dv[d];
        }
      }
      __syncthreads();
      if (stream == 0) {
        for (int u = 1; u < NS; ++u) {
          const f32x4* f =
              reinterpret_cast<const f32x4*>(lds + u * kDkvStages * kStage<DP, kKeyWaves>) + w * 64 + l;
#pragma unroll
          for (int d = 0; d < DP / 16; ++d) {
            st.dk[d] += f[2 * d * 64 * kKeyWaves];
            st.dv[d] += f[(2 * d + 1) * 64 * kKeyWaves];
          }
        }
      }
      __syncthreads();
    }
    if (stream > 0 || key >= sv.Lk) continue;
    uint16_t* kd = static_cast<uint16_t*>(a.dk.p) + (sv.k0 + key) * a.dk.st + hk * a.dk.sh;
    uint16_t* vd = static_cast<uint16_t*>(a.dv.p) + (sv.k0 + key) * a.dv.st + hk * a.dv.sh;
    const bool add = sink != nullptr && key < a.sinks && part == 0;
    float* share = CUT ? a.share + (((int64_t)part * a.Tk + sv.k0 + key) * a.Hkv + hk) * (2 * DP) : nullptr;
    const float* sp = sink + (((int64_t)b * a.Hkv + hk) * 2 * kMaxSinks + key) * DP;
#pragma unroll
    for (int d = 0; d < DP / 16; ++d) {
      const int col = 16 * d + 4 * (l >> 4);
      f32x4 ak = st.dk[d], av = st.dv[d];
      if (add) {
        ak += *reinterpret_cast<const f32x4*>(sp + col);
        av += *reinterpret_cast<const f32x4*>(sp + kMaxSinks * DP + col);
      }
      if constexpr (CUT) {
        *reinterpret_cast<f32x4*>(share + col) = ak;
        *reinterpret_cast<f32x4*>(share + DP + col) = av;
        continue;
      }
      if (col >= a.D) continue;
      *reinterpret_cast<uint2*>(kd + col) =
          make_uint2(pack_bf16(ak[0] * a.scale, ak[1] * a.scale), pack_bf16(ak[2] * a.scale, ak[3] * a.scale));
      *reinterpret_cast<uint2*>(vd + col) = make_uint2(pack_bf16(av[0], av[1]), pack_bf16(av[2], av[3]));
    }
  }
  if (!CUT && b == a.B - 1) {
    zero_rows(a.dk, hk, sv.k0 + sv.Lk, a.Tk, a.D, x, nk);
    zero_rows(a.dv, hk, sv.k0 + sv.Lk, a.Tk, a.D, x, nk);
  }
}

// dk and dv from the parts' shares, in order. A workgroup takes 8 keys of a
// key head at a time.
template <int DP>
__global__ __launch_bounds__(256) void attn_dkv_join_kernel(AttnArgs a) {
  constexpr int C = DP / 4;  // groups of 4 columns
  const int hk = blockIdx.y, b = blockIdx.z;
  const SeqView sv = seq_view(a, b);
  for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < (int64_t)sv.Lk * 2 * C; e += (int64_t)gridDim.x * 256) {
    const int col = (int)(e % C) * 4, which = (int)(e / C & 1);
    const int64_t row = sv.k0 + e / (2 * C);
    if (col >= a.D) continue;
    const float* p = a.share + (row * a.Hkv + hk) * (2 * DP) + which * DP + col;
    const int64_t step = a.Tk * a.Hkv * (2 * DP);
    f32x4 acc = *reinterpret_cast<const f32x4*>(p);
#pragma unroll 4
    for (int i = 1; i < a.parts; ++i) acc += *reinterpret_cast<const f32x4*>(p + i * step);
    if (which == 0) acc *= a.scale;
    const AttnTensor& t = which ? a.dv : a.dk;
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(t.p) + row * t.st + hk * t.sh + col) =
        make_uint2(pack_bf16(acc[0], acc[1]), pack_bf16(acc[2], acc[3]));
  }
  if (b == a.B - 1) {
    zero_rows(a.dk, hk, sv.k0 + sv.Lk, a.Tk, a.D, blockIdx.x, gridDim.x);
    zero_rows(a.dv, hk, sv.k0 + sv.Lk, a.Tk, a.D, blockIdx.x, gridDim.x);
  }
}

// ---------------------------------------------------------------------------
// first tokens, far queries
// ---------------------------------------------------------------------------
// Row range r of a sequence: `span` rows from far + r span. Shares are
// numbered slot = floor(cu_q[b] / span) + b + r, below Tq / span + B, per
// query head: float32 [slot][H][2][32][DP].
template <int DP>
__global__ __launch_bounds__(64 * kSinkWaves) void attn_sink_kernel(AttnArgs a, int nr, int span, float* share, UnitGrid ug) {
  extern __shared__ __align__(16) uint16_t lds[];
  const UnitItem ui = unit_item(ug);
  if (ui.item < 0) return;
  const int tid = threadIdx.x, l = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int group = a.H / a.Hkv;
  const int b = ui.unit / a.Hkv, hk = ui.unit % a.Hkv, hq = hk * group + ui.item % group, x = ui.item / group;
  const SeqView sv = seq_view(a, b);
  const float c = a.scale * kAttnLog2e;
  const int shift = sv.Lk - sv.Lq;
  const LaneOffsets lofs = lane_offsets16<DP>(l);
  const TileLoad<DP, kSinkWaves> load_q(a.q.st, a.D, w, l), load_g(a.d_o.st, a.D, w, l);
  const int far = far_row(sv, a.window);
  const int key = 16 * (w & 1) + (l & 15);  // two waves share a tile, one for each half of the keys
  const int64_t slot0 = sv.q0 / span + b;
  for (int y = x; (int64_t)far + (int64_t)y * span < sv.Lq; y += nr) {
    const int beg = far + y * span, end = min(sv.Lq, beg + span);
    DkvState<DP> st;
    load_keys<DP>(a, sv, hk, key, st, l);
    // 256 rows at a time, in 4 stages
    for (int i0 = beg; i0 < end; i0 += 256) {
#pragma unroll
      for (int t = 0; t < 4; ++t)
        load_queries<DP, kSinkWaves>(a, sv, load_q, load_g, hq, min(i0 + 64 * t, sv.Lq - 1), lds + t * kStage<DP, kSinkWaves>, w, l);
      wait_vm<0>();
      __builtin_amdgcn_s_barrier();
      const int i = i0 + 64 * (w >> 1);
      const int rows = min(64, end - i);
      if (rows > 0) {
        const uint16_t* t = lds + (w >> 1) * kStage<DP, kSinkWaves>;
        const float* ls = reinterpret_cast<const float*>(t + 128 * DP);
        // the sinks alone: a window of 0 hides every other key
        dkv_tile<DP>(t, t + 64 * DP, ls, ls + 64, st, i + shift, rows, key, 0, min(a.sinks, sv.Lk), c, lofs, l);
      }
      __builtin_amdgcn_s_barrier();
    }
    // the four stages' sums, in order
    float* f = reinterpret_cast<float*>(lds);
    float* out = share + ((slot0 + y) * a.H + hq) * (2 * kMaxSinks * DP);
#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
#pragma unroll
      for (int d = 0; d < DP / 16; ++d)
        *reinterpret_cast<f32x4*>(f + ((w >> 1) * 32 + key) * DP + 16 * d + 4 * (l >> 4)) = which ? st.dv[d] : st.dk[d];
      __syncthreads();
      for (int e = tid; e < 32 * DP; e += 64 * kSinkWaves)
        out[which * kMaxSinks * DP + e] = (f[e] + f[32 * DP + e]) + (f[2 * 32 * DP + e] + f[3 * 32 * DP + e]);
      __syncthreads();
    }
  }
}

// sink [B][Hkv][2][32][DP] = sum over the row ranges and the group's heads, in
// order (8 shares at a time on their way); the first tokens' rows only.
template <int DP>
__global__ __launch_bounds__(256) void attn_sink_join_kernel(AttnArgs a, int span, const float* share, float* sink) {
  const int hk = blockIdx.y, b = blockIdx.z;
  const int e = blockIdx.x * 256 + threadIdx.x;  // < 2 x 32 x DP
  if (e / DP % kMaxSinks >= a.sinks) return;
  const SeqView sv = seq_view(a, b);
  const int group = a.H / a.Hkv;
  const int far = far_row(sv, a.window);
  const int64_t slot0 = sv.q0 / span + b;
  const int n = (sv.Lq > far ? (sv.Lq - far + span - 1) / span : 0) * group;
  const float* p = share + (slot0 * a.H + hk * group) * (2 * kMaxSinks * DP) + e;
  float acc = 0.f;
  for (int u0 = 0; u0 < n; u0 += 8) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int u = min(u0 + i, n - 1);
      v[i] = p[((int64_t)(u / group) * a.H + u % group) * (2 * kMaxSinks * DP)];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (u0 + i < n) acc += v[i];
  }
  sink[((int64_t)b * a.Hkv + hk) * (2 * kMaxSinks * DP) + e] = acc;
}

template <int DP, int NS, bool CUT>
hipError_t run_dkv(const AttnArgs& a, const float* joined, hipStream_t s) {
  static std::atomic<uint32_t> done{0};
  const int bytes = NS * kDkvStages * kStage<DP, kKeyWaves> * 2;
  const hipError_t e = ensure_lds(reinterpret_cast<const void*>(attn_dkv_kernel<DP, NS, CUT>), bytes, done);
  if (e != hipSuccess) return e;
  const int64_t longest = a.max_k < a.Tk ? a.max_k : a.Tk;
  const int64_t units = (int64_t)a.B * a.Hkv, blocks = (longest + kKeys - 1) / kKeys;
  const int64_t parts = CUT ? a.parts : 1;
  const int nk = fit_groups(block_groups(blocks, blocks * units, 4), units, parts, 64 * kKeyWaves * NS);
  const UnitGrid ug(units, nk * parts);
  hipLaunchKernelGGL((attn_dkv_kernel<DP, NS, CUT>), ug.grid(), dim3(64 * kKeyWaves * NS), bytes, s, a, nk, joined, ug);
  const hipError_t le = hipGetLastError();
  if (le != hipSuccess || !CUT) return le;
  const int64_t join = (longest * 2 * (DP / 4) + 255) / 256;
  hipLaunchKernelGGL((attn_dkv_join_kernel<DP>), dim3((unsigned)join, a.Hkv, a.B), dim3(256), 0, s, a);
  return hipGetLastError();
}

template <int DP>
hipError_t run_bwd(const AttnArgs& a, hipStream_t s) {
  static std::atomic<uint32_t> done[2] = {{0}, {0}};
  const int dq_bytes = 4 * 64 * DP * 2;
  const int sink_bytes = 4 * kStage<DP, kSinkWaves> * 2;  // (more than the 4 x 32 x DP sums)
  hipError_t e = ensure_lds(reinterpret_cast<const void*>(attn_dq_kernel<DP>), dq_bytes, done[0]);
  if (e == hipSuccess) e = ensure_lds(reinterpret_cast<const void*>(attn_sink_kernel<DP>), sink_bytes, done[1]);
  if (e != hipSuccess) return e;
  const int64_t units = (int64_t)a.B * a.Hkv, group = a.H / a.Hkv;
  const int64_t bq = (a.max_q + kRows - 1) / kRows;
  const int nq = fit_groups(block_groups(bq, bq * units * group, 2), units, group, 256);
  const UnitGrid uq(units, nq * group);
  hipLaunchKernelGGL((attn_dq_kernel<DP>), uq.grid(), dim3(256), dq_bytes, s, a, nq, uq);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  float* joined = nullptr;
  if (attn_sink_apart(a.max_k, a.window, a.sinks)) {
    const int span = attn_sink_span(a.max_q);
    const int nr = fit_groups((a.max_q + span - 1) / span, units, group, 64 * kSinkWaves);
    float* share = a.sink;
    joined = share + attn_sink_slots(a.Tq, a.B, a.max_q) * a.H * (2 * kMaxSinks * DP);
    const UnitGrid ur(units, nr * group);
    hipLaunchKernelGGL((attn_sink_kernel<DP>), ur.grid(), dim3(64 * kSinkWaves), sink_bytes, s, a, nr, span, share, ur);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((attn_sink_join_kernel<DP>), dim3(2 * kMaxSinks * DP / 256, a.Hkv, a.B), dim3(256), 0, s, a,
                       span, share, joined);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  // Too many key blocks for parts of their own and too few to keep every compute
  // unit busy to the end: two streams (800 blocks of uneven sequences, heads of
  // 64: 261 -> 242 us, of 128: 420 -> 400; from 1032 blocks on it is 5 to 20 %
  // slower).
  if (a.parts > 1) return run_dkv<DP, 1, true>(a, joined, s);
  if (attn_key_blocks(a.Tk, a.B, a.Hkv) < 1024) return run_dkv<DP, 2, false>(a, joined, s);
  return run_dkv<DP, 1, false>(a, joined, s);
}

}  // namespace

hipError_t launch_attn_bwd(const AttnArgs& a, hipStream_t s) {
  return a.D <= 64 ? run_bwd<64>(a, s) : run_bwd<128>(a, s);
}

}  // namespace qlora
