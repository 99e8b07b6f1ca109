// Attention with a sliding window and first tokens that stay visible:
// forward pass over packed sequences.
//
//   s_ij = scale q_i . k_j over the keys that query i sees (attn.hpp)
//   lse_i = log sum_j exp(s_ij),  o_i = sum_j exp(s_ij - lse_i) v_j
// A query that sees no key gives o = 0 and lse = -inf.
//
// A workgroup of NW waves takes 32 NW queries of one head, a wave 32 of them;
// key and value tiles of 64 rows pass through LDS by LDS-DMA, NS stages, and
// each wave keeps the running maximum and sum of its queries (one pass, the
// sum over float32 probabilities) and its 32 x D result in registers. Only
// the tiles that hold visible keys are visited, and only those at an edge of
// the visible range are masked.
//
// Bound, long rows: no pipe is full. 8192 queries, window 4096, 32 heads of 128:
// 494 us, 834 TFLOP/s (a loop of the same products and exponentials, without
// loads or barriers, reached 1050 to 1175, a large product 1336); the matrix
// pipe is busy 38 % of the time, vector instructions issue in 38 % of it, LDS is
// read in 19 %, and 84 % of the compute units hold work on average. What is left
// is softmax and products of a wave taking turns, with two waves a SIMD to
// overlap them, and the last round of workgroups: with 1056 of them for 512 places
// (4097 queries after prefixes of 4095, 32 heads on 8, window 4096: 351 to 360 us,
// 780 TFLOP/s) matrix 35 %, vector 35 %, compute units 76 %.
// Short rows: HBM and the way to the first tile (16 x 512 tokens, 32 heads of 128,
// window 256: 92 us for 268 MB, matrix 14 %).
// 4 waves, two stages (64 KB) and two workgroups on a compute unit: 8 waves with
// three or four stages were slower, as was a form in which two halves of a
// workgroup take turns at the matrix pipe.
#include "attn.hpp"

namespace qlora {
namespace {

template <int DP>
struct FwdState {
  bf16x8 q[DP / 16];
  f32x16 o[DP / 32];
  float m, sum;  // reference maximum (raw score units), this lane's share of the sum
};

// The reference maximum follows a tile's scores when it falls 8 or more behind
// (in base-2 exponent): p stays below 2^8, and most tiles rescale nothing.
template <int DP>
__device__ __forceinline__ void follow_max(FwdState<DP>& st, const f32x16 (&s)[2], float c) {
  float top = s[0][0];
#pragma unroll
  for (int b = 0; b < 2; ++b)
#pragma unroll
    for (int r = 0; r < 16; ++r) top = fmaxf(top, s[b][r]);
  top = half_max(top);
  const bool grow = (top - st.m) * c > 8.f || (st.m == -__builtin_inff() && top > st.m);
  if (__any(grow)) {
    const float m = grow ? top : st.m;
    const float f = grow ? fast_exp2((st.m - m) * c) : 1.f;
    st.m = m;
    st.sum *= f;
#pragma unroll
    for (int d = 0; d < DP / 32; ++d)
#pragma unroll
      for (int r = 0; r < 16; ++r) st.o[d][r] *= f;
  }
}

// Result and lse of the lane's query.
template <int DP>
__device__ __forceinline__ void store_rows(const AttnArgs& a, const FwdState<DP>& st, const SeqView& sv, int hq, int iq,
                                           int l) {
  const float total = half_sum(st.sum);
  const float inv = total > 0.f ? 1.f / total : total;  // 0: nothing seen; NaN stays
  if (l < 32)
    a.lse[(int64_t)hq * a.Tq + sv.q0 + iq] = total == 0.f ? -__builtin_inff() : st.m * a.scale + __builtin_logf(total);
  uint16_t* op = static_cast<uint16_t*>(a.o.p) + (sv.q0 + iq) * a.o.st + hq * a.o.sh;
#pragma unroll
  for (int d = 0; d < DP / 32; ++d)
#pragma unroll
    for (int r = 0; r < 16; r += 4) {
      const int col = 32 * d + block_row(r, l >> 5);
      if (col < a.D)
        *reinterpret_cast<uint2*>(op + col) = make_uint2(pack_bf16(st.o[d][r] * inv, st.o[d][r + 1] * inv),
                                                         pack_bf16(st.o[d][r + 2] * inv, st.o[d][r + 3] * inv));
    }
}

// One key tile. kt, vt: this stage's tiles (restrict: the reads below do not
// touch the stage that the LDS-DMA in flight fills). EDGE: some pairs are
// hidden. The scheduling fences keep the fragment reads two groups of products
// ahead (the first two groups of values ahead of the softmax); without them
// each read was waited for just before its product.
template <int DP>
__device__ __forceinline__ void fwd_tile(const uint16_t* __restrict__ kt, const uint16_t* __restrict__ vt,
                                         FwdState<DP>& st, int j0, int pos, bool edge, int window, int sinks, float c, LaneOffsets lo,
                                         int l) {
  constexpr int KS = DP / 16, DB = DP / 32;
  constexpr int G = DB;           // fragments of a group
  constexpr int NK = 2 * KS / G;  // groups of the scores: 4
  bf16x8 f[3][G];                 // groups in flight
  auto read_k = [&](int g) {
#pragma unroll
    for (int i = 0; i < G; ++i) {
      const int n = g * G + i;
      f[g % 3][i] = row_frag<DP>(kt, 32 * (n / KS), n % KS, lo);
    }
  };
  auto read_v = [&](int g) {  // 16 rows of the value tile
#pragma unroll
    for (int i = 0; i < G; ++i) f[(g + NK) % 3][i] = col_frag<DP>(vt, 16 * g, i, lo);
  };
  read_k(0);
  read_k(1);
  f32x16 s[2] = {zero16(), zero16()};
#pragma unroll
  for (int g = 0; g < NK; ++g) {
    __builtin_amdgcn_sched_barrier(0);
    if (g + 2 < NK) read_k(g + 2);
    else read_v(g + 2 - NK);
#pragma unroll
    for (int i = 0; i < G; ++i) {
      const int n = g * G + i;
      s[n / KS] = mfma32(f[g % 3][i], st.q[n % KS], s[n / KS]);
    }
  }
  __builtin_amdgcn_sched_barrier(0);
  if (edge) {
    hide_keys(s[0], -__builtin_inff(), j0, pos, window, sinks, l);
    hide_keys(s[1], -__builtin_inff(), j0 + 32, pos, window, sinks, l);
  }
  follow_max<DP>(st, s, c);
  const float mc = st.m == -__builtin_inff() ? 0.f : st.m * c;
#pragma unroll
  for (int b = 0; b < 2; ++b)
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      s[b][r] = fast_exp2(__builtin_fmaf(s[b][r], c, -mc));
      st.sum += s[b][r];
    }
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    __builtin_amdgcn_sched_barrier(0);
    if (g + 2 < 4) read_v(g + 2);
    const bf16x8 p = pack_frag(s[g / 2], g % 2);
#pragma unroll
    for (int d = 0; d < DB; ++d) st.o[d] = mfma32(f[(g + NK) % 3][d], p, st.o[d]);
  }
}

template <int DP, int NW, int NS>
__global__ __launch_bounds__(64 * NW, 2) void attn_fwd_kernel(AttnArgs a, int nq, UnitGrid ug) {
  extern __shared__ __align__(16) uint16_t lds[];
  constexpr int kTile = 64 * DP, kQRows = 32 * NW;
  using Load = TileLoad<DP, NW>;
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
  const LaneOffsets lo = lane_offsets<DP>(l);
  const Load load_k(a.k.st, a.D, w, l), load_v(a.v.st, a.D, w, l);

  // later blocks see more keys: they start first
  const int blocks = (sv.Lq + kQRows - 1) / kQRows;
  for (int y = blocks - 1 - x; y >= 0; y -= nq) {
    const int i0 = y * kQRows, i1 = min(i0 + kQRows, sv.Lq) - 1;  // queries of the workgroup
    const int wi0 = i0 + 32 * w, wi1 = min(wi0 + 31, sv.Lq - 1);  // of the wave (wi1 < wi0: none)
    const int iq = wi0 + (l & 31);
    const bool have = iq < sv.Lq;
    const int pos = iq + shift;
    const TileWalk walk(i0 + shift, i1 + shift, wi0 + shift, wi1 + shift, sv.Lk, a.window, a.sinks);
    TileSource src_k(kp, a.k.st, walk), src_v(vp, a.v.st, walk);
    int last = sv.Lk - 1 - 64 * walk.tile(0);  // of the tile asked for next
    auto issue = [&](int i) {
      uint16_t* dst = lds + (i % NS) * 2 * kTile;
      load_k(src_k.p, last, dst, w);
      load_v(src_v.p, last, dst + kTile, w);
      src_k.next(i, walk);
      src_v.next(i, walk);
      last -= i + 1 == walk.first ? walk.jump : 64;
    };
#pragma unroll
    for (int i = 0; i < NS - 1; ++i)
      if (i < walk.n) issue(i);
    const uint16_t* qp = static_cast<const uint16_t*>(a.q.p) + (sv.q0 + (have ? iq : 0)) * a.q.st + hq * a.q.sh;
    FwdState<DP> st;
#pragma unroll
    for (int ks = 0; ks < DP / 16; ++ks) st.q[ks] = global_frag(qp, have, a.D, ks, l);
#pragma unroll
    for (int d = 0; d < DP / 32; ++d) st.o[d] = zero16();
    st.m = -__builtin_inff();
    st.sum = 0.f;
    // Everything so far has to be there: otherwise the compiler, which cannot
    // tell the queries' loads from the tiles' in flight, waits for all of them
    // in every pass of the loop.
    wait_vm<0>();
    // one pass per stage, so that the stage's place in LDS is a constant
    for (int t0 = 0; t0 < walk.n; t0 += NS) {
#pragma unroll
      for (int u = 0; u < NS; ++u) {
        const int i = t0 + u;
        if (i >= walk.n) break;
        // this tile's DMA has landed, and every wave is done with the stage of
        // tile i - 1, which tile i + NS - 1 takes
        wait_tile<2 * Load::NI, NS - 2>(i, walk.n);
        __builtin_amdgcn_s_barrier();
        if (i + NS - 1 < walk.n) issue(i + NS - 1);
        const int t = walk.tile(i);
        if (walk.hidden(t)) continue;
        const uint16_t* kt = lds + u * 2 * kTile;
        fwd_tile<DP>(kt, kt + kTile, st, 64 * t, min(pos, sv.Lk - 1), walk.edge(t), a.window, a.sinks, c, lo, l);
      }
    }
    __builtin_amdgcn_s_barrier();  // the tiles are free for the next block

    if (have) store_rows<DP>(a, st, sv, hq, iq, l);
  }
  if (b == a.B - 1) {  // rows past the last sequence see nothing
    const int64_t rest = sv.q0 + sv.Lq;
    zero_rows(a.o, hq, rest, a.Tq, a.D, x, nq);
    for (int64_t r = rest + x * blockDim.x + tid; r < a.Tq; r += nq * blockDim.x)
      a.lse[(int64_t)hq * a.Tq + r] = -__builtin_inff();
  }
}

template <int DP, int NW, int NS>
hipError_t run_fwd(const AttnArgs& a, hipStream_t s) {
  static std::atomic<uint32_t> done{0};
  const int bytes = NS * 2 * 64 * DP * 2;
  hipError_t e = ensure_lds(reinterpret_cast<const void*>(attn_fwd_kernel<DP, NW, NS>), bytes, done);
  if (e != hipSuccess) return e;
  const int64_t blocks = (a.max_q + 32 * NW - 1) / (32 * NW);
  const int64_t units = (int64_t)a.B * a.Hkv, group = a.H / a.Hkv;
  const int nq = fit_groups(block_groups(blocks, blocks * a.B * a.H, 2), units, group, 64 * NW);
  const UnitGrid ug(units, nq * group);
  hipLaunchKernelGGL((attn_fwd_kernel<DP, NW, NS>), ug.grid(), dim3(64 * NW), bytes, s, a, nq, ug);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_attn_fwd(const AttnArgs& a, hipStream_t s) {
  return a.D <= 64 ? run_fwd<64, 4, 2>(a, s) : run_fwd<128, 4, 2>(a, s);
}

}  // namespace qlora
