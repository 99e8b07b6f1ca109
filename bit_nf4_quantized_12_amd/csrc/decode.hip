// Attention of one new token per request over a key/value cache, with a
// sliding window and first tokens that stay visible.
//
// Request b holds n = lens[b] positions; its query stands at n - 1 and sees
// the first min(sinks, n) and the last min(window, n) of them:
//   o = sum_j exp(s_j - lse) v_j,  s_j = scale q . k_j        (n = 0: o = 0)
// The cache is read once per key head: up to 16 query heads that share a key
// head are the columns of the score product, S^T (keys x heads) = K Q^T, on
// v_mfma_f32_16x16x32_bf16, and the same lanes' probabilities are the right
// operand of O^T += V^T P^T (see attn.hpp for the order of the keys). Keys go
// from memory to registers, values by LDS-DMA to each wave's own LDS (read
// transposed), so the waves of a workgroup meet only once, at the end.
// HBM bound: 4 D bytes per key and key head (16 requests, 32 key heads of 128, up to
// 516 visible keys: 25.4 us, 4.7 TB/s; 3 requests over up to 64 K tokens, 8 key
// heads: 95.7 us, 5.13 TB/s; a large copy reaches 4.95). The visible keys of a request
// are cut into `nsplit` equal parts so that few requests fill the GPU; a
// second kernel joins the parts (none is needed for one part).
#include "attn.hpp"
#include "reduce.hpp"

namespace qlora {
namespace {

constexpr int kStep = 32;  // keys per wave and step
constexpr int kMaxD = 128;

// Row pitch of the cache in bytes may exceed 32 bits over a long cache: row
// addresses are 64-bit.
template <int DP>
__global__ __launch_bounds__(256) void decode_kernel(DecodeArgs a) {
  constexpr int CH = DP / 8;
  constexpr int NDB = DP / 16;
  extern __shared__ __align__(16) uint16_t lds[];
  const int tid = threadIdx.x, l = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int split = blockIdx.x % a.nsplit;
  const int hk = blockIdx.x / a.nsplit % a.Hkv;
  const int hb = blockIdx.y;  // block of 16 query heads of the group
  const int b = blockIdx.x / a.nsplit / a.Hkv;
  const int group = a.H / a.Hkv;
  const int heads = min(16, group - 16 * hb);
  const int h0 = hk * group + 16 * hb;

  const int n = min(max(a.lens[b], 0), a.cap);
  const int lo = max(0, n - a.window);
  const int first = min(a.sinks, lo);  // sinks in front of the window
  const int total = first + n - lo;    // visible keys
  int chunk = (total + a.nsplit - 1) / a.nsplit;
  chunk = (chunk + 4 * kStep - 1) / (4 * kStep) * (4 * kStep);
  // (of nearly 2^31 positions, the last part's own end would pass 2^31)
  const int beg = min(total, split * chunk), end = beg + min(total - beg, chunk);

  const uint16_t* kp = a.k + b * a.k_sb + hk * a.k_sh;
  const uint16_t* vp = a.v + b * a.v_sb + hk * a.v_sh;
  // visible place -> cache position; places past the part's end repeat its
  // last key (their probabilities are zero), so only filled rows are read
  auto position = [&](int place) {
    const int p = min(place, end - 1);
    return (int64_t)(p < first ? p : lo + p - first);
  };

  const float c = a.scale * kAttnLog2e;
  const int hq = l & 15, kg = l >> 4;
  bf16x8 q[DP / 32];
#pragma unroll
  for (int ks = 0; ks < DP / 32; ++ks) {
    const int col = 32 * ks + 8 * kg;
    q[ks] = __builtin_bit_cast(bf16x8, make_uint4(0, 0, 0, 0));
    if (hq < heads && col < a.D)
      q[ks] = *reinterpret_cast<const bf16x8*>(a.q + b * a.q_sb + (h0 + hq) * a.q_sh + col);
  }
  f32x4 o[NDB];
#pragma unroll
  for (int d = 0; d < NDB; ++d) o[d] = f32x4{0.f, 0.f, 0.f, 0.f};
  float m = -__builtin_inff(), sum = 0.f;

  uint16_t* vt = lds + w * 2 * kStep * DP;  // this wave's two value stages
  bf16x8 kr[2][DP / 32];
  auto fetch_k = [&](int place) {
#pragma unroll
    for (int blk = 0; blk < 2; ++blk) {
      const uint16_t* row = kp + position(place + 16 * blk + (l & 15)) * a.k_st;
#pragma unroll
      for (int ks = 0; ks < DP / 32; ++ks)
        kr[blk][ks] = *reinterpret_cast<const bf16x8*>(row + min(32 * ks + 8 * kg, a.D - 8));
    }
  };
  auto fetch_v = [&](int place, uint16_t* dst) {
#pragma unroll
    for (int i = 0; i < kStep * CH / 64; ++i) {
      const int r = i * (64 / CH) + l / CH;
      const int ch = min((l % CH) ^ tile_swz<DP>(r), a.D / 8 - 1);
      const uint16_t* src = vp + position(place + r) * a.v_st + 8 * ch;
      __builtin_amdgcn_global_load_lds((gbl_void_t*)src, (lds_void_t*)(dst + i * 512), 16, 0, 0);
    }
  };

  int place = beg + kStep * w;
  if (place < end) {
    fetch_k(place);
    fetch_v(place, vt);
  }
  for (int i = 0; place < end; ++i, place += 4 * kStep) {
    f32x4 s[2];
#pragma unroll
    for (int blk = 0; blk < 2; ++blk) {
      s[blk] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int ks = 0; ks < DP / 32; ++ks) s[blk] = mfma16(kr[blk][ks], q[ks], s[blk]);
    }
    const uint16_t* vs = vt + (i & 1) * kStep * DP;
    // this step's values have landed; the next step's loads follow
    __builtin_amdgcn_s_waitcnt(0);
    __builtin_amdgcn_sched_barrier(0);
    if (place + 4 * kStep < end) {
      fetch_k(place + 4 * kStep);
      fetch_v(place + 4 * kStep, vt + ((i + 1) & 1) * kStep * DP);
    }
    float top = -__builtin_inff();
#pragma unroll
    for (int blk = 0; blk < 2; ++blk)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        if (place + 16 * blk + 4 * kg + r >= end) s[blk][r] = -__builtin_inff();
        top = fmaxf(top, s[blk][r]);
      }
    top = fmaxf(top, __shfl_xor(top, 16));
    top = fmaxf(top, __shfl_xor(top, 32));
    if (__any(top > m)) {
      const float mn = fmaxf(m, top);
      const float f = mn == -__builtin_inff() ? 1.f : fast_exp2((m - mn) * c);
      m = mn;
      sum *= f;
#pragma unroll
      for (int d = 0; d < NDB; ++d)
#pragma unroll
        for (int r = 0; r < 4; ++r) o[d][r] *= f;
    }
    const float mc = m == -__builtin_inff() ? 0.f : m * c;
#pragma unroll
    for (int blk = 0; blk < 2; ++blk)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        s[blk][r] = fast_exp2(__builtin_fmaf(s[blk][r], c, -mc));
        sum += s[blk][r];
      }
    // probabilities as a sum of two bf16, 16 bits of them: the second product
    // costs nothing here, where the matrix pipe waits for the cache
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float p0 = s[i / 2][i % 2 * 2], p1 = s[i / 2][i % 2 * 2 + 1];
      hi[i] = pack_bf16(p0, p1);
      lo[i] = pack_bf16(p0 - bf16lo(hi[i]), p1 - bf16hi(hi[i]));
    }
    const bf16x8 p = __builtin_bit_cast(bf16x8, make_uint4(hi[0], hi[1], hi[2], hi[3]));
    const bf16x8 pr = __builtin_bit_cast(bf16x8, make_uint4(lo[0], lo[1], lo[2], lo[3]));
    // lane (kg, x): rows 4 kg + (x >> 2) and + 16, columns 16 d + 4 (x & 3)
    const int x = l & 15, R = 4 * kg + (x >> 2);
#pragma unroll
    for (int d = 0; d < NDB; ++d) {
      const int col = 16 * d + 4 * (x & 3);
      const uint16_t* p0 = vs + R * DP + 8 * ((col >> 3) ^ tile_swz<DP>(R)) + (col & 7);
      const uint16_t* p1 = vs + (R + 16) * DP + 8 * ((col >> 3) ^ tile_swz<DP>(R + 16)) + (col & 7);
      const uint2 v0 = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s_t*)p0));
      const uint2 v1 = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s_t*)p1));
      const bf16x8 vf = __builtin_bit_cast(bf16x8, make_uint4(v0.x, v0.y, v1.x, v1.y));
      o[d] = mfma16(vf, pr, mfma16(vf, p, o[d]));
    }
  }
  // join the four waves: sums and maxima, then the results (LDS is reused)
  sum += __shfl_xor(sum, 16);
  sum += __shfl_xor(sum, 32);
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
  float* f = reinterpret_cast<float*>(lds);  // [4][16] maxima, [4][16] sums, [4][16][DP + 4] results
  float* fo = f + 128;
  if (l < 16) {
    f[w * 16 + l] = m;
    f[64 + w * 16 + l] = sum;
  }
#pragma unroll
  for (int d = 0; d < NDB; ++d)
    *reinterpret_cast<f32x4*>(fo + (w * 16 + hq) * (DP + 4) + 16 * d + 4 * kg) = o[d];
  __syncthreads();
  const int64_t unit = ((int64_t)b * a.H + h0) * a.nsplit + split;
  for (int e = tid; e < heads * (DP / 4); e += 256) {
    const int h = e / (DP / 4), col = e % (DP / 4) * 4;
    float mm = f[h];
#pragma unroll
    for (int i = 1; i < 4; ++i) mm = fmaxf(mm, f[i * 16 + h]);
    float ss = 0.f;
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float mi = f[i * 16 + h];
      const float g = mi == -__builtin_inff() ? (f[64 + i * 16 + h] == 0.f ? 0.f : 1.f) : fast_exp2((mi - mm) * c);
      ss += g * f[64 + i * 16 + h];
      const f32x4 v = *reinterpret_cast<const f32x4*>(fo + (i * 16 + h) * (DP + 4) + col);
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[r] += g * v[r];
    }
    if (col >= a.D) continue;
    if (a.nsplit == 1) {
      const float inv = ss == 0.f ? 0.f : 1.f / ss;
      uint16_t* op = a.o + (b * (int64_t)a.H + h0 + h) * a.D + col;
      *reinterpret_cast<uint2*>(op) =
          make_uint2(pack_bf16(acc[0] * inv, acc[1] * inv), pack_bf16(acc[2] * inv, acc[3] * inv));
    } else {
      const int64_t at = unit + (int64_t)h * a.nsplit;
      *reinterpret_cast<f32x4*>(a.part + at * a.D + col) = acc;
      if (col == 0) {
        a.stat[2 * at] = mm;
        a.stat[2 * at + 1] = ss;
      }
    }
  }
}

// o of one head from its parts: lane i of every wave holds part i's weight
// (at most 64 parts). Wave w adds the parts 8 t + 2 w in its lower half and
// 8 t + 2 w + 1 in its upper half, t = 0, 1, ...; lane l & 31 of a half holds 4
// columns. The halves, then the waves, are added in order. Every lane runs every
// step, with columns or without: a lane that is switched off gives no weight.
// Steps past the last part repeat it with weight 0 (and the value 0, so that
// no infinity is multiplied by it).
__global__ __launch_bounds__(256) void decode_join_kernel(DecodeArgs a) {
  __shared__ f32x4 f[4][kMaxD / 4];
  const int64_t bh = blockIdx.x;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = threadIdx.x & 63;
  const float* st = a.stat + bh * 2 * a.nsplit;
  const bool in = l < a.nsplit;
  const float mi = in ? st[2 * l] : -__builtin_inff(), si = in ? st[2 * l + 1] : 0.f;
  const float m = wave_max(mi);
  const float g = mi == -__builtin_inff() ? (si == 0.f ? 0.f : 1.f) : fast_exp2((mi - m) * a.scale * kAttnLog2e);
  const float sum = wave_sum(g * si);
  const int cols = a.D / 4;  // at most 32
  const int half = l >> 5, col = l & 31;
  const float* p = a.part + bh * a.nsplit * a.D + 4 * min(col, cols - 1);
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  constexpr int U = 4;  // parts of a lane on their way together
  for (int i0 = 2 * w; i0 < a.nsplit; i0 += 8 * U) {  // (the same steps in all lanes of a wave)
    f32x4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = *reinterpret_cast<const f32x4*>(p + (int64_t)min(i0 + half + 8 * u, a.nsplit - 1) * a.D);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + half + 8 * u;
      const bool ok = i < a.nsplit;
      const float from = __shfl(g, i & 63);  // (outside of the choice)
      const float gi = ok ? from : 0.f;
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[r] = __builtin_fmaf(gi, ok ? v[u][r] : 0.f, acc[r]);
    }
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) acc[r] += __shfl_xor(acc[r], 32);
  if (half == 0) f[w][col] = acc;
  __syncthreads();
  if (w != 0 || half != 0 || col >= cols) return;
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  f32x4 o = f[0][col];
#pragma unroll
  for (int i = 1; i < 4; ++i) o += f[i][col];
  *reinterpret_cast<uint2*>(a.o + bh * a.D + 4 * col) =
      make_uint2(pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv));
}

template <int DP>
hipError_t run_decode(const DecodeArgs& a, hipStream_t s) {
  static std::atomic<uint32_t> done{0};
  constexpr int stages = 4 * 2 * kStep * DP * 2, joined = (128 + 4 * 16 * (DP + 4)) * 4;
  const int bytes = stages > joined ? stages : joined;
  hipError_t e = ensure_lds(reinterpret_cast<const void*>(decode_kernel<DP>), bytes, done);
  if (e != hipSuccess) return e;
  const int group = a.H / a.Hkv;
  hipLaunchKernelGGL((decode_kernel<DP>), dim3((unsigned)(a.B * a.Hkv * a.nsplit), (unsigned)((group + 15) / 16)),
                     dim3(256), bytes, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_decode(const DecodeArgs& a, hipStream_t s) {
  const hipError_t e = a.D <= 64 ? run_decode<64>(a, s) : run_decode<128>(a, s);
  if (e != hipSuccess || a.nsplit == 1) return e;
  hipLaunchKernelGGL(decode_join_kernel, dim3((unsigned)(a.B * a.H)), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace qlora
