// Layer norm of token rows, forward and backward.
//
// For a row x of C elements, with weight w and bias b:
//   mean = sum x / C,  rstd = 1 / sqrt(sum (x - mean)^2 / C + eps)
//   xh = (x - mean) rstd,  y = xh w + b
// and for the upstream gradient dy, with g = dy w:
//   dx = rstd (g - sum g / C - xh (sum g xh / C))
//   dw = sum over rows of dy xh,  db = sum over rows of dy
// A row sits in the registers of the threads that share it (TPR threads, NV
// vectors of VEC elements each), so x and dy are read once; the variance is
// the sum of the centred squares of those registers, not a difference of
// moments, and a large mean is corrected by what it leaves of them. All sums and the
// two saved statistics are float32; an output is rounded once, when it is stored.
//
// Bound: HBM; both directions touch each element once. At 8192 x 8192 bf16 the
// forward takes 54.2 us (268 MB, 4.95 TB/s, what a large copy reaches), the
// backward with dw and db 93 us (403 MB and the shares, 4.3 TB/s: 88 us for the
// rows, 5 for the shares' sum). One token of 4096: 2.7 us on the GPU, the call
// costs 11.6 on the host.
#include "launch.hpp"
#include "reduce.hpp"

namespace qlora {
namespace {

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<uint16_t>(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ uint16_t from_f32<uint16_t>(float v) {
  const __bf16 h = (__bf16)v;
  return __builtin_bit_cast(uint16_t, h);
}

// VEC consecutive elements as they lie in memory (16 bytes, or one element).
template <typename T, int VEC>
struct Pack {
  T v[VEC];
};
template <typename T, int VEC>
__device__ __forceinline__ Pack<T, VEC> load_pack(const T* p) {
  Pack<T, VEC> r;
  if constexpr (VEC * sizeof(T) == 16) {
    const u32x4 u = *reinterpret_cast<const u32x4*>(p);
    __builtin_memcpy(&r, &u, 16);
  } else if constexpr (VEC * sizeof(T) == 32) {
    const u32x4 u[2] = {reinterpret_cast<const u32x4*>(p)[0], reinterpret_cast<const u32x4*>(p)[1]};
    __builtin_memcpy(&r, &u, 32);
  } else if constexpr (VEC * sizeof(T) == 8) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    __builtin_memcpy(&r, &u, 8);
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) r.v[i] = p[i];
  }
  return r;
}
template <typename T, int VEC>
__device__ __forceinline__ void store_pack(T* p, const Pack<T, VEC>& r) {
  if constexpr (VEC * sizeof(T) == 16) {
    u32x4 u;
    __builtin_memcpy(&u, &r, 16);
    *reinterpret_cast<u32x4*>(p) = u;
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) p[i] = r.v[i];
  }
}

// Sum over the TPR threads of a row; `slot` is that call's own LDS, so one
// barrier is enough. Every thread adds the waves' sums in the same order.
template <int TPR, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float* slot) {
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = wave_sum(v[k]);
  if constexpr (TPR > 64) {
    constexpr int W = TPR / 64;
    const int w = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int k = 0; k < N; ++k) slot[k * W + w] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k) {
      float s = slot[k * W];
#pragma unroll
      for (int i = 1; i < W; ++i) s += slot[k * W + i];
      v[k] = s;
    }
  }
}

template <typename T, typename P, int VEC, int TPR, int NV>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void norm_fwd_kernel(
    const T* __restrict__ x, int64_t ldx, const P* __restrict__ w, const P* __restrict__ b, int64_t M, int C,
    float inv_c, float eps, T* __restrict__ y, float* __restrict__ mean, float* __restrict__ rstd) {
  constexpr int ROWS = TPR < 256 ? 256 / TPR : 1;
  __shared__ float red[2][2 * (TPR / 64)];
  const int t = threadIdx.x % TPR;
  const int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / TPR;
  if (row >= M) return;  // whole waves of a block without barriers (TPR = 64)
  const T* xr = x + row * ldx;
  Pack<T, VEC> px[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * TPR + t) * VEC;
    if (c < C) {
      px[i] = load_pack<T, VEC>(xr + c);
    } else {
#pragma unroll
      for (int k = 0; k < VEC; ++k) px[i].v[k] = from_f32<T>(0.f);
    }
  }
  float s[1] = {0.f};
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int k = 0; k < VEC; ++k) s[0] += to_f32<T>(px[i].v[k]);
  row_sum<TPR>(s, red[0]);
  const float mu = s[0] * inv_c;
  float q[2] = {0.f, 0.f};  // of the differences from mu: squares, and themselves
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if ((i * TPR + t) * VEC >= C) continue;
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      const float d = to_f32<T>(px[i].v[k]) - mu;
      q[0] = __builtin_fmaf(d, d, q[0]);
      q[1] += d;
    }
  }
  row_sum<TPR>(q, red[1]);
  // mu + dm is the mean, and x - mu - dm the centred value, without the rounding
  // of mu (its sum, 1 / C). That counts where values lie closer to the mean than
  // to zero; elsewhere the differences are themselves rounded, and mu is the
  // better mean (exact, often, for bf16).
  const float dm = q[0] * inv_c < mu * mu ? q[1] * inv_c : 0.f;
  float var = __builtin_fmaf(q[0], inv_c, -dm * dm);
  if (var < 0.f) var = 0.f;  // (by rounding, in rows of one value; NaN stays)
  const float rs = 1.0f / __builtin_sqrtf(var + eps);
  if (t == 0) {
    mean[row] = mu + dm;
    rstd[row] = rs;
  }
  T* yr = y + row * (int64_t)C;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * TPR + t) * VEC;
    if (c >= C) continue;
    const Pack<P, VEC> pw = load_pack<P, VEC>(w + c);
    Pack<P, VEC> pb;
    if (b) pb = load_pack<P, VEC>(b + c);
    Pack<T, VEC> o;
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      const float xh = (to_f32<T>(px[i].v[k]) - mu - dm) * rs;
      o.v[k] = from_f32<T>(__builtin_fmaf(xh, to_f32<P>(pw.v[k]), b ? to_f32<P>(pb.v[k]) : 0.f));
    }
    store_pack<T, VEC>(yr + c, o);
  }
}

// Workgroup g takes rows g, g + G, ... (times the rows it holds at once) and
// keeps its share of dw and db in registers, so a row's x and dy are read
// once for all three gradients; the next two rows are on their way while this
// one's two sums are joined. At the end the workgroup writes its float32
// shares, part [G][2][C], which norm_reduce_kernel adds in the order of g: the
// result does not change from run to run. G depends on M and C alone.
// dx may be dy: a row's dy is in registers before its dx is stored (and dx and dy
// are not declared apart).
template <typename T, typename P, int VEC, int TPR, int NV>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void norm_bwd_kernel(
    const T* __restrict__ x, int64_t ldx, const P* __restrict__ w, const T* dy, int64_t lddy,
    const float* __restrict__ mean, const float* __restrict__ rstd, int64_t M, int C, float inv_c,
    T* dx, float* __restrict__ part) {
  constexpr int ROWS = TPR < 256 ? 256 / TPR : 1;
  constexpr int W = TPR / 64;
  __shared__ float red[2][2 * W];
  __shared__ float join[ROWS > 1 ? (ROWS - 1) * TPR * NV * VEC * 2 : 1];
  const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  // What a thread of 1024 with 16 columns has no registers for: the weights
  // (read again for each row, from cache) and a second row in flight.
  constexpr bool kRoom = NV * VEC * TPR <= 8192;
  constexpr int D = kRoom ? 2 : 1;
  Pack<P, VEC> pw[NV];
  float aw[NV][VEC], ab[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * TPR + t) * VEC;
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      pw[i].v[k] = from_f32<P>(0.f);
      aw[i][k] = ab[i][k] = 0.f;
    }
    if (kRoom && c < C) pw[i] = load_pack<P, VEC>(w + c);
  }
  Pack<T, VEC> px[D][NV], pg[D][NV];
  float mu[D], rs[D];
  auto fetch = [&](int u, int64_t row) {
    if (row >= M) return;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + t) * VEC;
      if (c < C) {
        px[u][i] = load_pack<T, VEC>(x + row * ldx + c);
        pg[u][i] = load_pack<T, VEC>(dy + row * lddy + c);
      } else {
#pragma unroll
        for (int k = 0; k < VEC; ++k) px[u][i].v[k] = pg[u][i].v[k] = from_f32<T>(0.f);
      }
    }
    mu[u] = mean[row];
    rs[u] = rstd[row];
  };
  const int64_t step = (int64_t)gridDim.x * ROWS;
  auto work = [&](int u, int slot, int64_t row) {
    float xh[NV][VEC], g[NV][VEC];
    float s[2] = {0.f, 0.f};
    // past the row's end x, dy and w are zero, and so is what they add
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + t) * VEC;
      if (!kRoom && c < C) pw[i] = load_pack<P, VEC>(w + c);
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        const float d = to_f32<T>(pg[u][i].v[k]);
        xh[i][k] = (to_f32<T>(px[u][i].v[k]) - mu[u]) * rs[u];
        g[i][k] = d * to_f32<P>(pw[i].v[k]);
        s[0] += g[i][k];
        s[1] = __builtin_fmaf(g[i][k], xh[i][k], s[1]);
      }
    }
    if (part != nullptr) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          const float d = to_f32<T>(pg[u][i].v[k]);
          aw[i][k] = __builtin_fmaf(d, xh[i][k], aw[i][k]);
          ab[i][k] += d;
        }
    }
    const float rsc = rs[u];
    fetch(u, row + D * step);
    if (dx == nullptr) return;
    row_sum<TPR>(s, red[slot]);
    const float a = s[0] * inv_c * rsc, bb = s[1] * inv_c * rsc;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + t) * VEC;
      if (c >= C) continue;
      Pack<T, VEC> o;
#pragma unroll
      for (int k = 0; k < VEC; ++k) o.v[k] = from_f32<T>(__builtin_fmaf(-xh[i][k], bb, __builtin_fmaf(g[i][k], rsc, -a)));
      store_pack<T, VEC>(dx + row * (int64_t)C + c, o);
    }
  };
  int64_t row = (int64_t)blockIdx.x * ROWS + sub;
  fetch(0, row);
  // (the LDS of the sums alternates between rows)
  if constexpr (kRoom) {
    fetch(1, row + step);
    for (; row < M; row += 2 * step) {
      work(0, 0, row);
      if (row + step < M) work(1, 1, row + step);
    }
  } else {
    for (int slot = 0; row < M; row += step, slot ^= 1) work(0, slot, row);
  }
  if (part == nullptr) return;
  if constexpr (ROWS > 1) {  // the block's row streams, in order
    if (sub > 0) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          float* j = join + ((sub - 1) * 2 * NV * VEC + i * VEC + k) * TPR + t;
          j[0] = aw[i][k];
          j[NV * VEC * TPR] = ab[i][k];
        }
    }
    __syncthreads();
    if (sub > 0) return;
    for (int u = 0; u < ROWS - 1; ++u)
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          const float* j = join + (u * 2 * NV * VEC + i * VEC + k) * TPR + t;
          aw[i][k] += j[0];
          ab[i][k] += j[NV * VEC * TPR];
        }
  }
  float* pa = part + (int64_t)blockIdx.x * 2 * C;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      const int c = (i * TPR + t) * VEC + k;
      if (c < C) {
        pa[c] = aw[i][k];
        pa[C + c] = ab[i][k];
      }
    }
}

// dw, db [C] from part [G][2][C]: 32 threads share a column, each adds every
// 32nd share in order, then the 32 sums are added in order. (32 columns are one
// 128-byte line of a share; 64 columns and 16 threads left most of the GPU idle
// at C = 2048.)
template <typename P>
__global__ __launch_bounds__(1024) void norm_reduce_kernel(const float* __restrict__ part, int G, int C,
                                                           P* __restrict__ dw, P* __restrict__ db) {
  __shared__ float s[32][33];
  const int x = threadIdx.x & 31, k = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + x;
  float a = 0.f;
  if (col < 2 * C) {
#pragma unroll 8
    for (int g = k; g < G; g += 32) a += part[(int64_t)g * 2 * C + col];
  }
  s[k][x] = a;
  __syncthreads();
  if (k != 0 || col >= 2 * C) return;
#pragma unroll
  for (int i = 1; i < 32; ++i) a += s[i][x];
  if (col < C) {
    if (dw) dw[col] = from_f32<P>(a);
  } else if (db) {
    db[col - C] = from_f32<P>(a);
  }
}

template <typename T, typename P, int VEC, int TPR, int NV>
void run_fwd(const NormArgs& a, hipStream_t s) {
  constexpr int ROWS = TPR < 256 ? 256 / TPR : 1, THREADS = TPR < 256 ? 256 : TPR;
  const int64_t most = launch_limit(THREADS) * ROWS;  // 2^24 rows of 520 columns (17 GB of bf16) are more
  for (int64_t r = 0; r < a.M; r += most) {
    const int64_t n = a.M - r < most ? a.M - r : most;
    hipLaunchKernelGGL((norm_fwd_kernel<T, P, VEC, TPR, NV>), dim3((unsigned)((n + ROWS - 1) / ROWS)), dim3(THREADS), 0,
                       s, static_cast<const T*>(a.x) + r * a.ldx, a.ldx, static_cast<const P*>(a.w),
                       static_cast<const P*>(a.b), n, (int)a.C, 1.0f / (float)a.C, a.eps,
                       static_cast<T*>(a.y) + r * a.C, a.mean + r, a.rstd + r);
  }
}

template <typename T, typename P, int VEC, int TPR, int NV>
void run_bwd(const NormArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((norm_bwd_kernel<T, P, VEC, TPR, NV>), dim3((unsigned)norm_groups(a.M, a.C)),
                     dim3(TPR < 256 ? 256 : TPR), 0, s, static_cast<const T*>(a.x), a.ldx,
                     static_cast<const P*>(a.w), static_cast<const T*>(a.dy), a.lddy, a.mean, a.rstd, a.M, (int)a.C,
                     1.0f / (float)a.C, static_cast<T*>(a.dx), a.part);
}

// Threads of a row: as few as hold it in registers with 16-byte loads (up to 4
// vectors of bf16 each), because they all wait at the row's one barrier twice:
// a wave of its own for a row of 512 columns, 4 waves up to 8192 (8192 rows of
// 5120 bf16 out of cache: 31 us, 35 with 8 waves, 45 with 16; of 4096: 22 and 23;
// of 8192: 47, 47 and 55), 16 beyond.
template <typename T, typename P>
void pick_fwd(const NormArgs& a, bool vec, hipStream_t s) {
  const int64_t C = a.C;
  if (vec) {
    constexpr int V = 16 / sizeof(T);
    constexpr int B = sizeof(T) / 2;  // vectors per row double with float32
    if (C <= 512) return run_fwd<T, P, V, 64, B>(a, s);
    if (C <= 2048) return run_fwd<T, P, V, 256, B>(a, s);
    if (C <= 4096) return run_fwd<T, P, V, 256, 2 * B>(a, s);
    if (C <= 8192) return run_fwd<T, P, V, 256, 4 * B>(a, s);
    return run_fwd<T, P, V, 1024, 2 * B>(a, s);
  }
  if (C <= 512) return run_fwd<T, P, 1, 64, 8>(a, s);
  if (C <= 2048) return run_fwd<T, P, 1, 256, 8>(a, s);
  if (C <= 8192) return run_fwd<T, P, 1, 1024, 8>(a, s);
  return run_fwd<T, P, 1, 1024, 16>(a, s);
}

// 16 columns a thread where the row is wide enough for 512 threads: fewer
// threads wait at the row's barrier (8192 bf16 columns: 97 us with 512 threads,
// 118 us with 1024; 4096: 53 us with 256, 62 us with 512, at 8192 rows).
template <typename T, typename P>
void pick_bwd(const NormArgs& a, bool vec, hipStream_t s) {
  const int64_t C = a.C;
  if (vec) {
    constexpr int V = 16 / sizeof(T);
    constexpr int B = sizeof(T) / 2;
    if (C <= 512) return run_bwd<T, P, V, 64, B>(a, s);
    if (C <= 2048) return run_bwd<T, P, V, 256, B>(a, s);
    if (C <= 4096) return run_bwd<T, P, V, 256, 2 * B>(a, s);
    if (C <= 8192) return run_bwd<T, P, V, 512, 2 * B>(a, s);
    return run_bwd<T, P, V, 1024, 2 * B>(a, s);
  }
  if (C <= 512) return run_bwd<T, P, 1, 64, 8>(a, s);
  if (C <= 2048) return run_bwd<T, P, 1, 256, 8>(a, s);
  if (C <= 4096) return run_bwd<T, P, 1, 256, 16>(a, s);
  if (C <= 8192) return run_bwd<T, P, 1, 512, 16>(a, s);
  return run_bwd<T, P, 1, 1024, 16>(a, s);
}

// 16-byte vectors need every row to start on 16 bytes and to be whole vectors.
bool whole_vectors(const NormArgs& a, int64_t ld2) {
  const int64_t v = a.x_f32 ? 4 : 8;
  return a.C % v == 0 && a.ldx % v == 0 && ld2 % v == 0;
}

}  // namespace

hipError_t launch_norm_fwd(const NormArgs& a, hipStream_t s) {
  const bool vec = whole_vectors(a, a.C);
  if (a.x_f32) {
    a.w_f32 ? pick_fwd<float, float>(a, vec, s) : pick_fwd<float, uint16_t>(a, vec, s);
  } else {
    a.w_f32 ? pick_fwd<uint16_t, float>(a, vec, s) : pick_fwd<uint16_t, uint16_t>(a, vec, s);
  }
  return hipGetLastError();
}

hipError_t launch_norm_bwd(const NormArgs& a, hipStream_t s) {
  const bool vec = whole_vectors(a, a.lddy);
  if (a.x_f32) {
    a.w_f32 ? pick_bwd<float, float>(a, vec, s) : pick_bwd<float, uint16_t>(a, vec, s);
  } else {
    a.w_f32 ? pick_bwd<uint16_t, float>(a, vec, s) : pick_bwd<uint16_t, uint16_t>(a, vec, s);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !a.part) return e;
  const dim3 grid((unsigned)((2 * a.C + 31) / 32));
  const int G = (int)norm_groups(a.M, a.C);
  if (a.w_f32)
    hipLaunchKernelGGL(norm_reduce_kernel<float>, grid, dim3(1024), 0, s, a.part, G, (int)a.C,
                       static_cast<float*>(a.dw), static_cast<float*>(a.db));
  else
    hipLaunchKernelGGL(norm_reduce_kernel<uint16_t>, grid, dim3(1024), 0, s, a.part, G, (int)a.C,
                       static_cast<uint16_t*>(a.dw), static_cast<uint16_t*>(a.db));
  return hipGetLastError();
}

}  // namespace qlora
