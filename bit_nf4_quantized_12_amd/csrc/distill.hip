// Distillation from a teacher's top logits: loss and gradient.
//
// Row: student logits z [V], temperature tau, and K teacher entries (value
// t_k at vocabulary index i_k; an index outside [0, V) is no entry).
//   q = softmax(z / tau),  lse = log sum exp(z / tau)
//   p_k = softmax over the row's entries of t_k / tau, or, with the teacher's
//         own log sum exp given, exp(t_k / tau - t_lse);  P = sum p_k
//   loss = tau^2 sum_k p_k (log p_k - z[i_k] / tau + lse)
//   dz_j = weight tau (P q_j - sum over k with i_k = j of p_k)
// (tau^2 keeps the gradient's size independent of the temperature.) A row
// without an entry of positive probability, or of weight zero, gives a zero
// gradient whatever its logits hold; entries of probability zero add nothing to
// the loss.
//
// The one-pass kernel keeps the row in the registers of its workgroup, so a
// step reads the logits once and writes the gradient once: the loss alone
// reads M V, the step moves 2 M V elements, and a backward that follows a
// separate forward 2 M V more. Sums, maxima and probabilities are float32;
// exponentials run in base 2 on (z - reference) (log2 e / tau), the difference
// first, so that no masked value (down to the type's lowest) overflows.
//
// Bound: HBM. 8192 rows of 32000 bf16 logits with 64 entries: 222 us for loss and
// gradient (1.05 GB, 4.7 TB/s; a large copy reaches 4.95). 511 rows of 50021
// float32 logits: loss 29 us (102 MB, 3.5 TB/s: two rows fit a compute unit, so
// loads and sums of different rows hardly overlap), gradient 41 us (204 MB,
// 5 TB/s). Rows that pass the registers: 2048 of 151936 bf16 logits 340 us for loss
// and gradient (1.24 GB and a second read, 3.7 TB/s of the former), the loss alone
// 113 us (5.5 TB/s).
#include "launch.hpp"
#include "reduce.hpp"

namespace qlora {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float log2_hw(float x) { return __builtin_amdgcn_logf(x); }

// 16 bytes of a row: 8 bf16 or 4 float32 values.
template <typename T>
struct Chunk;
template <>
struct Chunk<uint16_t> {
  static constexpr int N = 8;
  static constexpr uint32_t kNegInf = 0xff80ff80u;
  static __device__ __forceinline__ void get(const u32x4& u, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = bf16lo(u[i]);
      f[2 * i + 1] = bf16hi(u[i]);
    }
  }
  static __device__ __forceinline__ u32x4 put(const float (&f)[8]) {
    return u32x4{pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7])};
  }
  static __device__ __forceinline__ float top(const u32x4& u, float m) {
#pragma unroll
    for (int i = 0; i < 4; ++i) m = fmaxf(m, fmaxf(bf16lo(u[i]), bf16hi(u[i])));
    return m;
  }
  static __device__ __forceinline__ float one(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
  static __device__ __forceinline__ uint16_t back(float v) {
    const __bf16 h = (__bf16)v;
    return __builtin_bit_cast(uint16_t, h);
  }
};
template <>
struct Chunk<float> {
  static constexpr int N = 4;
  static constexpr uint32_t kNegInf = 0xff800000u;
  static __device__ __forceinline__ void get(const u32x4& u, float (&f)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(u[i]);
  }
  static __device__ __forceinline__ u32x4 put(const float (&f)[4]) {
    return u32x4{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])};
  }
  static __device__ __forceinline__ float top(const u32x4& u, float m) {
#pragma unroll
    for (int i = 0; i < 4; ++i) m = fmaxf(m, __uint_as_float(u[i]));
    return m;
  }
  static __device__ __forceinline__ float one(float v) { return v; }
  static __device__ __forceinline__ float back(float v) { return v; }
};

// Chunk c of a row of V elements at `row`, which starts `a` elements past a
// 16-byte boundary: elements c N - a .. + N - 1. Chunks that reach past an
// end are read element by element, with minus infinity where there is none.
template <typename T>
__device__ __forceinline__ u32x4 load_chunk(const T* row, int64_t V, int a, int64_t c) {
  constexpr int N = Chunk<T>::N;
  const int64_t e = c * N - a;
  if (e >= 0 && e + N <= V) return *reinterpret_cast<const u32x4*>(row + e);
  T v[N];
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = (e + i >= 0 && e + i < V) ? row[e + i] : Chunk<T>::back(-__builtin_inff());
  u32x4 u;
  __builtin_memcpy(&u, v, 16);
  return u;
}
template <typename T>
__device__ __forceinline__ void store_chunk(T* row, int64_t V, int a, int64_t c, bool whole,
                                            const u32x4& u) {
  constexpr int N = Chunk<T>::N;
  const int64_t e = c * N - a;
  if (whole && e >= 0 && e + N <= V) {
    *reinterpret_cast<u32x4*>(row + e) = u;
    return;
  }
  T v[N];
  __builtin_memcpy(v, &u, 16);
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (e + i >= 0 && e + i < V) row[e + i] = v[i];
}

template <typename T>
__device__ __forceinline__ int misalign(const T* p) {
  return (int)((reinterpret_cast<uintptr_t>(p) & 15) / sizeof(T));
}

// Reductions over the workgroup; `slot` (2 x 16 floats) is that call's own.
struct MaxOf {
  static __device__ __forceinline__ float op(float a, float b) { return fmaxf(a, b); }
};
struct SumOf {
  static __device__ __forceinline__ float op(float a, float b) { return a + b; }
};
template <typename F>
__device__ __forceinline__ void block_reduce(float& a, float& b, float (*slot)[16]) {
  a = wave_reduce(a, F::op);
  b = wave_reduce(b, F::op);
  const int w = threadIdx.x >> 6, W = blockDim.x >> 6;
  if ((threadIdx.x & 63) == 0) {
    slot[0][w] = a;
    slot[1][w] = b;
  }
  __syncthreads();
  a = slot[0][0];
  b = slot[1][0];
  for (int i = 1; i < W; ++i) {
    a = F::op(a, slot[0][i]);
    b = F::op(b, slot[1][i]);
  }
}

// The row's teacher entries in LDS: index (-1: none), value, student logit at
// the index. Base-2 log probability of an entry: (t - base) c - shift.
struct Entries {
  __attribute__((aligned(16))) int idx[kDistillMaxK];
  float t[kDistillMaxK];
  float z[kDistillMaxK];
};

// Entry k of the row; the index -1 where there is none.
__device__ __forceinline__ int64_t entry_index(const DistillArgs& a, int64_t row, int k) {
  const int64_t at = row * a.K + k;
  const int64_t i = a.idx_64 ? static_cast<const int64_t*>(a.idx)[at] : (int64_t)static_cast<const int32_t*>(a.idx)[at];
  return i >= 0 && i < a.V ? i : -1;
}
__device__ __forceinline__ float entry_value(const DistillArgs& a, int64_t row, int k) {
  const int64_t at = row * a.K + k;
  return a.val_f32 ? static_cast<const float*>(a.val)[at] : Chunk<uint16_t>::one(static_cast<const uint16_t*>(a.val)[at]);
}

// Entry k of the row as it is loaded, before it goes to LDS.
struct Entry {
  int64_t i;
  float t, z;
};
__device__ __forceinline__ Entry load_entry(const DistillArgs& a, int64_t row, int k) {
  Entry e{-1, -__builtin_inff(), 0.f};
  if (k < a.K) {
    e.i = entry_index(a, row, k);
    e.t = entry_value(a, row, k);
    if (e.i < 0) e.t = -__builtin_inff();
  }
  return e;
}
template <typename T>
__device__ __forceinline__ void load_logit(Entry& e, const T* zr, int64_t keep0, int64_t keep1) {
  if (e.i >= keep0 && e.i < keep1) e.z = Chunk<T>::one(zr[e.i]);
}
// Puts the entry into LDS and returns its value for the row's maximum. A maximum
// skips NaN: infinity stands in for it, so that a row of NaN is not taken for
// one without entries and its sums of (t - maximum) become NaN.
__device__ __forceinline__ float keep_entry(const DistillArgs& a, const Entry& e, int k, Entries& en) {
  if (k < (a.K + 3) / 4 * 4) {  // whole groups of 4 are compared
    en.idx[k] = (int)e.i;
    en.t[k] = e.t;
    en.z[k] = e.z;
  }
  return e.t == e.t ? e.t : __builtin_inff();
}
// The entries past the first of each thread; returns the largest value.
template <typename T>
__device__ __forceinline__ float more_entries(const DistillArgs& a, int64_t row, const T* zr, int64_t keep0,
                                              int64_t keep1, Entries& en) {
  float top = -__builtin_inff();
  for (int k = threadIdx.x + blockDim.x; k < (a.K + 3) / 4 * 4; k += blockDim.x) {
    Entry e = load_entry(a, row, k);
    load_logit(e, zr, keep0, keep1);
    top = fmaxf(top, keep_entry(a, e, k, en));
  }
  return top;
}

// After the gradient's dense part and a barrier: the entries' own elements
// are written again with their probabilities taken off. Entries with the
// same index add up in their order, and the first of them writes. first ..
// last limits the indices to the caller's part; q = exp2((z - zbase) c - zshift).
template <typename T>
__device__ __forceinline__ void store_entries(T* dzr, const Entries& en, int K, float c, float zbase, float zshift,
                                              float base, float shift, float P, float g, int64_t first,
                                              int64_t last) {
  for (int k = threadIdx.x; k < K; k += blockDim.x) {
    const int i = en.idx[k];
    if (i < first || i >= last) continue;
    float p = 0.f;
    bool mine = true;
    for (int j = 0; j < K; j += 4) {
      const int4 v = *reinterpret_cast<const int4*>(en.idx + j);
      if (v.x != i && v.y != i && v.z != i && v.w != i) continue;
      const int w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (w[e] != i) continue;
        if (j + e < k) mine = false;
        p += exp2_hw((en.t[j + e] - base) * c - shift);
      }
    }
    if (!mine) continue;
    const float q = exp2_hw((en.z[k] - zbase) * c - zshift);
    dzr[i] = Chunk<T>::back(g * (P * q - p));
  }
}

// One workgroup per row. NV > 0: the row is held in NV chunks per thread;
// NV = 0: any length, the row is read twice (the second time mostly from
// cache). GRAD: the gradient is written too; dz may be z itself (a thread
// overwrites only chunks that it has read, and the entries' logits are read
// before the first barrier).
template <typename T, int NV, bool GRAD>
__global__ __launch_bounds__(1024) void distill_row_kernel(DistillArgs a) {
  constexpr int N = Chunk<T>::N;
  __shared__ Entries en;
  __shared__ float red[2][2][16];
  const int64_t row = blockIdx.x;
  const T* zr = static_cast<const T*>(a.z) + row * a.ldz;
  const int off = misalign(zr);
  const int64_t chunks = (a.V + off + N - 1) / N;
  const int nt = blockDim.x, tid = threadIdx.x;
  const float c = kLog2e * a.inv_tau;

  // The thread's entry is asked for before the row, its logit after it.
  Entry first = load_entry(a, row, tid);
  u32x4 raw[NV > 0 ? NV : 1];
  if constexpr (NV > 0) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t ch = (int64_t)i * nt + tid;
      if (ch < chunks) {
        raw[i] = load_chunk<T>(zr, a.V, off, ch);
      } else {
        const uint32_t ni = Chunk<T>::kNegInf;
        raw[i] = u32x4{ni, ni, ni, ni};
      }
    }
  }
  load_logit(first, zr, 0, a.V);
  float zmax = -__builtin_inff(), sum = 0.f;
  auto add = [&](const u32x4& u, float ref) {
    float f[N];
    Chunk<T>::get(u, f);
#pragma unroll
    for (int k = 0; k < N; ++k) sum += exp2_hw((f[k] - ref) * c);
  };
  if constexpr (NV > 0) {
#pragma unroll
    for (int i = 0; i < NV; ++i) zmax = Chunk<T>::top(raw[i], zmax);
  } else {
    // running maximum and sum of this thread's chunks
    for (int64_t ch = tid; ch < chunks; ch += nt) {
      raw[0] = load_chunk<T>(zr, a.V, off, ch);
      const float m = Chunk<T>::top(raw[0], zmax);
      if (m != zmax) sum *= exp2_hw((zmax - m) * c);
      zmax = m;
      add(raw[0], m == -__builtin_inff() ? 0.f : m);
    }
  }
  float tmax = keep_entry(a, first, tid, en);
  tmax = fmaxf(tmax, more_entries(a, row, zr, 0, a.V, en));
  const float mine = zmax;
  block_reduce<MaxOf>(zmax, tmax, red[0]);
  if constexpr (NV > 0) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      asm("" : "+v"(raw[i]));  // (unpacked anew by each pass: the values of two passes do not fit)
      add(raw[i], zmax);
    }
  } else if (mine != zmax) {
    sum *= exp2_hw((mine - zmax) * c);
  }
  // teacher: relative to the entries' maximum, or as recorded
  const bool none = tmax == -__builtin_inff();
  const float base = a.t_lse ? 0.f : none ? 0.f : tmax;
  float shift = a.t_lse ? a.t_lse[row] * kLog2e : 0.f;
  float tsum = 0.f;
  for (int k = tid; k < a.K; k += nt)
    if (en.idx[k] >= 0 && en.t[k] != -__builtin_inff()) tsum += exp2_hw((en.t[k] - base) * c - shift);
  block_reduce<SumOf>(sum, tsum, red[1]);
  const float lsum = log2_hw(sum);
  const float Z = zmax + lsum * (kLn2 * a.tau);  // tau lse
  if (!a.t_lse) shift = log2_hw(tsum);
  const float P = none ? 0.f : (a.t_lse || tsum != tsum ? tsum : 1.f);

  if (tid < 64) {
    float part = 0.f;
    for (int k = tid; k < a.K; k += 64) {
      if (en.idx[k] < 0 || none) continue;
      const float lp = (en.t[k] - base) * c - shift;
      const float p = exp2_hw(lp);
      if (p != 0.f) part += p * (lp - ((en.z[k] - zmax) * c - lsum));
    }
    part = wave_sum(part);
    if (tid == 0) {
      a.loss[row] = none ? 0.f : part * kLn2 * a.tau * a.tau;
      a.lse[row] = __builtin_fmaf(zmax, a.inv_tau, lsum * kLn2);
    }
  }
  if constexpr (!GRAD) return;

  const float w = a.weight ? a.weight[row] : 1.f;
  const float g = P == 0.f ? 0.f : w * a.tau;
  const float gp = g * P;
  T* dzr = static_cast<T*>(a.dz) + row * a.lddz;
  const bool whole = misalign(dzr) == off;
  auto grad = [&](const u32x4& u) -> u32x4 {
    if (g == 0.f) return u32x4{0, 0, 0, 0};
    float f[N];
    Chunk<T>::get(u, f);
#pragma unroll
    for (int k = 0; k < N; ++k) f[k] = gp * exp2_hw((f[k] - Z) * c);
    return Chunk<T>::put(f);
  };
  if constexpr (NV > 0) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t ch = (int64_t)i * nt + tid;
      asm("" : "+v"(raw[i]));
      if (ch < chunks) store_chunk<T>(dzr, a.V, off, ch, whole, grad(raw[i]));
    }
  } else {
    for (int64_t ch = tid; ch < chunks; ch += nt)
      store_chunk<T>(dzr, a.V, off, ch, whole, grad(load_chunk<T>(zr, a.V, off, ch)));
  }
  __syncthreads();  // the dense part is stored before the entries' elements
  if (g != 0.f) store_entries<T>(dzr, en, a.K, c, zmax, lsum, base, shift, P, g, 0, a.V);
}

// Gradient for a given upstream one, from the saved lse: a workgroup takes
// kBwdChunks chunks of a row, 4 of each thread on their way while it finishes
// the 4 before them (entries and their sums are done again by each part).
constexpr int kBwdChunks = 4096;
template <typename T>
__global__ __launch_bounds__(256) void distill_bwd_kernel(DistillArgs a, int parts) {
  constexpr int N = Chunk<T>::N;
  __shared__ Entries en;
  __shared__ float red[2][2][16];
  const int64_t row = blockIdx.x / parts;
  const int part = (int)(blockIdx.x % parts);
  const T* zr = static_cast<const T*>(a.z) + row * a.ldz;
  const int off = misalign(zr);
  const int64_t chunks = (a.V + off + N - 1) / N;
  const int64_t c0 = (int64_t)part * kBwdChunks, c1 = min(chunks, c0 + kBwdChunks);
  const float c = kLog2e * a.inv_tau;
  // The first chunks are asked for ahead of the entries' reductions; the logits
  // of entries only where this workgroup's part holds them: another may be
  // writing its own part of the row in place.
  constexpr int U = 4;
  const int64_t keep0 = max((int64_t)0, c0 * N - off), keep1 = min(a.V, c1 * N - off);
  Entry first = load_entry(a, row, threadIdx.x);
  u32x4 raw[U];
  auto fetch = [&](int64_t b) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t ch = b + u * 256 + threadIdx.x;
      if (ch < c1) raw[u] = load_chunk<T>(zr, a.V, off, ch);
    }
  };
  fetch(c0);
  load_logit(first, zr, keep0, keep1);
  float tmax = keep_entry(a, first, threadIdx.x, en), zero = 0.f;
  tmax = fmaxf(tmax, more_entries(a, row, zr, keep0, keep1, en));
  block_reduce<MaxOf>(tmax, zero, red[0]);
  const bool none = tmax == -__builtin_inff();
  const float base = a.t_lse ? 0.f : none ? 0.f : tmax;
  float shift = a.t_lse ? a.t_lse[row] * kLog2e : 0.f;
  float tsum = 0.f;
  for (int k = threadIdx.x; k < a.K; k += 256)
    if (en.idx[k] >= 0 && en.t[k] != -__builtin_inff()) tsum += exp2_hw((en.t[k] - base) * c - shift);
  block_reduce<SumOf>(tsum, zero, red[1]);
  if (!a.t_lse) shift = log2_hw(tsum);
  const float P = none ? 0.f : (a.t_lse || tsum != tsum ? tsum : 1.f);
  const float Z = a.lse[row] * a.tau;
  const float g = P == 0.f ? 0.f : (a.weight ? a.weight[row] : 1.f) * a.tau;
  const float gp = g * P;
  T* dzr = static_cast<T*>(a.dz) + row * a.lddz;
  const bool whole = misalign(dzr) == off;
  for (int64_t b = c0; b < c1; b += 256 * U) {
    u32x4 now[U];
#pragma unroll
    for (int u = 0; u < U; ++u) now[u] = raw[u];
    fetch(b + 256 * U);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t ch = b + u * 256 + threadIdx.x;
      if (ch >= c1) continue;
      u32x4 o{0, 0, 0, 0};
      if (g != 0.f) {
        float f[N];
        Chunk<T>::get(now[u], f);
#pragma unroll
        for (int k = 0; k < N; ++k) f[k] = gp * exp2_hw((f[k] - Z) * c);
        o = Chunk<T>::put(f);
      }
      store_chunk<T>(dzr, a.V, off, ch, whole, o);
    }
  }
  __syncthreads();  // the dense part is stored before the entries' elements
  if (g != 0.f) store_entries<T>(dzr, en, a.K, c, Z, 0.f, base, shift, P, g, keep0, keep1);
}

// Rows r .. r + n - 1 of a call: what one launch takes of more rows.
DistillArgs rows_of(const DistillArgs& a, int64_t r, int64_t n) {
  DistillArgs b = a;
  b.M = n;
  auto from = [](const void* p, int64_t elements, int size) { return static_cast<const char*>(p) + elements * size; };
  b.z = from(a.z, r * a.ldz, a.z_f32 ? 4 : 2);
  b.val = from(a.val, r * a.K, a.val_f32 ? 4 : 2);
  b.idx = from(a.idx, r * a.K, a.idx_64 ? 8 : 4);
  if (a.t_lse) b.t_lse = a.t_lse + r;
  if (a.weight) b.weight = a.weight + r;
  if (a.loss) b.loss = a.loss + r;
  b.lse = a.lse + r;
  if (a.dz) b.dz = static_cast<char*>(a.dz) + r * a.lddz * (a.z_f32 ? 4 : 2);
  return b;
}

template <typename T, bool GRAD>
hipError_t run_row(const DistillArgs& a, hipStream_t s) {
  constexpr int N = Chunk<T>::N;
  const int64_t chunks = (a.V + N - 1) / N + 1;  // one more where the row starts inside a chunk
  // Threads per row: 16 chunks each when there are rows enough to fill the
  // GPU, 4 each (up to 1024 threads) when there are few (32000 bf16 logits: 14.4
  // and 15.5 us with 4 and 16 chunks at 128 rows, 21.7 and 22.5 at 512, 39 and 36 at
  // 1024, 134 and 120 at 4096).
  auto threads = [&](int64_t nv) { return ((chunks + nv - 1) / nv + 63) / 64 * 64; };
  const int64_t nv = a.M >= 1024 ? 16 : 4;
  const bool few = threads(4) <= 1024 && (nv == 4 || threads(16) < 128), held = threads(16) <= 1024;
  const int64_t nt = few ? threads(4) : held ? threads(16) : 1024, most = launch_limit(nt);
  for (int64_t r = 0; r < a.M; r += most) {
    const DistillArgs b = rows_of(a, r, a.M - r < most ? a.M - r : most);
    const dim3 grid((unsigned)b.M), block((unsigned)nt);
    if (few)
      hipLaunchKernelGGL((distill_row_kernel<T, 4, GRAD>), grid, block, 0, s, b);
    else if (held)
      hipLaunchKernelGGL((distill_row_kernel<T, 16, GRAD>), grid, block, 0, s, b);
    else
      hipLaunchKernelGGL((distill_row_kernel<T, 0, GRAD>), grid, block, 0, s, b);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_distill_fwd(const DistillArgs& a, bool grad, hipStream_t s) {
  if (a.z_f32) return grad ? run_row<float, true>(a, s) : run_row<float, false>(a, s);
  return grad ? run_row<uint16_t, true>(a, s) : run_row<uint16_t, false>(a, s);
}

hipError_t launch_distill_bwd(const DistillArgs& a, hipStream_t s) {
  const int64_t n = a.z_f32 ? 4 : 8;
  const int64_t chunks = (a.V + n - 1) / n + 1;
  const int parts = (int)((chunks + kBwdChunks - 1) / kBwdChunks);
  const int64_t most = launch_limit(256) / parts;
  for (int64_t r = 0; r < a.M; r += most) {
    const DistillArgs b = rows_of(a, r, a.M - r < most ? a.M - r : most);
    const dim3 grid((unsigned)(b.M * parts));
    if (a.z_f32)
      hipLaunchKernelGGL(distill_bwd_kernel<float>, grid, dim3(256), 0, s, b, parts);
    else
      hipLaunchKernelGGL(distill_bwd_kernel<uint16_t>, grid, dim3(256), 0, s, b, parts);
  }
  return hipGetLastError();
}

}  // namespace qlora
