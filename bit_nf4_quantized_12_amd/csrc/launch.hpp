// Host-side launchers of the library's kernels (one per .hip file).
#pragma once

#include <atomic>

#include "common.hpp"

namespace qlora {

// Opt kernel fn in to `bytes` of dynamic LDS (above the default 64 KB) on
// the current device. The attribute is per device, so `done` keeps one bit
// per device (devices past 31 set it on every call).
inline hipError_t ensure_lds(const void* fn, int bytes, std::atomic<uint32_t>& done) {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const uint32_t bit = dev < 32 ? (1u << dev) : 0u;
  if (bit && (done.load(std::memory_order_acquire) & bit)) return hipSuccess;
  e = hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == hipSuccess && bit) done.fetch_or(bit, std::memory_order_release);
  return e;
}

// Workgroups that one launch takes along x. A grid of 2^32 threads or more is
// not refused: its workgroups past that count do not run, without an error.
inline int64_t launch_limit(int64_t threads) { return ((int64_t(1) << 32) - 1) / threads; }

struct GemmParams {
  const uint16_t* act;     // [M, Kred] bf16, row pitch Kred
  const uint8_t* codes;    // NF4 codes of W [wN, wK]
  const uint8_t* c2;
  const float* c1;
  const float* absmax;     // fp32 block constants (no double quantisation), or null
  int64_t wN, wK;
  const uint16_t* lora_l;  // [M, lora_ld] bf16 (scale folded in), or null
  const uint16_t* lora_r;  // [Nout, rp] bf16, or null
  int rp;                  // multiple of 64, columns past r are zero
  int lora_ld;             // row pitch of lora_l (rp, or more for grouped linears)
  int lora_seg;            // > 0: output columns n use lora_l columns (n / lora_seg) rp .. + rp
  uint16_t* out;           // [M, Nout] bf16
  int M, Nout, Kred;
  Levels lv;
  // split reduction: ksplit > 1 splits of kchunk 64-deep steps write float32
  // partial tiles to part [ksplit][M][Nout], summed into out afterwards
  int ksplit = 1, kchunk = 0;
  float* part = nullptr;
};

// Output tile of the GEMM: 512 x 128 from 1024 rows on (half the unpacking
// per MFMA), else 256 x 256; when that leaves fewer than 192 tiles (most of
// the 256 CUs idle), 128 x 128.
enum GemmTile { kTile512x128 = 0, kTile256x256 = 1, kTile128x128 = 2 };
inline int64_t gemm_tiles(int64_t M, int64_t Nout, int64_t bm, int64_t bn) {
  return ((M + bm - 1) / bm) * ((Nout + bn - 1) / bn);
}
inline GemmTile gemm_tile(int64_t M, int64_t Nout) {
  const bool big = M >= 1024;
  if (gemm_tiles(M, Nout, big ? 512 : 256, big ? 128 : 256) >= 192) return big ? kTile512x128 : kTile256x256;
  return kTile128x128;
}

// Splits of the reduction: with 128 x 128 tiles, enough splits for ~256
// workgroups, at most 4, each at least 4 steps of 64; none otherwise.
// Returns the split count (every split non-empty) and the steps per split.
inline int gemm_ksplit(int64_t M, int64_t Nout, int64_t Kred, int* kchunk) {
  const int64_t nk = (Kred + 63) / 64;
  int64_t ks = 1;
  if (gemm_tile(M, Nout) == kTile128x128) {
    const int64_t tiles = gemm_tiles(M, Nout, 128, 128);
    ks = (256 + tiles - 1) / tiles;
    if (ks > 4) ks = 4;
    if (ks > nk / 4) ks = nk / 4;
    if (ks < 1) ks = 1;
  }
  const int64_t ch = (nk + ks - 1) / ks;
  *kchunk = (int)ch;
  return (int)((nk + ch - 1) / ch);
}

// Several tensors quantised by one launch: workgroups gstart[t] ..
// gstart[t+1]-1 take the 16384-weight groups of tensor t.
constexpr int kQuantBatch = 16;
struct QuantBatch {
  int count;
  int64_t gstart[kQuantBatch + 1];
  const uint16_t* w[kQuantBatch];
  int64_t n[kQuantBatch];
  uint8_t* codes[kQuantBatch];
  uint8_t* c2[kQuantBatch];
  float* c1[kQuantBatch];
  float* absmax[kQuantBatch];
};
hipError_t launch_quantize_batch(const QuantBatch& b, int codebook, hipStream_t s);

// Double-quantised constants (c2, c1) when absmax is null; otherwise the
// fp32 block absmax, and c2 / c1 are unused.
hipError_t launch_quantize(const void* w, int64_t n, int codebook, uint8_t* codes, uint8_t* c2, float* c1,
                           float* absmax, hipStream_t s);
hipError_t launch_dequant(const uint8_t* codes, const uint8_t* c2, const float* c1, const float* absmax,
                          int64_t n, int codebook, bool bf16_out, void* out, hipStream_t s);
hipError_t launch_gemm(const GemmParams& p, bool transposed_w, hipStream_t s);
hipError_t launch_proj(const uint16_t* L, const uint16_t* R, int M, int Kr, int r, int rp,
                       int nsplit, float* part, hipStream_t s);
// Streamed projection (Kr % 64 == 0, rp_total % 64 == 0), part
// [nsplit][M][rp_total]. The result's 64-column blocks come in segments of
// zper blocks; segment g multiplies L + g segL by rows of R + g segR (r_seg
// valid rows), row pitches ldL / ldR.
hipError_t launch_proj_seg(const uint16_t* L, int64_t ldL, int64_t segL, const uint16_t* R, int64_t ldR,
                           int64_t segR, int zper, int M, int Kr, int r_seg, int rp_total, int nsplit, float* part,
                           hipStream_t s);
hipError_t launch_finalize(const float* part, int nsplit, int M, int Mp, int r, int rp, float scale,
                           float* P32, uint16_t* Ph, uint16_t* Pl, hipStream_t s);
hipError_t launch_grad(const float* P, const uint16_t* Q, int M, int C, int r, int rp, int nsplit,
                       float* part, hipStream_t s);
hipError_t launch_grad_reduce(const float* part, int nsplit, int r, int rp, int C, float scale,
                              bool transpose, bool part_trans, uint16_t* out, hipStream_t s);
// segC > 0: the columns of segment c / segC pair only with plane columns
// (c / segC) rseg .. + rseg (grouped linears); the result then has rseg rows.
hipError_t launch_grad_tr(const uint16_t* Ph, const uint16_t* Pl, const uint16_t* Q, int M, int Mp, int C,
                          int rp, int nsplit, bool trans, float* part, hipStream_t s, int segC = 0,
                          int rseg = 0);
hipError_t launch_relayout(const uint16_t* in, int64_t rows_in, int64_t cols_in, int64_t ldi,
                           bool transpose, uint16_t* out, int64_t rows_out, int64_t cols_out,
                           int64_t ldo, hipStream_t s);
// Bt [r, N] = B^T for B [N, r]; At [K, rp] = A^T zero-padded for A [rA, K] (if At).
hipError_t launch_transpose2(const uint16_t* B, const uint16_t* A, int N, int K, int r, int rA, int rp,
                             uint16_t* Bt, uint16_t* At, hipStream_t s);
hipError_t launch_finalize2(const float* part, int nsplit, int M, int Mp, int r, int rp, float scale,
                            float* P32, uint16_t* Ph, uint16_t* Pl, const float* T, uint16_t* Th,
                            uint16_t* Tl, hipStream_t s);
hipError_t launch_grad_reduce2(const float* partA, int nsA, int C1, uint16_t* dA, const float* partB, int nsB,
                               int C2, uint16_t* dB, int rA, int rpA, int rB, int rpB, float scale, hipStream_t s);
// Few tokens (M <= 16): T [M, R] = X A^T (float32, A the R rows of the
// segments' adapters stacked), then Y [M, N] = X W~^T + scale T_z B^T (rows
// of segment z = n / segN use T columns z rseg .. + rseg; segN = 0: one
// segment, rseg = R), two launches. Y null: T only.
hipError_t launch_fewtok(const uint16_t* X, const uint8_t* codes, const uint8_t* c2, const float* c1,
                         const float* absmax, int codebook, int N, int K, int M, const uint16_t* A, int R,
                         const uint16_t* B, int rseg, int segN, float scale, uint16_t* Y, float* T,
                         hipStream_t s);

// Merged weight out [N, K] = bf16(W^ + scale B A) (merge.hip); absmax null:
// double-quantised constants.
hipError_t launch_merge(const uint8_t* codes, const uint8_t* c2, const float* c1, const float* absmax, int codebook,
                        const uint16_t* A, const uint16_t* B, int N, int K, int r, float scale, uint16_t* out,
                        hipStream_t s);

// AdamW step (optim.hip): bc1 = 1 / (1 - beta1^t), bc2 = 1 / (1 - beta2^t).
struct AdamW {
  float lr, beta1, beta2, one_minus_beta1, one_minus_beta2, eps, weight_decay, bc1, bc2;
};
hipError_t launch_adamw(float* p, uint16_t* p16, const uint16_t* g, float* m, float* v, int64_t n,
                        const AdamW& a, hipStream_t s);

// Layer norm (norm.hip). ldx, lddy: row pitches in elements; y and dx have
// pitch C. b, dx, dw and db may be null; part is null when neither dw nor db
// is wanted, else float32 [norm_groups][2][C].
struct NormArgs {
  const void* x;
  const void* w;
  const void* b;
  const void* dy;
  int64_t ldx, lddy, M, C;
  bool x_f32, w_f32;
  float eps;
  void* y;
  float* mean;
  float* rstd;
  void* dx;
  void* dw;
  void* db;
  float* part;
};
constexpr int64_t kNormMaxC = 16384;  // widest row that one workgroup holds in registers
// Workgroups of the backward pass: what fits the GPU at once (fewer, larger
// shares of dw and db against fewer bytes in flight: 8192 bf16 columns 95 us
// with 256, 136 with 128, 106 with 512; 4096: 54 with 512, 61 and 66; 2048: 34
// with 512, 38 with 1024, all at 8192 rows; 1024 columns and 65536 rows: 169 with
// 1024, 233 with 512), at most one for 8 rows past 256 of them, at most one for
// the rows that it takes side by side.
inline int64_t norm_groups(int64_t M, int64_t C) {
  const int64_t rows = C <= 512 ? 4 : 1;
  const int64_t cap = C <= 1024 ? 1024 : C <= 4096 ? 512 : 256;
  int64_t g = (M + 7) / 8;
  if (g < 256) g = 256;
  if (g > cap) g = cap;
  const int64_t most = (M + rows - 1) / rows;
  return g < most ? g : most;
}
hipError_t launch_norm_fwd(const NormArgs& a, hipStream_t s);
hipError_t launch_norm_bwd(const NormArgs& a, hipStream_t s);

// Distillation from a teacher's top logits (distill.hip). z, dz: [M, V] with
// row pitches ldz, lddz; val, idx: [M, K] contiguous. t_lse and weight may be
// null. inv_tau = 1 / temperature.
struct DistillArgs {
  const void* z;
  int64_t ldz, M, V;
  bool z_f32;
  const void* val;
  bool val_f32;
  const void* idx;
  bool idx_64;
  int K;
  const float* t_lse;
  float tau, inv_tau;
  const float* weight;
  float* loss;
  float* lse;
  void* dz;
  int64_t lddz;
};
constexpr int kDistillMaxK = 1024;
hipError_t launch_distill_fwd(const DistillArgs& a, bool grad, hipStream_t s);
hipError_t launch_distill_bwd(const DistillArgs& a, hipStream_t s);

// Attention with a sliding window and first tokens that stay visible
// (attn.hip, attn_bwd.hip, decode.hip). Token and head pitches in elements.
struct AttnTensor {
  void* p;
  int64_t st, sh;  // pitch of a token, of a head
};
struct AttnArgs {
  AttnTensor q, k, v, o, d_o, dq, dk, dv;
  float* lse;  // [H, Tq]
  const int32_t* cu_q;
  const int32_t* cu_k;
  int64_t Tq, Tk;
  int B, H, Hkv, D;
  int max_q, max_k;
  int window, sinks;
  float scale;
  float* delta;  // [H, Tq]
  float* lse2;   // [H, Tq], lse in base 2
  float* sink;   // float32 shares of the first tokens' dK and dV
  int parts;     // of a key block's steps; above 1:
  float* share;  // float32 shares of dK and dV [parts][Tk][Hkv][2][64 or 128]
};
constexpr int kMaxSinks = 32;
// Backward: rows of a range of far queries, and the number of range slots. At
// least 512 rows: shares cost more than the shorter walk saves when there are
// many (2 x 4096 tokens, 32 heads of 64: 250 us, 261 with 256 rows; 2048 tokens, 8
// heads of 128: 53 and 49).
inline int attn_sink_span(int64_t max_q) {
  const int64_t sp = (max_q / 16 + 127) / 128 * 128;
  return (int)(sp < 512 ? 512 : sp);
}
// Whether the first tokens' gradients from far queries have kernels (and a
// workspace) of their own. Without them key block 0 walks over every later query
// itself, which is not worth a kernel while its walk stays within twice the
// others' and 1024 rows (window 256, with and without: 16 x 512 tokens 639 and
// 506 us, 8 x 1024 347 and 312, 4 x 2048 340 and 351, 2 x 4096 with 8 key heads
// 287 and 575).
inline bool attn_sink_apart(int64_t max_k, int64_t window, int64_t sinks) {
  return sinks > 0 && max_k > 2 * (64 + window) + 1024;
}
inline int64_t attn_sink_slots(int64_t Tq, int64_t B, int64_t max_q) { return Tq / attn_sink_span(max_q) + B; }
// Backward: key blocks of 64 in the batch (at most), and the parts that the
// steps (query tile and head) of each are cut into, 4 steps or more to a part,
// so that there are up to 1024 workgroups: the first keys' walk over all later
// queries and heads is what the kernel otherwise waits for (one sequence of 2048
// tokens, 4 heads of 128 on one: 240 us whole, 88 us in 16 parts; 500 tokens, 8
// heads on 2: 72 and 41; 2048 tokens, 32 heads on 8: 278 and 240 in 3 parts;
// 8 heads on 8, with fewer steps, 107 and 110).
inline int64_t attn_key_blocks(int64_t Tk, int64_t B, int64_t Hkv) { return (Tk / 64 + B) * Hkv; }
inline int attn_dkv_parts(int64_t Tk, int64_t B, int64_t Hkv, int64_t group, int64_t max_q, int64_t window) {
  const int64_t rows = max_q < window + 64 ? max_q : window + 64;
  int64_t n = 1024 / attn_key_blocks(Tk, B, Hkv);
  const int64_t most = (rows / 64 + 1) * group / 4;
  if (n > most) n = most;
  if (n > 16) n = 16;
  return n < 1 ? 1 : (int)n;
}
hipError_t launch_attn_fwd(const AttnArgs& a, hipStream_t s);
hipError_t launch_attn_bwd(const AttnArgs& a, hipStream_t s);

// One new token per request over a cache (decode.hip): q [B, H, D], k and v
// [B, cap, Hkv, D] with pitches of a request, a token and a head (elements),
// o [B, H, D] contiguous. nsplit > 1: part float32 [B, H, nsplit, D] and stat
// [B, H, nsplit, 2] hold the parts' results, maxima and sums.
struct DecodeArgs {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  int64_t q_sb, q_sh, k_sb, k_st, k_sh, v_sb, v_st, v_sh;
  const int32_t* lens;
  int B, H, Hkv, D, cap;
  int window, sinks;
  float scale;
  uint16_t* o;
  int nsplit;
  float* part;
  float* stat;
};
// Parts of the visible keys: up to a workgroup for each of 256 compute units
// (512 workgroups: 33.5 us against 32.3 with 256 for 4 requests of 8192 keys, 108
// against 104 for one of 131072, both with 8 key heads), each with at least 512
// keys (256: 16 us against 12 for 512 keys, which then take one kernel; 1024: 19
// against 16 for 2048), at most 64 parts (a wave joins them).
inline int decode_splits(int64_t B, int64_t Hkv, int64_t group, int64_t most) {
  const int64_t units = B * Hkv * ((group + 15) / 16);
  int64_t n = 256 / units;
  if (n > most / 512) n = most / 512;
  if (n > 64) n = 64;
  return n < 1 ? 1 : (int)n;
}
hipError_t launch_decode(const DecodeArgs& a, hipStream_t s);

}  // namespace qlora
