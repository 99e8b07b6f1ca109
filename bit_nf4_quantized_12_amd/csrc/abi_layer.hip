// C ABI of the operators around a decoder layer's linears: argument
// validation (before any HIP call), workspace layout and launches of layer
// norm, sliding-window attention and distillation. The operations are defined
// in include/qlora.h.
#include <algorithm>
#include <cmath>

#include "qlora.h"
#include "launch.hpp"

using namespace qlora;

namespace {

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline size_t al256(size_t x) { return (x + 255) & ~size_t(255); }
constexpr int64_t kInt32 = int64_t(1) << 31;

inline bool dtype_ok(int d) { return d == QLORA_F32 || d == QLORA_BF16; }
inline int status_of(hipError_t e) { return e == hipSuccess ? QLORA_OK : QLORA_ERR_DEVICE; }

// ---------------------------------------------------------------------------
// layer norm
// ---------------------------------------------------------------------------
int check_norm(const void* x, int64_t ldx, int x_dtype, const void* w, int w_dtype, const float* mean,
               const float* rstd, int64_t M, int64_t C) {
  if (!x || !w || !mean || !rstd) return QLORA_ERR_NULL;
  if (M < 1 || M >= kInt32 || C < 1 || C > kNormMaxC || ldx < C || ldx >= (int64_t(1) << 40)) return QLORA_ERR_SHAPE;
  if (!dtype_ok(x_dtype) || !dtype_ok(w_dtype)) return QLORA_ERR_UNSUPPORTED;
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(mean, 4) || !aligned(rstd, 4)) return QLORA_ERR_ALIGN;
  return QLORA_OK;
}

// ---------------------------------------------------------------------------
// attention
// ---------------------------------------------------------------------------
// threads: of the largest workgroup that takes a sequence's head (forward 256,
// backward 512). A launch has room for one of them for each (fit_groups).
constexpr int kFwdThreads = 256, kBwdThreads = 512;
int check_attn_sizes(const qlora_window_attn* a, int threads) {
  if (a->B < 1 || a->B >= 65536 || a->Tq < 1 || a->Tq >= kInt32 || a->Tk < 1 || a->Tk >= kInt32) return QLORA_ERR_SHAPE;
  if (a->H < 1 || a->Hkv < 1 || a->H % a->Hkv != 0 || a->H >= 65536) return QLORA_ERR_SHAPE;
  if (a->max_q < 1 || a->max_q >= kInt32 - 256 || a->max_k < 1 || a->max_k >= kInt32 - 256) return QLORA_ERR_SHAPE;
  const int64_t blocks = a->B * ((std::max(a->max_q, a->max_k) + 127) / 128);
  if (blocks * a->H >= kInt32 / 4 || (a->B + 7) * a->H > launch_limit(threads) - 256) return QLORA_ERR_SHAPE;
  if (a->D < 8 || a->D > 128 || a->D % 8 != 0) return QLORA_ERR_UNSUPPORTED;
  if (a->window < 1 || a->sinks < 0 || a->sinks > kMaxSinks) return QLORA_ERR_UNSUPPORTED;
  if (!std::isfinite(a->scale) || !(a->scale > 0.0f)) return QLORA_ERR_UNSUPPORTED;
  return QLORA_OK;
}

int view_heads(const qlora_heads* t, AttnTensor& v) {
  if (!t || !t->p) return QLORA_ERR_NULL;
  if (t->token_pitch <= 0 || t->token_pitch >= (int64_t(1) << 24) || t->head_pitch < 0 || t->head_pitch >= kInt32)
    return QLORA_ERR_SHAPE;
  if (!aligned(t->p, 16) || t->token_pitch % 8 != 0 || t->head_pitch % 8 != 0) return QLORA_ERR_ALIGN;
  v.p = t->p;
  v.st = t->token_pitch;
  v.sh = t->head_pitch;
  return QLORA_OK;
}

int fill_attn(const qlora_window_attn* a, AttnArgs& r, int threads) {
  if (!a->cu_q || !a->cu_k) return QLORA_ERR_NULL;
  const int st = check_attn_sizes(a, threads);
  if (st != QLORA_OK) return st;
  if (!aligned(a->cu_q, 4) || !aligned(a->cu_k, 4)) return QLORA_ERR_ALIGN;
  r.cu_q = a->cu_q;
  r.cu_k = a->cu_k;
  r.Tq = a->Tq;
  r.Tk = a->Tk;
  r.B = (int)a->B;
  r.H = (int)a->H;
  r.Hkv = (int)a->Hkv;
  r.D = (int)a->D;
  r.max_q = (int)a->max_q;
  r.max_k = (int)a->max_k;
  // a window past every position is no window; 2^30 keeps sums in 32 bits
  r.window = (int)std::min(a->window, int64_t(1) << 30);
  r.sinks = (int)a->sinks;
  r.scale = a->scale;
  return QLORA_OK;
}

struct BwdLayout {
  size_t delta = 0, lse2 = 0, sink = 0, share = 0, total = 0;
  int parts = 1;
};
BwdLayout plan_bwd(const qlora_window_attn* a) {
  BwdLayout L;
  size_t o = 0;
  const int64_t dp = a->D <= 64 ? 64 : 128;
  L.delta = o;
  o = al256(o + (size_t)a->H * a->Tq * 4);
  L.lse2 = o;
  o = al256(o + (size_t)a->H * a->Tq * 4);
  L.sink = o;
  if (attn_sink_apart(a->max_k, std::min(a->window, int64_t(1) << 30), a->sinks)) {
    const int64_t units = attn_sink_slots(a->Tq, a->B, a->max_q) * a->H + a->B * a->Hkv;
    o = al256(o + (size_t)units * 2 * kMaxSinks * dp * 4);
  }
  L.share = o;
  L.parts = attn_dkv_parts(a->Tk, a->B, a->Hkv, a->H / a->Hkv, a->max_q, std::min(a->window, int64_t(1) << 30));
  if (L.parts > 1) o = al256(o + (size_t)L.parts * a->Tk * a->Hkv * 2 * dp * 4);
  L.total = o;
  return L;
}

int check_decode(int64_t B, int64_t H, int64_t Hkv, int64_t D, int64_t cap, int64_t window, int64_t sinks) {
  if (B < 1 || H < 1 || Hkv < 1 || H % Hkv != 0 || H >= 65536 || cap < 1 || cap >= kInt32 - 4096) return QLORA_ERR_SHAPE;
  if (B >= kInt32 / 128 || B * H >= kInt32 / 128) return QLORA_ERR_SHAPE;
  if (D < 8 || D > 128 || D % 8 != 0) return QLORA_ERR_UNSUPPORTED;
  if (window < 1 || sinks < 0 || sinks > kMaxSinks) return QLORA_ERR_UNSUPPORTED;
  return QLORA_OK;
}
int splits_of(int64_t B, int64_t H, int64_t Hkv, int64_t cap, int64_t window, int64_t sinks) {
  const int64_t most = std::min(cap, std::min(window, cap) + sinks);
  return decode_splits(B, Hkv, H / Hkv, most);
}
size_t decode_bytes(int64_t B, int64_t H, int64_t D, int nsplit, size_t* stat) {
  const size_t part = al256((size_t)B * H * nsplit * D * 4);
  if (stat) *stat = part;
  return nsplit == 1 ? 0 : part + al256((size_t)B * H * nsplit * 2 * 4);
}
int check_cache(const qlora_cache* t, bool tokens) {
  if (!t || !t->p) return QLORA_ERR_NULL;
  const int64_t top = int64_t(1) << 48;
  if (t->request_pitch < 0 || t->head_pitch < 0 || t->request_pitch >= top || t->head_pitch >= top) return QLORA_ERR_SHAPE;
  if (!aligned(t->p, 16) || t->request_pitch % 8 != 0 || t->head_pitch % 8 != 0) return QLORA_ERR_ALIGN;
  if (!tokens) return QLORA_OK;
  if (t->token_pitch < 0 || t->token_pitch >= kInt32) return QLORA_ERR_SHAPE;
  return t->token_pitch % 8 != 0 ? QLORA_ERR_ALIGN : QLORA_OK;
}

// ---------------------------------------------------------------------------
// distillation
// ---------------------------------------------------------------------------
int fill_distill(const qlora_topk_distill* d, DistillArgs& a) {
  if (!d || !d->z || !d->val || !d->idx) return QLORA_ERR_NULL;
  if (d->M < 1 || d->M >= kInt32 || d->V < 1 || d->V >= kInt32 - 64 || d->K < 1 || d->K > kDistillMaxK ||
      d->ldz < d->V || d->ldz >= (int64_t(1) << 40) || d->M * (d->V / 16384 + 1) >= kInt32)
    return QLORA_ERR_SHAPE;
  if (!dtype_ok(d->z_dtype) || !dtype_ok(d->val_dtype) || (d->idx_is_64 != 0 && d->idx_is_64 != 1))
    return QLORA_ERR_UNSUPPORTED;
  if (!std::isfinite(d->temperature) || !(d->temperature > 0.0f) || !std::isfinite(1.0f / d->temperature))
    return QLORA_ERR_UNSUPPORTED;
  if (!aligned(d->z, 16) || !aligned(d->val, 16) || !aligned(d->idx, 16) || !aligned(d->t_lse, 4)) return QLORA_ERR_ALIGN;
  a = DistillArgs{};
  a.z = d->z;
  a.ldz = d->ldz;
  a.M = d->M;
  a.V = d->V;
  a.z_f32 = d->z_dtype == QLORA_F32;
  a.val = d->val;
  a.val_f32 = d->val_dtype == QLORA_F32;
  a.idx = d->idx;
  a.idx_64 = d->idx_is_64 == 1;
  a.K = (int)d->K;
  a.t_lse = d->t_lse;
  a.tau = d->temperature;
  a.inv_tau = 1.0f / d->temperature;
  return QLORA_OK;
}

int check_dz(const qlora_topk_distill* d, const void* dz, int64_t lddz, const float* weight) {
  if (!dz) return QLORA_ERR_NULL;
  if (lddz < d->V || lddz >= (int64_t(1) << 40)) return QLORA_ERR_SHAPE;
  return aligned(dz, 16) && aligned(weight, 4) ? QLORA_OK : QLORA_ERR_ALIGN;
}

}  // namespace

extern "C" {

int qlora_layer_norm_fwd(const void* x, int64_t ldx, int x_dtype, const void* w, const void* b, int w_dtype,
                         int64_t M, int64_t C, float eps, void* y, float* mean, float* rstd, void* stream) {
  const int st = check_norm(x, ldx, x_dtype, w, w_dtype, mean, rstd, M, C);
  if (st != QLORA_OK) return st;
  if (!y) return QLORA_ERR_NULL;
  if (!aligned(y, 16) || !aligned(b, 16)) return QLORA_ERR_ALIGN;
  if (!std::isfinite(eps) || eps < 0.0f) return QLORA_ERR_UNSUPPORTED;
  try {
    NormArgs a{};
    a.x = x;
    a.ldx = ldx;
    a.w = w;
    a.b = b;
    a.M = M;
    a.C = C;
    a.x_f32 = x_dtype == QLORA_F32;
    a.w_f32 = w_dtype == QLORA_F32;
    a.eps = eps;
    a.y = y;
    a.mean = mean;
    a.rstd = rstd;
    return status_of(launch_norm_fwd(a, (hipStream_t)stream));
  } catch (...) {
    return QLORA_ERR_DEVICE;
  }
}

size_t qlora_layer_norm_workspace_bytes(int64_t M, int64_t C) {
  if (M < 1 || M >= kInt32 || C < 1 || C > kNormMaxC) return 0;
  return al256((size_t)norm_groups(M, C) * 2 * C * 4);
}

int qlora_layer_norm_bwd(const void* x, int64_t ldx, int x_dtype, const void* w, int w_dtype, const void* dy,
                         int64_t lddy, const float* mean, const float* rstd, int64_t M, int64_t C, void* dx,
                         void* dw, void* db, void* ws, size_t ws_bytes, void* stream) {
  const int st = check_norm(x, ldx, x_dtype, w, w_dtype, mean, rstd, M, C);
  if (st != QLORA_OK) return st;
  if (!dy || (!dx && !dw && !db)) return QLORA_ERR_NULL;
  if (lddy < C || lddy >= (int64_t(1) << 40)) return QLORA_ERR_SHAPE;
  if (!aligned(dy, 16) || !aligned(dx, 16) || !aligned(dw, 16) || !aligned(db, 16)) return QLORA_ERR_ALIGN;
  if (dw || db) {
    if (!ws || ws_bytes < qlora_layer_norm_workspace_bytes(M, C)) return QLORA_ERR_WORKSPACE;
    if (!aligned(ws, 256)) return QLORA_ERR_ALIGN;
  }
  try {
    NormArgs a{};
    a.x = x;
    a.ldx = ldx;
    a.w = w;
    a.dy = dy;
    a.lddy = lddy;
    a.M = M;
    a.C = C;
    a.x_f32 = x_dtype == QLORA_F32;
    a.w_f32 = w_dtype == QLORA_F32;
    a.mean = const_cast<float*>(mean);
    a.rstd = const_cast<float*>(rstd);
    a.dx = dx;
    a.dw = dw;
    a.db = db;
    a.part = dw || db ? static_cast<float*>(ws) : nullptr;
    return status_of(launch_norm_bwd(a, (hipStream_t)stream));
  } catch (...) {
    return QLORA_ERR_DEVICE;
  }
}

int qlora_window_attn_fwd(const qlora_window_attn* a, const qlora_heads* q, const qlora_heads* k,
                          const qlora_heads* v, const qlora_heads* o, float* lse, void* stream) {
  if (!a || !lse) return QLORA_ERR_NULL;
  AttnArgs r{};
  int st = fill_attn(a, r, kFwdThreads);
  if (st == QLORA_OK) st = view_heads(q, r.q);
  if (st == QLORA_OK) st = view_heads(k, r.k);
  if (st == QLORA_OK) st = view_heads(v, r.v);
  if (st == QLORA_OK) st = view_heads(o, r.o);
  if (st != QLORA_OK) return st;
  if (!aligned(lse, 4)) return QLORA_ERR_ALIGN;
  r.lse = lse;
  try {
    return status_of(launch_attn_fwd(r, (hipStream_t)stream));
  } catch (...) {
    return QLORA_ERR_DEVICE;
  }
}

size_t qlora_window_attn_bwd_workspace_bytes(const qlora_window_attn* a) {
  return a && check_attn_sizes(a, kBwdThreads) == QLORA_OK ? plan_bwd(a).total : 0;
}

int qlora_window_attn_bwd(const qlora_window_attn* a, const qlora_heads* q, const qlora_heads* k,
                          const qlora_heads* v, const qlora_heads* o, const float* lse, const qlora_heads* d_o,
                          const qlora_heads* dq, const qlora_heads* dk, const qlora_heads* dv, void* ws,
                          size_t ws_bytes, void* stream) {
  if (!a || !lse) return QLORA_ERR_NULL;
  AttnArgs r{};
  int st = fill_attn(a, r, kBwdThreads);
  if (st == QLORA_OK) st = view_heads(q, r.q);
  if (st == QLORA_OK) st = view_heads(k, r.k);
  if (st == QLORA_OK) st = view_heads(v, r.v);
  if (st == QLORA_OK) st = view_heads(o, r.o);
  if (st == QLORA_OK) st = view_heads(d_o, r.d_o);
  if (st == QLORA_OK) st = view_heads(dq, r.dq);
  if (st == QLORA_OK) st = view_heads(dk, r.dk);
  if (st == QLORA_OK) st = view_heads(dv, r.dv);
  if (st != QLORA_OK) return st;
  if (!aligned(lse, 4)) return QLORA_ERR_ALIGN;
  const BwdLayout L = plan_bwd(a);
  if (!ws || ws_bytes < L.total) return QLORA_ERR_WORKSPACE;
  if (!aligned(ws, 256)) return QLORA_ERR_ALIGN;
  r.lse = const_cast<float*>(lse);
  r.delta = reinterpret_cast<float*>(static_cast<char*>(ws) + L.delta);
  r.lse2 = reinterpret_cast<float*>(static_cast<char*>(ws) + L.lse2);
  r.sink = reinterpret_cast<float*>(static_cast<char*>(ws) + L.sink);
  r.parts = L.parts;
  r.share = reinterpret_cast<float*>(static_cast<char*>(ws) + L.share);
  try {
    return status_of(launch_attn_bwd(r, (hipStream_t)stream));
  } catch (...) {
    return QLORA_ERR_DEVICE;
  }
}

size_t qlora_window_attn_decode_workspace_bytes(int64_t B, int64_t H, int64_t Hkv, int64_t D, int64_t cap,
                                                int64_t window, int64_t sinks) {
  if (check_decode(B, H, Hkv, D, cap, window, sinks) != QLORA_OK) return 0;
  return decode_bytes(B, H, D, splits_of(B, H, Hkv, cap, window, sinks), nullptr);
}

int qlora_window_attn_decode(const qlora_cache* q, const qlora_cache* k, const qlora_cache* v, const int32_t* lens,
                             int64_t B, int64_t H, int64_t Hkv, int64_t D, int64_t cap, int64_t window,
                             int64_t sinks, float scale, void* o, void* ws, size_t ws_bytes, void* stream) {
  if (!lens || !o) return QLORA_ERR_NULL;
  int st = check_decode(B, H, Hkv, D, cap, window, sinks);
  if (st != QLORA_OK) return st;
  if (!std::isfinite(scale) || !(scale > 0.0f)) return QLORA_ERR_UNSUPPORTED;
  st = check_cache(q, false);
  if (st == QLORA_OK) st = check_cache(k, true);
  if (st == QLORA_OK) st = check_cache(v, true);
  if (st != QLORA_OK) return st;
  if (!aligned(lens, 4) || !aligned(o, 16)) return QLORA_ERR_ALIGN;
  const int nsplit = splits_of(B, H, Hkv, cap, window, sinks);
  size_t stat = 0;
  const size_t need = decode_bytes(B, H, D, nsplit, &stat);
  if (need > 0) {
    if (!ws || ws_bytes < need) return QLORA_ERR_WORKSPACE;
    if (!aligned(ws, 256)) return QLORA_ERR_ALIGN;
  }
  try {
    DecodeArgs a{};
    a.q = static_cast<const uint16_t*>(q->p);
    a.q_sb = q->request_pitch;
    a.q_sh = q->head_pitch;
    a.k = static_cast<const uint16_t*>(k->p);
    a.k_sb = k->request_pitch;
    a.k_st = k->token_pitch;
    a.k_sh = k->head_pitch;
    a.v = static_cast<const uint16_t*>(v->p);
    a.v_sb = v->request_pitch;
    a.v_st = v->token_pitch;
    a.v_sh = v->head_pitch;
    a.lens = lens;
    a.B = (int)B;
    a.H = (int)H;
    a.Hkv = (int)Hkv;
    a.D = (int)D;
    a.cap = (int)cap;
    a.window = (int)std::min(window, cap);
    a.sinks = (int)sinks;
    a.scale = scale;
    a.o = static_cast<uint16_t*>(o);
    a.nsplit = nsplit;
    if (need > 0) {
      a.part = static_cast<float*>(ws);
      a.stat = reinterpret_cast<float*>(static_cast<char*>(ws) + stat);
    }
    return status_of(launch_decode(a, (hipStream_t)stream));
  } catch (...) {
    return QLORA_ERR_DEVICE;
  }
}

int qlora_topk_distill_fwd(const qlora_topk_distill* d, float* loss, float* lse, void* stream) {
  DistillArgs a;
  const int st = fill_distill(d, a);
  if (st != QLORA_OK) return st;
  if (!loss || !lse) return QLORA_ERR_NULL;
  if (!aligned(loss, 4) || !aligned(lse, 4)) return QLORA_ERR_ALIGN;
  a.loss = loss;
  a.lse = lse;
  try {
    return status_of(launch_distill_fwd(a, false, (hipStream_t)stream));
  } catch (...) {
    return QLORA_ERR_DEVICE;
  }
}

int qlora_topk_distill_bwd(const qlora_topk_distill* d, const float* lse, const float* weight, void* dz,
                           int64_t lddz, void* stream) {
  DistillArgs a;
  int st = fill_distill(d, a);
  if (st != QLORA_OK) return st;
  if (!lse) return QLORA_ERR_NULL;
  st = check_dz(d, dz, lddz, weight);
  if (st != QLORA_OK) return st;
  if (!aligned(lse, 4)) return QLORA_ERR_ALIGN;
  a.lse = const_cast<float*>(lse);
  a.weight = weight;
  a.dz = dz;
  a.lddz = lddz;
  try {
    return status_of(launch_distill_bwd(a, (hipStream_t)stream));
  } catch (...) {
    return QLORA_ERR_DEVICE;
  }
}

int qlora_topk_distill_fwd_bwd(const qlora_topk_distill* d, const float* weight, float* loss, float* lse, void* dz,
                               int64_t lddz, void* stream) {
  DistillArgs a;
  int st = fill_distill(d, a);
  if (st != QLORA_OK) return st;
  if (!loss || !lse) return QLORA_ERR_NULL;
  st = check_dz(d, dz, lddz, weight);
  if (st != QLORA_OK) return st;
  if (!aligned(loss, 4) || !aligned(lse, 4)) return QLORA_ERR_ALIGN;
  a.loss = loss;
  a.lse = lse;
  a.weight = weight;
  a.dz = dz;
  a.lddz = lddz;
  try {
    return status_of(launch_distill_fwd(a, true, (hipStream_t)stream));
  } catch (...) {
    return QLORA_ERR_DEVICE;
  }
}

}  // extern "C"
