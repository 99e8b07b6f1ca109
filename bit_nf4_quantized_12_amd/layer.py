"""Operators around the linears of a decoder layer: layer norm, attention with a
sliding window and first tokens that stay visible, and distillation against a
teacher's top logits.

Argument marshalling for the C ABI (include/qlora.h), with the conventions of
the package: every tensor on one GPU, work on that GPU's current stream, outputs
new tensors unless the caller hands in his own, ``QloraError`` for a status of
the library. The ``...Function`` classes at the end wrap the calls for torch's
automatic differentiation, once: the gradient of a gradient is refused.
"""

import ctypes

import torch
from torch.autograd.function import once_differentiable

from . import QLORA_BF16, QLORA_F32, _check, load_library, new_workspace

_DTYPES = {torch.float32: QLORA_F32, torch.bfloat16: QLORA_BF16}
_vp, _i64, _i32, _f32, _sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_size_t


class _Heads(ctypes.Structure):
    _fields_ = [("p", _vp), ("token_pitch", _i64), ("head_pitch", _i64)]


class _Cache(ctypes.Structure):
    _fields_ = [("p", _vp), ("request_pitch", _i64), ("token_pitch", _i64), ("head_pitch", _i64)]


class _WindowAttn(ctypes.Structure):
    _fields_ = [("cu_q", _vp), ("cu_k", _vp), ("B", _i64), ("Tq", _i64), ("Tk", _i64), ("H", _i64), ("Hkv", _i64),
                ("D", _i64), ("max_q", _i64), ("max_k", _i64), ("window", _i64), ("sinks", _i64), ("scale", _f32)]


class _TopkDistill(ctypes.Structure):
    _fields_ = [("M", _i64), ("V", _i64), ("K", _i64), ("z", _vp), ("ldz", _i64), ("z_dtype", _i32), ("val", _vp),
                ("val_dtype", _i32), ("idx", _vp), ("idx_is_64", _i32), ("t_lse", _vp), ("temperature", _f32)]


def signatures():
    """Argument and result types of this module's library calls."""
    heads, cache, attn, dist = (ctypes.POINTER(t) for t in (_Heads, _Cache, _WindowAttn, _TopkDistill))
    return {
        "qlora_layer_norm_fwd": ([_vp, _i64, _i32, _vp, _vp, _i32, _i64, _i64, _f32, _vp, _vp, _vp, _vp], _i32),
        "qlora_layer_norm_workspace_bytes": ([_i64, _i64], _sz),
        "qlora_layer_norm_bwd": ([_vp, _i64, _i32, _vp, _i32, _vp, _i64, _vp, _vp, _i64, _i64, _vp, _vp, _vp, _vp, _sz,
                                  _vp], _i32),
        "qlora_window_attn_fwd": ([attn, heads, heads, heads, heads, _vp, _vp], _i32),
        "qlora_window_attn_bwd_workspace_bytes": ([attn], _sz),
        "qlora_window_attn_bwd": ([attn, heads, heads, heads, heads, _vp, heads, heads, heads, heads, _vp, _sz, _vp],
                                  _i32),
        "qlora_window_attn_decode_workspace_bytes": ([_i64] * 7, _sz),
        "qlora_window_attn_decode": ([cache, cache, cache, _vp, _i64, _i64, _i64, _i64, _i64, _i64, _i64, _f32, _vp,
                                      _vp, _sz, _vp], _i32),
        "qlora_topk_distill_fwd": ([dist, _vp, _vp, _vp], _i32),
        "qlora_topk_distill_bwd": ([dist, _vp, _vp, _vp, _i64, _vp], _i32),
        "qlora_topk_distill_fwd_bwd": ([dist, _vp, _vp, _vp, _vp, _i64, _vp], _i32),
    }


def _stream(dev):
    """Address of the current stream of dev (a torch Stream object costs 2 us more: as much as a small kernel)."""
    return torch._C._cuda_getCurrentRawStream(dev.index)


def _gpu(t, dtype, dev, name):
    """t is a GPU tensor of this type (a torch dtype or several) on device dev (None: any)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    if t.dtype != dtype and not (isinstance(dtype, tuple) and t.dtype in dtype):
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if dev is not None and t.device != dev:
        raise ValueError(f"{name} is on {t.device}, the other operands on {dev}")


def _whole(t, shape, dtype, dev, name):
    """t is a contiguous GPU tensor of this shape and type."""
    _gpu(t, dtype, dev, name)
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _out(t, shape, dtype, dev, name):
    if t is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    _whole(t, shape, dtype, dev, name)
    return t


def _scratch(t, need, dev):
    """The caller's workspace when it is large enough, else a new one."""
    if t is None:
        return new_workspace(need, dev)
    _gpu(t, torch.uint8, dev, "workspace")
    if not t.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return t if t.numel() >= need else new_workspace(need, dev)


def _pitch(t, name):
    """Row pitch of a 2-D tensor whose rows are contiguous."""
    rows, cols = t.shape
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have contiguous rows")
    ld = t.stride(0) if rows > 1 else cols
    if ld < cols:
        raise ValueError(f"{name} must have rows that do not overlap")
    return ld


_FLOATS = (torch.float32, torch.bfloat16)


# ---------------------------------------------------------------------------
# layer norm
# ---------------------------------------------------------------------------

def qlora_layer_norm_fwd(x, weight, bias=None, eps=1e-5, y=None, mean=None, rstd=None):
    """y = (x - mean) rstd weight + bias over the rows of x [M, C] (bf16 or float32).

    Returns (y, mean, rstd) with the statistics float32 [M]. weight and bias [C] are of
    one type, bf16 or float32; rows of x may have any pitch.
    """
    _gpu(x, _FLOATS, None, "x")
    if x.dim() != 2:
        raise ValueError("x must be 2-D [M, C]")
    M, C = x.shape
    dev, ld = x.device, _pitch(x, "x")
    _whole(weight, (C,), _FLOATS, dev, "weight")
    if bias is not None:
        _whole(bias, (C,), weight.dtype, dev, "bias")
    y = _out(y, (M, C), x.dtype, dev, "y")
    mean = _out(mean, (M,), torch.float32, dev, "mean")
    rstd = _out(rstd, (M,), torch.float32, dev, "rstd")
    _check(load_library().qlora_layer_norm_fwd(
        x.data_ptr(), ld, _DTYPES[x.dtype], weight.data_ptr(), None if bias is None else bias.data_ptr(),
        _DTYPES[weight.dtype], M, C, eps, y.data_ptr(), mean.data_ptr(), rstd.data_ptr(), _stream(dev)))
    return y, mean, rstd


def qlora_layer_norm_workspace_bytes(M, C):
    return int(load_library().qlora_layer_norm_workspace_bytes(M, C))


def qlora_layer_norm_bwd(x, weight, dy, mean, rstd, need_dx=True, need_dw=True, need_db=True, dx=None, dw=None,
                         db=None, workspace=None):
    """Gradients (dx, dw, db) of qlora_layer_norm_fwd for dy; None in the place of one that is not needed."""
    _gpu(x, _FLOATS, None, "x")
    if x.dim() != 2:
        raise ValueError("x must be 2-D [M, C]")
    M, C = x.shape
    dev, ld = x.device, _pitch(x, "x")
    _whole(weight, (C,), _FLOATS, dev, "weight")
    _gpu(dy, x.dtype, dev, "dy")
    if dy.shape != x.shape:
        raise ValueError(f"dy must have shape {tuple(x.shape)}, got {tuple(dy.shape)}")
    lddy = _pitch(dy, "dy")
    _whole(mean, (M,), torch.float32, dev, "mean")
    _whole(rstd, (M,), torch.float32, dev, "rstd")
    if not (need_dx or need_dw or need_db):
        return None, None, None
    dx = _out(dx, (M, C), x.dtype, dev, "dx") if need_dx else None
    dw = _out(dw, (C,), weight.dtype, dev, "dw") if need_dw else None
    db = _out(db, (C,), weight.dtype, dev, "db") if need_db else None
    lib = load_library()
    if need_dw or need_db:
        need = lib.qlora_layer_norm_workspace_bytes(M, C)
        ws = _scratch(workspace, need, dev)
        wp, wn = ws.data_ptr(), ws.numel()
    else:
        wp, wn = None, 0
    _check(lib.qlora_layer_norm_bwd(
        x.data_ptr(), ld, _DTYPES[x.dtype], weight.data_ptr(), _DTYPES[weight.dtype], dy.data_ptr(), lddy,
        mean.data_ptr(), rstd.data_ptr(), M, C, None if dx is None else dx.data_ptr(),
        None if dw is None else dw.data_ptr(), None if db is None else db.data_ptr(), wp, wn, _stream(dev)))
    return dx, dw, db


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

def _heads(t, dev, name, shape=None):
    """[tokens, heads, D] bf16 with contiguous D as the library's view of it."""
    _gpu(t, torch.bfloat16, dev, name)
    if t.dim() != 3:
        raise ValueError(f"{name} must be 3-D [tokens, heads, D]")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    st, sh, sd = t.stride()
    if t.shape[2] > 1 and sd != 1:
        raise ValueError(f"{name} must be contiguous along D")
    if t.shape[0] == 1:
        st = max(8, t.shape[1] * t.shape[2])  # never used: one token
    if t.shape[1] == 1:
        sh = t.shape[2]
    return _Heads(t.data_ptr(), st, sh)


def _heads_out(t, shape, dev, name):
    """A new [tokens, heads, D] tensor, or the caller's (a slice of a larger one, or heads first, for instance)
    after checking that its elements lie apart."""
    if t is None:
        t = torch.empty(shape, dtype=torch.bfloat16, device=dev)
        return t, _Heads(t.data_ptr(), shape[1] * shape[2], shape[2])
    view = _heads(t, dev, name, shape)
    # from the smaller pitch to the larger, each steps over all that lies below it (a pitch of one element is not used)
    below = shape[2]
    for pitch, n in sorted((p, n) for p, n in ((view.token_pitch, shape[0]), (view.head_pitch, shape[1])) if n > 1):
        if pitch < below:
            raise ValueError(f"{name} must not overlap itself")
        below += (n - 1) * pitch
    return t, view


def _packed(q, k, v, cu_q, cu_k, max_q, max_k, window, sinks, scale):
    """(device, struct of sizes, views of q, k, v)."""
    hq = _heads(q, None, "q")
    dev = q.device
    Tq, H, D = q.shape
    hk = _heads(k, dev, "k")
    Tk, Hkv, Dk = k.shape
    if Dk != D:
        raise ValueError(f"q has {D} columns a head, k {Dk}")
    hv = _heads(v, dev, "v", k.shape)
    if cu_k is None:
        cu_k, max_k = cu_q, max_q if max_k is None else max_k
    for t, name in ((cu_q, "cu_q"),) if cu_k is cu_q else ((cu_q, "cu_q"), (cu_k, "cu_k")):
        _gpu(t, torch.int32, dev, name)
        if t.dim() != 1 or t.numel() < 2 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous int32 vector of the sequences' starts and the end")
    if cu_k.numel() != cu_q.numel():
        raise ValueError("cu_q and cu_k must name the same number of sequences")
    a = _WindowAttn(cu_q.data_ptr(), cu_k.data_ptr(), cu_q.numel() - 1, Tq, Tk, H, Hkv, D, max_q,
                    Tk if max_k is None else max_k, window, sinks, D ** -0.5 if scale is None else scale)
    return dev, a, hq, hk, hv


def qlora_window_attn_fwd(q, k, v, cu_q, max_q, window, sinks=0, cu_k=None, scale=None, o=None, lse=None):
    """Attention of packed sequences with a sliding window and first tokens that stay visible.

    q [Tq, H, D], k and v [Tk, Hkv, D] bf16 (any token and head pitch of 16-byte multiples),
    cu_q and cu_k int32 [B + 1] starts of the sequences (cu_k None: those of q). The queries
    of a sequence stand at the end of its keys; one at position p sees key j when j <= p and
    (j > p - window or j < sinks). max_q: the longest sequence's queries. scale: D^-1/2 when
    None. Returns (o [Tq, H, D] bf16, lse [H, Tq] float32). Rows past the last sequence's
    end get o = 0 and lse = -inf (zeros in the backward).
    """
    dev, a, hq, hk, hv = _packed(q, k, v, cu_q, cu_k, max_q, max_q, window, sinks, scale)
    o, ho = _heads_out(o, q.shape, dev, "o")
    lse = _out(lse, (q.shape[1], q.shape[0]), torch.float32, dev, "lse")
    _check(load_library().qlora_window_attn_fwd(a, hq, hk, hv, ho, lse.data_ptr(), _stream(dev)))
    return o, lse


def qlora_window_attn_bwd(q, k, v, o, lse, d_o, cu_q, max_q, window, sinks=0, cu_k=None, max_k=None, scale=None,
                          dq=None, dk=None, dv=None, workspace=None):
    """Gradients (dq, dk, dv), bf16, of qlora_window_attn_fwd for d_o, from its o and lse.

    max_k: the longest sequence's keys (None: those of q without cu_k, else all of k).
    """
    dev, a, hq, hk, hv = _packed(q, k, v, cu_q, cu_k, max_q, max_k, window, sinks, scale)
    ho = _heads(o, dev, "o", q.shape)
    _whole(lse, (q.shape[1], q.shape[0]), torch.float32, dev, "lse")
    hg = _heads(d_o, dev, "d_o", q.shape)
    dq, gq = _heads_out(dq, q.shape, dev, "dq")
    dk, gk = _heads_out(dk, k.shape, dev, "dk")
    dv, gv = _heads_out(dv, k.shape, dev, "dv")
    lib = load_library()
    need = lib.qlora_window_attn_bwd_workspace_bytes(a)
    ws = _scratch(workspace, need, dev)
    _check(lib.qlora_window_attn_bwd(a, hq, hk, hv, ho, lse.data_ptr(), hg, gq, gk, gv, ws.data_ptr(), ws.numel(),
                                     _stream(dev)))
    return dq, dk, dv


def _cache_view(t, dev, name, shape=None):
    _gpu(t, torch.bfloat16, dev, name)
    if t.dim() != 4:
        raise ValueError(f"{name} must be 4-D [requests, positions, heads, D]")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.shape[3] > 1 and t.stride(3) != 1:
        raise ValueError(f"{name} must be contiguous along D")
    pitch = [s if n > 1 else 0 for n, s in zip(t.shape[:3], t.stride()[:3])]
    return _Cache(t.data_ptr(), *pitch)


def qlora_window_attn_decode(q, k_cache, v_cache, lens, window, sinks=0, scale=None, o=None, workspace=None):
    """One new token per request: q [B, H, D] against the caches [B, cap, Hkv, D] (bf16), of
    which request b holds lens[b] (int32 [B]) positions, the new token's own the last of them.
    Returns o [B, H, D]; a request of length 0 gives zeros.
    """
    _gpu(q, torch.bfloat16, None, "q")
    if q.dim() != 3 or (q.shape[2] > 1 and q.stride(2) != 1):
        raise ValueError("q must be 3-D [B, H, D], contiguous along D")
    dev = q.device
    B, H, D = q.shape
    ck = _cache_view(k_cache, dev, "k_cache")
    cv = _cache_view(v_cache, dev, "v_cache", k_cache.shape)
    if k_cache.shape[0] != B or k_cache.shape[3] != D:
        raise ValueError("shape mismatch: q [B, H, D], caches [B, cap, Hkv, D]")
    cap, Hkv = k_cache.shape[1], k_cache.shape[2]
    _whole(lens, (B,), torch.int32, dev, "lens")
    o = _out(o, (B, H, D), torch.bfloat16, dev, "o")
    cq = _Cache(q.data_ptr(), q.stride(0) if B > 1 else 0, 0, q.stride(1) if H > 1 else 0)
    lib = load_library()
    need = lib.qlora_window_attn_decode_workspace_bytes(B, H, Hkv, D, cap, window, sinks)
    ws = _scratch(workspace, need, dev) if need else None
    wp, wn = (None, 0) if ws is None else (ws.data_ptr(), ws.numel())
    _check(lib.qlora_window_attn_decode(cq, ck, cv, lens.data_ptr(), B, H, Hkv, D, cap, window, sinks,
                                        D ** -0.5 if scale is None else scale, o.data_ptr(), wp, wn, _stream(dev)))
    return o


# ---------------------------------------------------------------------------
# distillation
# ---------------------------------------------------------------------------

def _distill(logits, t_val, t_idx, temperature, t_lse):
    _gpu(logits, _FLOATS, None, "logits")
    if logits.dim() != 2:
        raise ValueError("logits must be 2-D [M, V]")
    M, V = logits.shape
    dev = logits.device
    _gpu(t_val, _FLOATS, dev, "t_val")
    if t_val.dim() != 2 or t_val.shape[0] != M:
        raise ValueError(f"t_val must have shape [{M}, K]")
    K = t_val.shape[1]
    _whole(t_val, (M, K), _FLOATS, dev, "t_val")
    _whole(t_idx, (M, K), (torch.int32, torch.int64), dev, "t_idx")
    if t_lse is not None:
        _whole(t_lse, (M,), torch.float32, dev, "t_lse")
    d = _TopkDistill(M, V, K, logits.data_ptr(), _pitch(logits, "logits"), _DTYPES[logits.dtype], t_val.data_ptr(),
                     _DTYPES[t_val.dtype], t_idx.data_ptr(), 1 if t_idx.dtype == torch.int64 else 0,
                     None if t_lse is None else t_lse.data_ptr(), temperature)
    return dev, M, V, d


def _dlogits(t, logits, weight, name):
    """The gradient's tensor and pitch, and the weights' address."""
    M, V = logits.shape
    dev = logits.device
    if weight is not None:
        _whole(weight, (M,), torch.float32, dev, name)
    if t is None:
        t = torch.empty((M, V), dtype=logits.dtype, device=dev)
    else:
        _gpu(t, logits.dtype, dev, "dlogits")
        if t.shape != logits.shape:
            raise ValueError(f"dlogits must have shape {(M, V)}, got {tuple(t.shape)}")
    return t, _pitch(t, "dlogits"), None if weight is None else weight.data_ptr()


def qlora_topk_distill_fwd(logits, t_val, t_idx, temperature=1.0, t_lse=None, loss=None, lse=None):
    """Loss of each row of logits [M, V] (bf16 or float32) against a teacher's top entries.

    t_val [M, K] (bf16 or float32) teacher logits at the vocabulary indices t_idx [M, K]
    (int32 or int64; one outside [0, V), such as -1, is no entry). The teacher's
    probabilities are the softmax of t_val / temperature over the row's entries or, with
    t_lse [M], exp(t_val / temperature - t_lse). Returns (loss, lse), float32 [M]:
    loss = temperature^2 sum_k p_k (log p_k - log softmax(logits / temperature)[idx_k]).
    """
    dev, M, _, d = _distill(logits, t_val, t_idx, temperature, t_lse)
    loss = _out(loss, (M,), torch.float32, dev, "loss")
    lse = _out(lse, (M,), torch.float32, dev, "lse")
    _check(load_library().qlora_topk_distill_fwd(d, loss.data_ptr(), lse.data_ptr(), _stream(dev)))
    return loss, lse


def qlora_topk_distill_bwd(logits, t_val, t_idx, lse, dloss=None, temperature=1.0, t_lse=None, dlogits=None):
    """Gradient [M, V] of qlora_topk_distill_fwd for the rows' upstream gradients dloss (float32
    [M]; None: ones). dlogits may be logits itself."""
    dev, M, _, d = _distill(logits, t_val, t_idx, temperature, t_lse)
    _whole(lse, (M,), torch.float32, dev, "lse")
    dlogits, ld, w = _dlogits(dlogits, logits, dloss, "dloss")
    _check(load_library().qlora_topk_distill_bwd(d, lse.data_ptr(), w, dlogits.data_ptr(), ld, _stream(dev)))
    return dlogits


def qlora_topk_distill_fwd_bwd(logits, t_val, t_idx, row_weight=None, temperature=1.0, t_lse=None, dlogits=None,
                               loss=None, lse=None):
    """Loss and gradient in one pass over the logits, for row weights that are known beforehand
    (1 / tokens for a mean, 0 for tokens without loss; None: ones). Returns (loss, lse,
    dlogits); loss is not weighted. dlogits may be logits itself."""
    dev, M, _, d = _distill(logits, t_val, t_idx, temperature, t_lse)
    loss = _out(loss, (M,), torch.float32, dev, "loss")
    lse = _out(lse, (M,), torch.float32, dev, "lse")
    dlogits, ld, w = _dlogits(dlogits, logits, row_weight, "row_weight")
    _check(load_library().qlora_topk_distill_fwd_bwd(d, w, loss.data_ptr(), lse.data_ptr(), dlogits.data_ptr(), ld,
                                                     _stream(dev)))
    return loss, lse, dlogits


# ---------------------------------------------------------------------------
# automatic differentiation
# ---------------------------------------------------------------------------

# Other operations leave slices that start off 16 bytes (rows of an odd width from the second on), expanded and
# transposed tensors; the calls above refuse them, the functions below copy them.

def _aligned(t):
    """t as a contiguous tensor that starts on 16 bytes (itself, or a copy); None stays."""
    if t is None:
        return None
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


def _rows(t):
    """[M, C] t itself where the calls take it: contiguous rows that lie apart and start on 16 bytes; else a copy."""
    if t.dim() != 2:
        return t
    ok = (t.shape[1] == 1 or t.stride(1) == 1) and (t.shape[0] == 1 or t.stride(0) >= t.shape[1])
    return t if ok and t.data_ptr() % 16 == 0 else t.clone(memory_format=torch.contiguous_format)


def _head_rows(t):
    """[tokens, heads, D] t itself where the calls take it (contiguous along D, pitches of 16-byte multiples within
    their limits); else a copy."""
    if t.dim() != 3:
        return t
    (T, H, D), (st, sh, sd) = t.shape, t.stride()
    ok = ((D == 1 or sd == 1) and (T == 1 or (0 < st < 1 << 24 and st % 8 == 0))
          and (H == 1 or (sh < 1 << 31 and sh % 8 == 0)))
    return t if ok and t.data_ptr() % 16 == 0 else t.clone(memory_format=torch.contiguous_format)


class LayerNormFunction(torch.autograd.Function):
    """y = layer norm of x [M, C] with weight and bias (bias may be None)."""

    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        x, weight, bias = _rows(x), _aligned(weight), _aligned(bias)
        y, mean, rstd = qlora_layer_norm_fwd(x, weight, bias, eps)
        ctx.save_for_backward(x, weight, mean, rstd)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, weight, mean, rstd = ctx.saved_tensors
        need = ctx.needs_input_grad
        return (*qlora_layer_norm_bwd(x, weight, _aligned(dy), mean, rstd, *need[:3]), None)


class WindowAttnFunction(torch.autograd.Function):
    """o of qlora_window_attn_fwd for q, k, v of sequences that start at cu [B + 1]; after prefixes, keys and
    values of sequences that start at cu_k (longest_k: the longest one's keys, None: all of k)."""

    @staticmethod
    def forward(ctx, q, k, v, cu, longest, window, sinks, scale, cu_k=None, longest_k=None):
        q, k, v = _head_rows(q), _head_rows(k), _head_rows(v)
        o, lse = qlora_window_attn_fwd(q, k, v, cu, longest, window, sinks, cu_k=cu_k, scale=scale)
        ctx.save_for_backward(q, k, v, o, lse, cu, cu_k)
        ctx.rest = (longest, window, sinks)
        ctx.opts = dict(max_k=longest_k, scale=scale)
        return o

    @staticmethod
    @once_differentiable
    def backward(ctx, d_o):
        q, k, v, o, lse, cu, cu_k = ctx.saved_tensors
        grads = qlora_window_attn_bwd(q, k, v, o, lse, _aligned(d_o), cu, *ctx.rest, cu_k=cu_k, **ctx.opts)
        return (*grads, None, None, None, None, None, None, None)


class TopkDistillFunction(torch.autograd.Function):
    """Loss [M] of logits against a teacher's entries (qlora_topk_distill_fwd)."""

    @staticmethod
    def forward(ctx, logits, t_val, t_idx, temperature, t_lse):
        logits, t_val, t_idx = _rows(logits), _aligned(t_val), _aligned(t_idx)
        loss, lse = qlora_topk_distill_fwd(logits, t_val, t_idx, temperature, t_lse)
        ctx.save_for_backward(logits, t_val, t_idx, lse, t_lse)
        ctx.temperature = temperature
        return loss

    @staticmethod
    @once_differentiable
    def backward(ctx, dloss):
        logits, t_val, t_idx, lse, t_lse = ctx.saved_tensors
        grad = qlora_topk_distill_bwd(logits, t_val, t_idx, lse, dloss.contiguous(), ctx.temperature, t_lse)
        return grad, None, None, None, None
