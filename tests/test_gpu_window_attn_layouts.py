"""Attention into tensors that the caller lays out, and packed batches whose
arrays are longer than their sequences."""

import pytest
import torch

import bit_nf4_quantized_12_amd as q
from tests import test_gpu_window_attn as wa
from tests.parity import report

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
NAN = float("nan")


def _calls(lens, h, hkv, d, make):
    """o, lse, dq, dk, dv with the bf16 ones written into make(shape), and the same from the call's own tensors."""
    qt, kt, vt, gt = wa._make(lens, lens, h, hkv, d, 2)
    cu, n, args = wa._starts(lens), max(lens), (40, 3)
    want = q.qlora_window_attn_fwd(qt, kt, vt, cu, n, *args)
    o, lse = q.qlora_window_attn_fwd(qt, kt, vt, cu, n, *args, o=make(qt.shape))
    grads = q.qlora_window_attn_bwd(qt, kt, vt, o, lse, gt, cu, n, *args, dq=make(qt.shape), dk=make(kt.shape),
                                    dv=make(kt.shape))
    return (o, lse, *grads), (*want, *q.qlora_window_attn_bwd(qt, kt, vt, *want, gt, cu, n, *args))


@pytest.mark.parametrize("lens,h,hkv,d", [([90, 41], 4, 2, 64), ([7], 3, 3, 128), ([1], 4, 2, 64), ([50], 1, 1, 64)])
@pytest.mark.parametrize("form", ["heads first", "every second head", "a wider token"])
def test_outputs_in_other_orders(lens, h, hkv, d, form):
    report(f"attention outputs, {form}: {lens} H={h}/{hkv} D={d}")
    around = []

    def make(shape):
        t, n, c = shape
        if form == "heads first":
            whole = torch.full((n, t + 3, c), NAN, dtype=torch.bfloat16, device=DEV)
            view, rest = whole[:, :t].transpose(0, 1), whole[:, t:]
        elif form == "every second head":
            whole = torch.full((t, 2 * n, c), NAN, dtype=torch.bfloat16, device=DEV)
            view, rest = whole[:, ::2], whole[:, 1::2]
        else:
            whole = torch.full((t, n, c + 8), NAN, dtype=torch.bfloat16, device=DEV)
            view, rest = whole[:, :, :c], whole[:, :, c:]
        around.append(rest)
        return view

    got, want = _calls(lens, h, hkv, d, make)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert all(r.isnan().all() for r in around)


def test_outputs_that_overlap_themselves_are_refused():
    qt, kt, vt, gt = wa._make([20], [20], 4, 2, 64, 0)
    whole = torch.zeros(20 * 4 * 64 + 1024, dtype=torch.bfloat16, device=DEV)
    for strides in ((0, 64, 1), (256, 0, 1), (128, 64, 1), (64, 64 * 19, 1), (256, 32, 1), (32, 1280, 1)):
        with pytest.raises(ValueError, match="overlap"):
            q.qlora_window_attn_fwd(qt, kt, vt, wa._starts([20]), 20, 8, o=whole.as_strided((20, 4, 64), strides))


# one to many key blocks: the gradients' kernels in parts, in two streams, whole; and sequences that are all empty
@pytest.mark.parametrize("lens,h,hkv,window", [([70, 0, 300], 8, 1, 300), ([130] * 90, 4, 4, 40), ([3, 1, 0, 70] * 300, 2, 1, 20),
                                               ([0, 0], 2, 2, 9), ([1500, 0], 2, 1, 64)])
@pytest.mark.parametrize("d", [64, 128])
def test_rows_of_no_sequence(lens, h, hkv, window, d):
    """Arrays of a fixed size hold batches of any: what lies past the last sequence sees nothing and is not seen."""
    rest, sinks = 77, 2
    report(f"rows of no sequence: {len(lens)} sequences, {sum(lens)} + {rest} rows, H={h}/{hkv} D={d}")
    n = sum(lens)
    qt, kt, vt, gt = wa._make([n + rest], [n + rest], h, hkv, d, 2)
    cu, longest = wa._starts(lens), max(max(lens), 1)
    for t in (qt, kt, vt, gt):
        t[n:] = NAN
    fill = lambda t: torch.full_like(t, NAN)  # noqa: E731
    lse = torch.full((h, n + rest), NAN, device=DEV)
    o, _ = q.qlora_window_attn_fwd(qt, kt, vt, cu, longest, window, sinks, o=fill(qt), lse=lse)
    assert torch.all(o[n:] == 0) and torch.isneginf(lse[:, n:]).all()
    grads = q.qlora_window_attn_bwd(qt, kt, vt, o, lse, gt, cu, longest, window, sinks, dq=fill(qt), dk=fill(kt),
                                    dv=fill(vt))
    for t in grads:
        assert torch.all(t[n:] == 0) and torch.isfinite(t).all()
    if n == 0:
        return
    cut = [t[:n] for t in (qt, kt, vt)]
    want = q.qlora_window_attn_fwd(*cut, cu, longest, window, sinks)
    assert torch.equal(o[:n], want[0]) and torch.equal(lse[:, :n], want[1])
    back = q.qlora_window_attn_bwd(*cut, *want, gt[:n], cu, longest, window, sinks)
    assert torch.equal(grads[0][:n], back[0])
    # (one more row can change how the walks over the queries are cut: another order of float32 sums)
    wa._oracle_check(qt[:n], kt[:n], vt[:n], gt[:n], lens, lens, window, sinks, d ** -0.5, want, [t[:n] for t in grads])


def test_rows_of_no_sequence_under_autograd():
    qt, kt, vt, gt = wa._make([90], [90], 2, 2, 64, 6)
    leaf = [t.clone().requires_grad_() for t in (qt, kt, vt)]
    torch.full((1 << 24,), NAN, device=DEV)  # (memory that new tensors may get)
    o = q.WindowAttnFunction.apply(*leaf, wa._starts([50, 20]), 50, 30, 2, None)
    o.backward(gt)
    assert torch.all(o[70:] == 0) and all(torch.all(t.grad[70:] == 0) for t in leaf)
