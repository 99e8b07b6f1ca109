"""Attention into tensors that the caller lays out."""

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
