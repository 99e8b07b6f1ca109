"""The autograd functions of the linears, norm, attention and distillation inside
larger graphs."""

import pytest
import torch

import bit_nf4_quantized_12_amd as q
from tests import test_gpu_distill as td
from tests import test_gpu_window_attn as wa

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _randn(g, *shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g).to(dtype).to(DEV)


def _attn(qt, kt, vt, cu, n, *rest):
    return q.WindowAttnFunction.apply(qt, kt, vt, cu, n, 30, 2, None, *rest)


def _norm_graph():
    g = torch.Generator().manual_seed(1)
    x, w, b = (_randn(g, *s, dtype=torch.float32).requires_grad_() for s in ((4, 32), (32,), (32,)))
    return q.LayerNormFunction.apply(x, w, b, 1e-5), x


def _attn_graph():
    leaf = [t.requires_grad_() for t in wa._make([20], [20], 2, 2, 64, 1)[:3]]
    return _attn(*leaf, wa._starts([20]), 20), leaf[0]


def _distill_graph():
    z, val, idx, _, _ = td._make(4, 50, 6, "f32", 2.0, False, 7)
    z.requires_grad_()
    return q.TopkDistillFunction.apply(z, val, idx, 2.0, None), z


def _linear_graph():
    g = torch.Generator().manual_seed(1)
    weight = q.quantize_weight(_randn(g, 64, 64))
    x, a, b = (_randn(g, *s).requires_grad_() for s in ((8, 64), (8, 64), (64, 8)))
    return q.LoRALinear4bitFunction.apply(x, a, b, weight, 2.0), x


@pytest.mark.parametrize("graph", [_linear_graph, _norm_graph, _attn_graph, _distill_graph])
def test_derivatives_of_gradients_are_refused(graph):
    out, leaf = graph()
    grad, = torch.autograd.grad(out.float().square().sum(), leaf, create_graph=True)
    # a penalty on the gradient beside another term: it must not be left out in silence
    with pytest.raises(RuntimeError, match="once_differentiable"):
        (grad.float().square().sum() + leaf.float().sum()).backward()


def test_attention_after_a_prefix():
    lq, lk = [30, 1, 50], [90, 200, 50]
    qt, kt, vt, gt = wa._make(lq, lk, 4, 2, 64, 6)
    cu_q, cu_k = wa._starts(lq), wa._starts(lk)
    leaf = [t.clone().requires_grad_() for t in (qt, kt, vt)]
    o = _attn(*leaf, cu_q, 50, cu_k, 200)
    o.backward(gt)
    fwd = q.qlora_window_attn_fwd(qt, kt, vt, cu_q, 50, 30, 2, cu_k=cu_k)
    assert torch.equal(o, fwd[0])
    for t, x in zip(leaf, q.qlora_window_attn_bwd(qt, kt, vt, *fwd, gt, cu_q, 50, 30, 2, cu_k=cu_k, max_k=200)):
        assert torch.equal(t.grad, x)
    wa._oracle_check(qt, kt, vt, gt, lq, lk, 30, 2, 64 ** -0.5, fwd, [t.grad for t in leaf])
