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


def test_norm_of_rows_as_other_operations_leave_them():
    g = torch.Generator().manual_seed(2)
    w, b = _randn(g, 65), _randn(g, 65)
    big, grad = _randn(g, 9, 65), _randn(g, 18, 65)

    def check(make, n):
        """make(leaf) -> rows [n, 65]; its norm is joined to others, so that the gradient is a slice of a larger one."""
        a, c = big.clone().requires_grad_(), big.clone().requires_grad_()
        y = q.LayerNormFunction.apply(make(a), w, b, 1e-5)
        torch.cat((big[:1], y)).backward(grad[:n + 1])
        yc = q.LayerNormFunction.apply(make(c).clone(memory_format=torch.contiguous_format), w, b, 1e-5)
        yc.backward(grad[1:n + 1].clone())
        assert y.shape == (n, 65) and torch.equal(y, yc) and torch.equal(a.grad, c.grad)

    check(lambda t: t[1:], 8)                      # rows that start off 16 bytes
    check(lambda t: t[3:4].expand(6, 65), 6)       # one row many times
    check(lambda t: t[:, :13].t().contiguous().t().expand(9, 13).repeat(1, 5), 9)
    check(lambda t: torch.cat((t, t)).t().contiguous().t()[:5], 5)  # columns contiguous


def test_attention_of_heads_as_other_operations_leave_them():
    T = 40
    qt, kt, vt, gt = wa._make([T], [T], 2, 2, 64, 3)
    cu = wa._starts([T])
    wide = _randn(torch.Generator().manual_seed(4), T, 2, 68)
    forms = [lambda t: t.permute(0, 2, 1).contiguous().permute(0, 2, 1),   # columns apart
             lambda t: torch.cat((wide[:, :, :4], t), 2)[:, :, 4:],         # rows that start off 16 bytes
             lambda t: torch.cat((wide[:, :, :4], t), 2)[:, :, 4:].contiguous()[:1].expand(T, 2, 64)]  # one token many times
    for f in forms:
        a = [t.clone().requires_grad_() for t in (qt, kt, vt)]
        c = [t.clone().requires_grad_() for t in (qt, kt, vt)]
        o = _attn(*(f(t) for t in a), cu, T)
        ref = _attn(*(f(t).clone(memory_format=torch.contiguous_format) for t in c), cu, T)
        o.backward(f(gt))
        ref.backward(f(gt).clone(memory_format=torch.contiguous_format))
        assert torch.equal(o, ref)
        for s, t in zip(a, c):
            assert torch.equal(s.grad, t.grad)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_distillation_of_rows_as_other_operations_leave_them(dt):
    z, val, idx, t_lse, weight = td._make(9, 101, 5, dt, 2.0, True, 7)
    # the next token's entries for each token: rows from the second on
    forms = [(lambda t: t[1:], slice(1, None)), (lambda t: t[2:3].expand(8, 101), slice(1, None)),
             (lambda t: t.t().contiguous().t()[1:], slice(0, 8))]
    for f, rows in forms:
        a, c = z.clone().requires_grad_(), z.clone().requires_grad_()
        loss = q.TopkDistillFunction.apply(f(a), val[rows], idx[rows], 2.0, t_lse[rows])
        loss.backward(weight[rows])
        ref = q.TopkDistillFunction.apply(f(c).clone(memory_format=torch.contiguous_format), val[rows].clone(),
                                          idx[rows].clone(), 2.0, t_lse[rows].clone())
        ref.backward(weight[rows].clone())
        assert torch.equal(loss, ref) and torch.equal(a.grad, c.grad)
