"""Sizes beyond what one launch takes (fewer than 2^32 threads along a grid's
first dimension): the rows are dealt to several launches, the blocks of a
sequence to fewer workgroups, and the results are those of smaller calls."""

import pytest
import torch

import bit_nf4_quantized_12_amd as q
from tests import test_gpu_window_attn as wa
from tests.parity import report

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BASE = 4093  # rows that are repeated: a prime, so that no launch's share is a multiple of it


def _repeat(t, times):
    return t.expand(times, *t.shape).reshape(times * t.shape[0], *t.shape[1:])


def _repeats(got, base):
    """got is base again and again (looked at in pieces: it may be as large as a quarter of memory)."""
    n = base.shape[0]
    assert got.shape[0] % n == 0
    return all(torch.equal(p, _repeat(base, p.shape[0] // n)) for p in got.split(256 * n))


def test_layer_norm_rows():
    times, C = 4100, 520  # a workgroup of 256 threads per row: 2^24 rows are too many for one launch
    report(f"layer norm: M={times * BASE} C={C}")
    assert times * BASE > 1 << 24
    g = torch.Generator().manual_seed(1)
    x, w, b = (torch.randn(s, generator=g).bfloat16().to(DEV) for s in ((BASE, C), (C,), (C,)))
    want = q.qlora_layer_norm_fwd(x, w, b)
    got = q.qlora_layer_norm_fwd(_repeat(x, times), w, b)
    for a, t in zip(got, want):
        assert _repeats(a, t)


def test_distillation_rows():
    times, V, K = 16400, 16, 2  # loss: 64 threads per row, gradient: 256
    report(f"distill: M={times * BASE} V={V} K={K}")
    assert times * BASE > 1 << 26
    g = torch.Generator().manual_seed(2)
    z, val = torch.randn(BASE, V, generator=g).bfloat16().to(DEV), torch.randn(BASE, K, generator=g).to(DEV)
    idx = torch.randint(-1, V, (BASE, K), generator=g).int().to(DEV)
    t_lse, weight = torch.rand(BASE, generator=g).to(DEV) + 2, torch.rand(BASE, generator=g).to(DEV)
    small = (z, val, idx, t_lse, weight)
    big = [_repeat(t, times) for t in small]
    want = q.qlora_topk_distill_fwd_bwd(*small[:3], weight, 2.0, t_lse)
    got = q.qlora_topk_distill_fwd_bwd(*big[:3], big[4], 2.0, big[3])
    for a, t in zip(got, want):
        assert _repeats(a, t)
    loss, lse = q.qlora_topk_distill_fwd(*big[:3], 2.0, big[3])
    assert torch.equal(loss, got[0]) and torch.equal(lse, got[1])
    dz = q.qlora_topk_distill_bwd(*big[:3], lse, big[4], 2.0, big[3])
    assert _repeats(dz, q.qlora_topk_distill_bwd(*small[:3], want[1], weight, 2.0, t_lse))


def test_many_sequences_with_a_long_one():
    """65535 sequences, one of 16384 tokens: every kernel's grid of sequences x heads x longest is too large. The call with
    small longest lengths makes the same sums in a query's own order, so o, lse and dq have the same bits; dk and dv of the
    long sequence's first tokens come in another order: each float32 sum of n terms is off by at most n 2^-24 of the sum of
    their sizes, and rounded to bf16."""
    h, d, n, window, sinks = 8, 8, 16384, 64, 4
    lens = [1] * 65535
    lens[40000] = n
    report(f"window attention: {len(lens)} sequences, longest {n}, H={h} D={d}")
    qt, kt, vt, gt = wa._make([sum(lens)], [sum(lens)], h, h, d, 5)
    cu = wa._starts(lens)
    f = lambda most: q.qlora_window_attn_fwd(qt, kt, vt, cu, most, window, sinks)  # noqa: E731
    o, lse = f(n)
    assert all(torch.equal(a, b) for a, b in zip((o, lse), f(64)))
    b = lambda most: q.qlora_window_attn_bwd(qt, kt, vt, o, lse, gt, cu, most, window, sinks, max_k=most)  # noqa: E731
    got, want = b(n), b(64)
    assert torch.equal(got[0], want[0])
    first = torch.arange(40000, 40000 + sinks, device=DEV)
    rest = torch.ones(qt.shape[0], dtype=torch.bool, device=DEV)
    rest[first] = False
    # sizes of the terms of dv: probabilities (at most 1) times |do|, and of dk: |ds| <= 2 |do| |v| times scale |q|
    rows = slice(40000, 40000 + n)
    go, qo = gt[rows].float().abs(), qt[rows].float().abs()
    p = torch.exp(qt[rows].float().transpose(0, 1) @ kt[first].float().permute(1, 2, 0).contiguous() * d ** -0.5
                  - lse[:, rows, None])  # [h, n, sinks]
    size_v = p.transpose(1, 2).contiguous() @ go.transpose(0, 1).contiguous()
    reach = go.transpose(0, 1).sum(2) * vt[rows].float().abs().amax()
    size_k = (2 * p * reach[:, :, None] * d ** -0.5).transpose(1, 2).contiguous() @ qo.transpose(0, 1).contiguous()
    for a, c, size in zip(got[1:], want[1:], (size_k, size_v)):
        assert torch.equal(a[rest], c[rest])
        x, y = a[first].float(), c[first].float()
        assert torch.all((x - y).abs() <= wa.H * (x.abs() + y.abs()) + 2 * n * wa.U * size.transpose(0, 1))
