"""Sizes beyond what one launch takes (fewer than 2^32 threads along a grid's
first dimension): the rows are dealt to several launches, and the results
are those of smaller calls."""

import pytest
import torch

import bit_nf4_quantized_12_amd as q
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
