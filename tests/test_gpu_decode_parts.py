"""Single-token attention over caches that are cut into many parts: parity with
the float64 oracle for every width of the join (heads below 128 columns leave
lanes of it idle) and for odd and even counts of parts up to 64, filled and
empty.

The bound is that of tests/test_gpu_window_attn.py. The values have a mean of 1,
so a part that is left out moves the result by its share of the probabilities,
several times the bound."""

import numpy as np
import pytest
import torch

import bit_nf4_quantized_12_amd as q
from oracle import layer as ol
from tests import test_gpu_window_attn as wa
from tests.parity import report

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
PART = 512  # keys of a part, at least


def _check(lens, cap, h, hkv, d, seed=0):
    report(f"decode in parts: lens={lens} cap={cap} H={h}/{hkv} D={d}")
    g = torch.Generator().manual_seed(seed)
    b = len(lens)
    qt, kc = wa._rand(g, b, h, d), wa._rand(g, b, cap, hkv, d)
    vc = (1 + torch.randn(b, cap, hkv, d, generator=g)).bfloat16().to(DEV)
    for i, n in enumerate(lens):
        kc[i, n:], vc[i, n:] = float("nan"), float("inf")
    o = q.qlora_window_attn_decode(qt, kc, vc, torch.tensor(lens, dtype=torch.int32, device=DEV), 1 << 30, 4)
    scale = d ** -0.5
    Q = wa._np(qt)
    for i, n in enumerate(lens):
        for j in range(h):
            kk, vv = wa._np(kc[i, :n, j // (h // hkv)]), wa._np(vc[i, :n, j // (h // hkv)])
            r, _, p = ol.attention(Q[i, j][None], kk, vv, 1 << 30, 4, scale)
            es = d * wa.U * scale * (np.abs(Q[i, j]) @ np.abs(kk).T).max() + 4 * wa.U * scale * np.abs(Q[i, j] @ kk.T).max()
            bound = (wa.H + 2 * es + 16 * wa.U + n * wa.U) * (p[0] @ np.abs(vv)) + 1.01 * wa.H * np.abs(r[0])
            wa._within(o[i, j], r[0], bound, "o")


@pytest.mark.parametrize("parts", [3, 17, 18, 32, 33, 35, 63, 64])
@pytest.mark.parametrize("d", [8, 32, 64, 72, 80, 96, 128])
def test_filled_parts(d, parts):
    _check([parts * PART], parts * PART, 2, 1, d, seed=parts)


@pytest.mark.parametrize("d", [64, 128])
def test_parts_that_a_short_request_leaves_empty(d):
    _check([40000, 39999, 39, 8704], 40000, 2, 1, d)
    _check([16384, 700], 16384, 16, 2, d)


def test_a_cache_of_nearly_2_31_positions():
    """The last of 64 parts ends past 2^31 - 128. Keys that are all one row (token pitch 0) give every position the same
    probability, 1 / cap; all sums are whole numbers below 2^24 or counts of 32 keys, so only the quotient rounds."""
    cap, ones = (1 << 31) - 4097, 1 << 24
    report(f"decode: cap={cap} D=8")
    vc = torch.zeros(1, cap, 1, 8, dtype=torch.bfloat16, device=DEV)
    vc[:, cap - ones:] = 1
    kc = torch.ones(1, 1, 1, 8, dtype=torch.bfloat16, device=DEV).expand(1, cap, 1, 8)
    lens = torch.tensor([cap], dtype=torch.int32, device=DEV)
    o = q.qlora_window_attn_decode(torch.ones(1, 1, 8, dtype=torch.bfloat16, device=DEV), kc, vc, lens, 1 << 40, 0)
    ref = np.full(8, ones / cap)
    wa._within(o[0, 0], ref, (wa.H + 16 * wa.U) * ref, "o")
