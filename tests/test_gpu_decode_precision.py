"""Single-token attention keeps 16 bits of its probabilities beside the values.

With u = 2^-24, a score off by es = D u scale sum |q_d k_d| + 4 u |s|, n visible
keys and an output rounded to bf16 once (h = 2^-8), as in
tests/test_gpu_window_attn.py, but 2^-16 in place of h for the probabilities:
  |o - ref| <= (2^-16 + 2 es + 16 u + n u) sum p |v| + h |o|"""

import numpy as np
import pytest
import torch

import bit_nf4_quantized_12_amd as q
from oracle import layer as ol
from tests import test_gpu_window_attn as wa
from tests.parity import report

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("lens,cap,h,hkv", [([40, 33, 1, 300], 300, 8, 2), ([3000], 3000, 4, 1)])
@pytest.mark.parametrize("d", [8, 64, 80, 128])
def test_probabilities(lens, cap, h, hkv, d):
    report(f"decode, probabilities: lens={lens} H={h}/{hkv} D={d}")
    g = torch.Generator().manual_seed(d)
    b = len(lens)
    kc, vc, qt = wa._rand(g, b, cap, hkv, d), wa._rand(g, b, cap, hkv, d), wa._rand(g, b, h, d)
    o = q.qlora_window_attn_decode(qt, kc, vc, torch.tensor(lens, dtype=torch.int32, device=DEV), 1 << 30)
    scale = d ** -0.5
    Q = wa._np(qt)
    for i, n in enumerate(lens):
        for j in range(h):
            kk, vv = wa._np(kc[i, :n, j // (h // hkv)]), wa._np(vc[i, :n, j // (h // hkv)])
            r, _, p = ol.attention(Q[i, j][None], kk, vv, 1 << 30, 0, scale)
            es = d * wa.U * scale * (np.abs(Q[i, j]) @ np.abs(kk).T).max() + 4 * wa.U * scale * np.abs(Q[i, j] @ kk.T).max()
            wa._within(o[i, j], r[0], (2.0 ** -16 + 2 * es + 16 * wa.U + n * wa.U) * (p[0] @ np.abs(vv))
                       + 1.01 * wa.H * np.abs(r[0]), "o")
