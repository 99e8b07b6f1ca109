"""Layer norm's backward with dx in dy's place, in each layout of a row over
threads, with fewer and more rows than workgroups: the bits of separate tensors."""

import pytest
import torch

import bit_nf4_quantized_12_amd as q
from tests import test_gpu_layer_norm as tn
from tests.parity import report

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("M,C", [(3000, 256), (5, 512), (1300, 520), (2100, 2048), (1100, 4096), (600, 8192), (530, 16384),
                                 (3000, 77), (1300, 1001), (1100, 3001), (530, 5003), (270, 16383)])
def test_gradient_in_place(M, C, dt):
    report(f"layer norm backward in place: M={M} C={C} {dt}")
    x, w, b, dy = tn._inputs(M, C, dt, dt, M + C)
    _, mean, rstd = q.qlora_layer_norm_fwd(x, w, b)
    want = q.qlora_layer_norm_bwd(x, w, dy, mean, rstd)
    g = dy.clone()
    got = q.qlora_layer_norm_bwd(x, w, g, mean, rstd, dx=g)
    assert got[0] is g
    for s, t in zip(got, want):
        assert torch.equal(s, t)
