"""Distillation with values that are no numbers: what a row's formula makes of
them stays in that row, and is not taken for a row without entries."""

import pytest
import torch

import bit_nf4_quantized_12_amd as q
from tests import test_gpu_distill as td
from tests.parity import report

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
NAN, INF = float("nan"), float("inf")


def _both(z, val, idx, weight, t_lse):
    """(loss, gradient) from the pass over the logits that makes both, and from loss and gradient apart."""
    loss, lse, dz = q.qlora_topk_distill_fwd_bwd(z, val, idx, weight, 2.0, t_lse)
    apart, lse2 = q.qlora_topk_distill_fwd(z, val, idx, 2.0, t_lse)
    return (loss, dz), (apart, q.qlora_topk_distill_bwd(z, val, idx, lse2, weight, 2.0, t_lse))


# a row in registers of few and of many threads, and one past the registers
@pytest.mark.parametrize("dt,V", [("f32", 300), ("bf16", 32000), ("bf16", 140001)])
@pytest.mark.parametrize("mass", [False, True])
@pytest.mark.parametrize("K", [1, 9])
def test_teacher_values_that_are_nan(K, mass, dt, V):
    report(f"distill, NaN values: V={V} K={K} {dt} mass={mass}")
    z, val, idx, t_lse, weight = td._make(7, V, K, dt, 2.0, mass, 3, ragged=False)
    weight[3], weight[4] = 1, 0
    good = _both(z, val, idx, weight, t_lse)
    val[1] = NAN            # all of a row's
    val[2, K // 2] = NAN    # one of them
    val[4] = NAN            # without weight
    val[5], idx[5] = NAN, -1  # no entries
    for (loss, dz), (loss0, dz0) in zip(_both(z, val, idx, weight, t_lse), good):
        assert loss[[1, 2, 4]].isnan().all() and dz[[1, 2]].isnan().all()
        assert torch.all(dz[[4, 5]] == 0) and loss[5] == 0
        for i in (0, 3, 6):
            assert torch.equal(loss[i], loss0[i]) and torch.equal(dz[i], dz0[i])


@pytest.mark.parametrize("dt,V", [("f32", 300), ("bf16", 32000), ("bf16", 140001)])
def test_entries_of_probability_zero_and_logits_that_are_no_numbers(dt, V):
    report(f"distill, probabilities of zero: V={V} {dt}")
    z, val, idx, t_lse, weight = td._make(6, V, 5, dt, 2.0, True, 3, ragged=False)
    weight[:] = 1
    t_lse[1:4] = 1e30  # exp(val / tau - t_lse) = 0
    z[1, 7], z[2, 8], z[3, 9] = NAN, INF, -INF
    for loss, dz in _both(z, val, idx, weight, t_lse):
        assert torch.all(loss[1:4] == 0) and torch.all(dz[1:4] == 0)
        assert torch.all(loss[[0, 4, 5]] != 0) and torch.isfinite(dz).all()
