"""Layer norm of rows whose values lie close together around a large mean: the
centred values are exact differences from the mean, not from its rounding.

Bounds (u = 2^-24, sums at most 48 additions deep within a row): a first mean is
off by t <= 50 u mean|x|, and the mean of what is left of the row's values less
that first one, d, corrects it up to 50 u mean|d|, so for float32
  |y - ref| <= 64 u (|w| rstd (|d| + mean|d|) + |xh w| + |b|),  |d| <= |x - mean| + t
  |mean - ref| <= u |mean| + 64 u mean|d|
  |rstd - ref| <= (4 u + 64 u rstd^2 mean d^2) rstd
since a variance is mean d^2 less the square of a mean of d that is no larger."""

import numpy as np
import pytest
import torch

import bit_nf4_quantized_12_amd as q
from oracle import layer as ol
from tests.parity import report

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
EPS = 1e-5


def _np(t):
    return t.detach().cpu().double().numpy()


def _check(x, w, b):
    y, mean, rstd = (_np(t) for t in q.qlora_layer_norm_fwd(x.to(DEV), w.to(DEV), b.to(DEV), EPS))
    X, W, B = _np(x), _np(w), _np(b)
    yr, mr, rr = ol.layer_norm_fwd(X, W, B, EPS)
    d = np.abs(X - mr[:, None]) + 50 * U * np.abs(X).mean(axis=1)[:, None]
    rs, dm = rr[:, None], d.mean(axis=1)
    bounds = (64 * U * (np.abs(W) * rs * (d + dm[:, None]) + np.abs(yr - B) + np.abs(B)), U * np.abs(mr) + 64 * U * dm,
              (4 * U + 64 * U * rr * rr * (d * d).mean(axis=1)) * rr)
    for name, got, ref, bound in zip(("y", "mean", "rstd"), (y, mean, rstd), (yr, mr, rr), bounds):
        worst = np.max(np.abs(got - ref) / (bound + 1e-37))
        assert worst <= 1.0, f"{name}: an error is {worst:.3f} of its bound"


@pytest.mark.parametrize("C", [1, 7, 100, 520, 1000, 2049, 4097, 5000, 16383])
@pytest.mark.parametrize("value", [1000.1, -77.7, 3e-3])
def test_constant_rows(C, value):
    report(f"layer norm: constant rows of {value}, C={C}")
    g = torch.Generator().manual_seed(C)
    _check(torch.full((3, C), value), 1 + torch.rand(C, generator=g), torch.randn(C, generator=g))


@pytest.mark.parametrize("C", [1000, 4097, 8192])
@pytest.mark.parametrize("spread", [0.01, 1.0])
def test_rows_close_to_a_large_mean(C, spread):
    report(f"layer norm: rows around 1000, spread {spread}, C={C}")
    g = torch.Generator().manual_seed(C)
    _check(1000 + spread * torch.randn(5, C, generator=g), 1 + torch.rand(C, generator=g), torch.randn(C, generator=g))


@pytest.mark.parametrize("C", [512, 4096, 8192])
def test_mean_of_bf16_rows_around_zero(C):
    """bf16 values of exponents -3 to 2 are multiples of 2^-10; float32 sums of both signs stay multiples of that below 2^14,
    so they are exact, and with a power of two for C the mean as well."""
    report(f"layer norm: mean of bf16 rows around zero, C={C}")
    g = torch.Generator().manual_seed(C)
    size = (1 + torch.rand(64, C, generator=g)) * 2.0 ** torch.randint(-3, 3, (64, C), generator=g)
    x = torch.where(torch.rand(64, C, generator=g) < 0.5, size, -size).bfloat16()
    x = torch.where(x.abs() >= 7.9, 1.0, x.float()).bfloat16()  # (nothing rounded up to 8)
    _, mean, _ = q.qlora_layer_norm_fwd(x.to(DEV), torch.ones(C, device=DEV), None, EPS)
    assert np.array_equal(_np(mean), _np(x).mean(axis=1))
