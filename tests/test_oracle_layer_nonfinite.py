"""The oracle's distillation: entries of minus infinity are left out, entries
that are NaN are not."""

import numpy as np

from oracle import layer as ol


def test_teacher_values_that_are_no_numbers():
    rng = np.random.default_rng(0)
    z, val = rng.standard_normal((4, 6)), rng.standard_normal((4, 3))
    idx = np.array([[0, 1, 2], [3, 4, 5], [0, 2, 4], [1, 3, 5]])
    val[0], val[1, 1], val[2] = np.nan, np.nan, -np.inf
    loss, lse, dz = ol.topk_distill(z, val, idx, 2.0)
    assert np.isnan(loss[:2]).all() and np.isnan(dz[:2]).all() and np.isfinite(lse).all()
    assert loss[2] == 0 and np.all(dz[2] == 0) and loss[3] > 0 and np.isfinite(dz[3]).all()
