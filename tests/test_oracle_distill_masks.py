"""Pin of the distillation oracle under masks: a mask of a number is the mask of -inf where it leaves the others nothing."""
import numpy as np
import pytest

import oracle.distill as odist


@pytest.mark.parametrize("mask", [-1e3, -1e9, -3.4e38])
def test_finite_masks_are_masks(mask):
    r = np.random.default_rng(0)
    z = np.full(50, mask)
    z[:4] = r.standard_normal(4)
    token = np.array([0, 1, 2, 3, 7, -1])
    p = np.append(r.dirichlet(np.ones(4)) * (1 - 3e-7), [0.0, 0.0])
    with np.errstate(divide="ignore"):
        value = np.log(p)
    hidden = np.where(z < -900, -np.inf, z)
    for T in (0.5, 2.0):
        loss, grad, _ = odist.row_distill(z, token, value, T, odist.REST)
        want, wg, _ = odist.row_distill(hidden, token, value, T, odist.REST)
        assert loss == want and np.abs(grad - wg).max() < 1e-200
        # a rest that is more than a rounding costs what the mask says
        value[0] -= 0.5
        assert odist.row_distill(z, token, value, T, odist.REST)[0] > 0.1 * abs(mask) / T * (1 - np.exp(value).sum())
        value[0] += 0.5
