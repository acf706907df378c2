"""ssv_distill where its rules for what is not a number and for rows of nothing meet."""
import numpy as np
import pytest
import torch

from diffusion_speculative_verification_gb300 import ssv, workloads as W
from gpu_common import ensure_built
from logits_common import store

pytestmark = pytest.mark.gpu


def setup_module():
    ensure_built()


@pytest.mark.parametrize("dtype", [W.F32, W.BF16])
@pytest.mark.parametrize("mode", [ssv.RENORM, ssv.REST])
def test_nothing_and_no_number(mode, dtype):
    """Rows of nothing but -inf: the loss is NaN where the target has a NaN, infinite where it has a probability, 0 where it
    has none; the gradient is 0."""
    for v in (7, 3001):
        x = store(np.full((4, v), -np.inf), dtype)[1]
        token = torch.tensor([[0, 1], [2, 3], [4, -1], [-1, -1]], dtype=torch.int32, device="cuda")
        value = torch.tensor([[-1.0, float("nan")], [-1.0, -1.0], [-1.0, float("nan")], [float("nan"), 0.0]], device="cuda")
        loss, stats, grad = ssv.distill(x, token, value, 1.5, mode, grad=True)
        alone, _, _ = ssv.distill(x, token, value, 1.5, mode)
        back = ssv.distill_backward(x, token, value, stats, None, 1.5, mode)
        for y in (loss, alone):
            assert y[0].isnan() and y[1] == np.inf and y[2] == np.inf    # what an absent token comes with is not read
            assert y[3] == (np.inf if mode == ssv.REST else 0.0)         # all of the target's probability is the others'
        assert (grad == 0).all() and (back == 0).all()
