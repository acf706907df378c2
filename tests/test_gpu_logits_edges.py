"""The operators on logits where their rules for what is not a number, for rows of nothing and for numbers beyond fp32 meet."""
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


@pytest.mark.parametrize("dtype", [W.F32, W.BF16])
def test_differences_beyond_fp32(dtype):
    """Logits further apart than fp32's largest number: the lower one is as if it were -inf, at any temperature."""
    for v in (9, 3001):
        x = np.zeros((2, v))
        x[:, 1], x[:, 5] = 3e38, -3e38
        ref, t = store(x, dtype)
        hidden = t.clone()
        hidden[:, 5] = float("-inf")
        T = 1e37
        token = torch.tensor([5, 1], dtype=torch.int32, device="cuda")
        lp, rank, ent, lse, tl, tt = ssv.logprobs(t, token, v if v < 128 else 4, T)
        want = ssv.logprobs(hidden, token, 4, T)
        assert lp[0] == -np.inf and torch.equal(lp, want[0]) and torch.equal(lse, want[3]) and torch.equal(ent, want[2])
        assert rank.tolist() == [v, 1] and torch.equal(tl[:, :4], want[4]) and torch.equal(tt[:, :4], want[5])
        if v < 128:
            assert (tt[:, v - 1] == 5).all() and (tl[:, v - 1] == -np.inf).all()     # listed all the same: it is not -inf
        listed = torch.tensor([[1, 5], [1, 0]], dtype=torch.int32, device="cuda")
        value = torch.full((2, 2), -1.0, device="cuda")
        for mode in (ssv.RENORM, ssv.REST):
            got = ssv.distill(t, listed, value, T, mode, grad=True)
            want = ssv.distill(hidden, listed, value, T, mode, grad=True)
            assert got[0][0] == np.inf and torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])
            assert got[2].isfinite().all()
            assert torch.equal(ssv.distill_backward(t, listed, value, got[1], None, T, mode), got[2])
