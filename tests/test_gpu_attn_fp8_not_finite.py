"""ssv_verify_attn_fp8 with queries that are not finite: such a (row, head) gives NaN, as the formula does, and every
other one what it gives beside finite rows."""
import numpy as np
import pytest
import torch

from diffusion_speculative_verification_gb300 import ssv, io as sio, workloads as W
from gpu_common import ensure_built
from paged_common import PagedBatch
from test_gpu_attn_fp8 import call, reference

pytestmark = pytest.mark.gpu
INF, NINF, NAN = 0x7F80, 0xFF80, 0x7FC0


def setup_module():
    ensure_built()


@pytest.mark.parametrize("bits", [INF, NINF, NAN])
@pytest.mark.parametrize("C,N", [([0, 0], [0, 3]), ([300, 64], [0, 3]), ([20011, 5], [1, 200])])
def test_queries_that_are_not_finite(C, N, bits):
    x = PagedBatch(C, N, [8, 4], 4, 2, 128, 64, seed=sum(C) + 1)
    o, tol = reference(x)
    q = x.q.copy()
    bad = [(0, 1), (9, 3), (x.rows - 1, 0), (x.rows - 5, 2)]
    for n, (row, head) in enumerate(bad):
        q[row, head, n * 41] = bits
    t = x.device()
    t["q"].copy_(sio.tensor(q, W.BF16, "cuda"))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = call(t, dev_status=status).double().cpu().numpy()
    assert ssv.get_status(status) == ssv.SSV_OK
    for row, head in bad:
        assert np.isnan(got[row, head]).all()
        o[row, head], tol[row, head], got[row, head] = 0, 0, 0
    assert (np.abs(got - o) <= tol).all()


def test_every_score_below_all_numbers():
    """Scores of minus infinity alone: a weight of 0 / 0."""
    x = PagedBatch([0], [4], [3], 2, 1, 128, 64, seed=3)
    x.k_new[:, 0, 5] = W.f32_to_bf16_bits(np.float32([1.0]))
    q = x.q.copy()
    q[2, 1, 5] = NINF
    t = x.device()
    t["q"].copy_(sio.tensor(q, W.BF16, "cuda"))
    got = call(t).double().cpu().numpy()
    assert np.isnan(got[2, 1]).all()
    got[2, 1] = 0
    assert np.isfinite(got).all()
