"""ssv_verify_attn_fp8 under bounds far above what a batch holds, as a loop states them once for all its passes, and with
one long prompt among many decoding requests."""
import numpy as np
import pytest
import torch

from diffusion_speculative_verification_gb300 import ssv, io as sio
from gpu_common import ensure_built
from paged_common import PagedBatch
from test_gpu_attn_fp8 import call, check, reference

pytestmark = pytest.mark.gpu
WIDE = dict(max_cache=131072, max_new=32768, max_block=64)


def setup_module():
    ensure_built()


def many(n, seed, idle=(), prompt=0):
    r = np.random.default_rng(seed)
    N = r.integers(0, 2, n)
    N[n // 2] = prompt
    return PagedBatch(r.integers(0, 120, n), N, r.integers(1, 9, n), 4, 1, 128, 16, seed=seed + 1, idle=idle)


def wide(x):
    t = x.device()
    for k, v in WIDE.items():
        setattr(t["batch"], k, v)
    return t


@pytest.mark.parametrize("n", [40, 700])
def test_bounds_far_above_the_batch(n):
    x = many(n, n, idle=(0, 3, n - 1), prompt=300)
    check(x, t=wide(x))


def test_rows_shared_with_an_earlier_sequence():
    """Within these bounds the plan holds for sequences that share no rows: one that does is refused, with its rows left
    to the earlier one; in a warp's 32 and from one such group to the next."""
    x = many(600, 3)
    o, tol = reference(x)
    seqs = x.seqs.copy()
    bad = [7, 32, 64, 599]
    for b in bad:
        seqs[b, 3] = seqs[b - 1, 3]
    t = wide(x)
    t["batch"].dev.copy_(sio.int_tensor(seqs, "cuda"))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = call(t, dev_status=status).double().cpu().numpy()
    assert ssv.get_status(status) == ssv.SSV_ERR_INVALID
    keep = np.ones(x.rows, bool)
    for b in bad:
        keep[x.seqs[b, 3]: x.seqs[b, 3] + x.seqs[b, 1] + 2 * x.seqs[b, 2]] = False
    assert (np.abs(got[keep] - o[keep]) <= tol[keep]).all()
