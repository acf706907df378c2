"""What the paged-cache operators promise beyond single calls, as far as the
host shows it (no GPU)."""
import ctypes as C

import pytest
import torch

from diffusion_speculative_verification_gb300 import build, ssv
from test_abi_paged import _attn


@pytest.fixture(scope="module")
def L():
    build.build()
    return ssv.lib()


def test_attn_workspace_counters_have_one_place(L):
    """The counters' extent and place hang on no argument: a longer prompt over the same rows asks for nothing more, and
    sixteen more sequences ask for their plan tables alone (four ints each for every CTA, 152 without a device)."""
    def need(**kw):
        n = C.c_size_t(0)
        assert L.ssv_verify_attn_fp8_workspace(C.byref(_attn(total_rows=4000, max_block=32, **kw)), C.byref(n)) == ssv.SSV_OK
        return n.value

    assert need(max_new=2048) == need(max_new=100)
    if not torch.cuda.is_available():
        assert need(batch=47) - need(batch=31) == 152 * 16 * 16


def test_commit_refuses_lengths_of_another_batch():
    seqs = torch.zeros((2, 6), dtype=torch.int32)
    batch = ssv.Batch.from_device(seqs, 8, 4, 10, 0, 2)
    tau, acc = torch.zeros(4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    cache, scale = torch.zeros((3, 2, 16, 128), dtype=torch.uint8), torch.zeros((3, 2))
    pages, rows = torch.zeros(6, dtype=torch.int32), torch.zeros((8, 2, 128), dtype=torch.bfloat16)
    for bad in (acc[:1], acc.long(), torch.zeros(4, dtype=torch.int32)[::2]):
        with pytest.raises(ssv.SsvError, match="shapes|contiguous int32"):
            ssv.commit_fp8(rows, rows, cache, cache, scale, scale, pages, batch, tau, acc, cache_len=bad)
