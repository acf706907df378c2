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
