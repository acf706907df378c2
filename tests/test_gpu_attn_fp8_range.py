"""ssv_verify_attn_fp8 where the cached values are far smaller than the fresh
ones: zero pages (ssv_commit_fp8 gives them the scale 2^-100), and scales down
to the smallest that fp32 has.  The tolerance is that of test_gpu_attn_fp8.py: the
cached values' own rounding, at most 2^-25 of the unit, lies far below it beside
fresh values of 2^-52 and more."""
import numpy as np
import pytest

from diffusion_speculative_verification_gb300 import workloads as W
from gpu_common import ensure_built
from paged_common import PagedBatch
from test_gpu_attn_fp8 import check

pytestmark = pytest.mark.gpu


def setup_module():
    ensure_built()


def batch(C, N, B, seed, codes=None, v_scale=None, k_scale=None, v_new=None, **kw):
    """A PagedBatch with its cached codes and scales replaced where a page is in use."""
    x = PagedBatch(C, N, B, 4, 2, 128, 64, seed=seed, **kw)
    for i, s in ((0, k_scale), (1, v_scale)):
        if s is not None:
            x.scale[i] = np.where(np.isnan(x.scale[i]), x.scale[i], np.float32(s))
    if codes is not None:
        x.codes[1] = np.where(x.codes[1] == 0x7F, x.codes[1], np.uint8(codes))
    if v_new is not None:
        x.v_new = W.f32_to_bf16_bits(np.asarray(v_new(W.bf16_bits_to_f32(x.v_new)), np.float32))
    return x


@pytest.mark.parametrize("v", [1.0, 32.0, 300.0])
def test_zero_pages_and_a_long_prompt(v):
    """Flat scores over 2048 fresh keys of one sign: the sum of weights times values is large."""
    check(batch([260], [2048], [4], 1, codes=0, v_scale=2.0 ** -100, v_new=lambda y: np.abs(y) * v, qstd=2.0 ** -20))


def test_zero_pages_of_keys_and_values():
    x = batch([300, 64, 0], [40, 300, 3], [8, 2, 5], 2, codes=0, v_scale=2.0 ** -100, k_scale=2.0 ** -100)
    x.codes[0] = np.where(x.codes[0] == 0x7F, x.codes[0], np.uint8(0))
    check(x)


@pytest.mark.parametrize("e", [-148, -120, -105, -70])
def test_scales_below_every_fresh_value(e):
    check(batch([500, 130], [300, 1], [8, 4], 3, v_scale=2.0 ** e, v_new=lambda y: 8 * np.abs(y), qstd=2.0 ** -10))


def test_running_maximum_lags_at_the_fresh_keys():
    """256 fresh keys whose scores lie just under 8 (in powers of two) above the cached ones: the reference stays."""
    x = batch([128], [256], [4], 4, codes=0, v_scale=2.0 ** -100, v_new=lambda y: 4 + 0 * y)
    q, k = W.bf16_bits_to_f32(x.q), W.bf16_bits_to_f32(x.k_new)
    q[:], k[:] = 0, 0
    q[:, :, 0], k[:, :, 0] = 1, 7.75 * np.log(2) * np.sqrt(128)
    x.q, x.k_new = W.f32_to_bf16_bits(q), W.f32_to_bf16_bits(k)
    x.codes[0] = np.where(x.codes[0] == 0x7F, x.codes[0], np.uint8(0))
    check(x)


def test_zero_pages_beside_others():
    """Zero pages first, in the middle and last; a unit cut over CTAs meets only zero pages in some of its parts."""
    x = batch([6400, 700], [40, 0], [8, 4], 5)
    for b, pages in ((0, list(range(0, 30)) + list(range(60, 64)) + [99]), (1, [0, 5])):
        for j in pages:
            p = x.table[b, j]
            x.scale[1][p] = 2.0 ** -100
            x.codes[1][p] = np.where(x.codes[1][p] == 0x7F, x.codes[1][p], np.uint8(0))
    check(x)


@pytest.mark.parametrize("e", [-30, -50])
def test_small_values_everywhere(e):
    """Cached and fresh values of one small size keep their relative precision."""
    x = batch([500, 130], [30, 1], [8, 4], 6, v_new=lambda y: y * 2.0 ** e)
    x.scale[1] = x.scale[1] * np.float32(2.0 ** e)
    check(x)


def test_large_scales():
    x = batch([500, 130], [30, 1], [8, 4], 7, v_new=lambda y: y * 2.0 ** 90)
    x.scale[1] = x.scale[1] * np.float32(2.0 ** 90)
    check(x)
