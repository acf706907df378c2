"""Host-side refusals of the paged-cache operators (no GPU): bad arguments
return synchronously, nothing is launched; empty batches are no-ops."""
import ctypes as C

import numpy as np
import pytest
import torch

from diffusion_speculative_verification_gb300 import build, ssv


@pytest.fixture(scope="module")
def L():
    build.build()
    return ssv.lib()


M = 1 << 20  # made-up addresses a megabyte apart


def _plan(**kw):
    base = dict(cache_len=M, new_len=2 * M, block=3 * M, held=4 * M, pages=5 * M, free_list=6 * M, n_free=7 * M,
                batch=4, max_pages=8, page_size=64, n_pages=32, total_rows=100, seqs=8 * M, slot_map=9 * M,
                slot_off=10 * M, held_out=11 * M, n_free_out=12 * M, dev_status=None)
    base.update(kw)
    return ssv.PagePlanArgs(**base)


def test_plan_validation(L):
    cases = [(dict(batch=-1), ssv.SSV_ERR_INVALID), (dict(page_size=48), ssv.SSV_ERR_INVALID),
             (dict(page_size=256), ssv.SSV_ERR_INVALID), (dict(n_pages=1 << 26), ssv.SSV_ERR_INVALID),
             (dict(batch=4097), ssv.SSV_ERR_UNSUPPORTED), (dict(cache_len=None), ssv.SSV_ERR_INVALID),
             (dict(pages=None), ssv.SSV_ERR_INVALID), (dict(slot_map=None), ssv.SSV_ERR_INVALID),
             (dict(held_out=4 * M), ssv.SSV_ERR_INVALID),                 # over its input
             (dict(n_free_out=7 * M), ssv.SSV_ERR_INVALID), (dict(seqs=9 * M + 16), ssv.SSV_ERR_INVALID),
             (dict(batch=1 << 10, max_pages=1 << 22), ssv.SSV_ERR_INVALID), (dict(total_rows=-1), ssv.SSV_ERR_INVALID)]
    for kw, code in cases:
        assert L.ssv_page_plan(C.byref(_plan(**kw)), None) == code, kw
    assert L.ssv_page_plan(None, None) == ssv.SSV_ERR_INVALID
    assert L.ssv_page_plan(C.byref(_plan(batch=0)), None) == ssv.SSV_OK


def _norm(**kw):
    base = dict(q_in=M, k_in=2 * M, q_out=3 * M, k_out=4 * M, q_weight=5 * M, k_weight=6 * M, q_in_stride=0,
                k_in_stride=0, q_out_stride=0, k_out_stride=0, dtype=ssv.SSV_BF16, Hq=4, Hkv=2, d=128, eps=1e-6,
                base=10000.0, seqs=7 * M, batch=1, total_rows=10, positions=None, dev_status=None)
    base.update(kw)
    return ssv.NormRopeArgs(**base)


def test_norm_validation(L):
    cases = [(dict(d=96), ssv.SSV_ERR_UNSUPPORTED), (dict(q_weight=None), ssv.SSV_ERR_INVALID),
             (dict(eps=-1.0), ssv.SSV_ERR_INVALID), (dict(eps=float("nan")), ssv.SSV_ERR_INVALID),
             (dict(base=1.0), ssv.SSV_ERR_INVALID), (dict(q_out=3 * M + 8), ssv.SSV_ERR_INVALID),
             (dict(k_weight=6 * M + 2), ssv.SSV_ERR_INVALID), (dict(q_in_stride=511), ssv.SSV_ERR_INVALID),
             (dict(q_in_stride=516), ssv.SSV_ERR_INVALID), (dict(k_out_stride=-256), ssv.SSV_ERR_INVALID),
             (dict(dtype=3), ssv.SSV_ERR_INVALID), (dict(Hkv=0), ssv.SSV_ERR_INVALID), (dict(batch=-1), ssv.SSV_ERR_INVALID)]
    for kw, code in cases:
        assert L.ssv_norm_rope_copy(C.byref(_norm(**kw)), None) == code, kw
    assert L.ssv_norm_rope_copy(None, None) == ssv.SSV_ERR_INVALID
    assert L.ssv_norm_rope_copy(C.byref(_norm(total_rows=0)), None) == ssv.SSV_OK


def _attn(**kw):
    base = dict(q=M, k_cache=2 * M, v_cache=3 * M, k_scale=4 * M, v_scale=5 * M, pages=6 * M, k_new=7 * M,
                v_new=8 * M, o=9 * M, k_stride=0, v_stride=0, Hq=32, Hkv=8, d=128, page_size=64, n_pages=10,
                table_len=10, scale=0.0, seqs=10 * M, batch=2, tau=11 * M, total_rows=40, total_slots=20,
                max_cache=50, max_new=0, max_block=10, dev_status=None)
    base.update(kw)
    return ssv.AttnFp8Args(**base)


def test_attn_validation(L):
    n = C.c_size_t(0)
    cases = [(dict(d=64), ssv.SSV_ERR_UNSUPPORTED), (dict(Hq=30), ssv.SSV_ERR_INVALID),
             (dict(Hq=129, Hkv=1), ssv.SSV_ERR_UNSUPPORTED), (dict(page_size=8), ssv.SSV_ERR_INVALID),
             (dict(max_block=65), ssv.SSV_ERR_INVALID), (dict(max_cache=-1), ssv.SSV_ERR_INVALID),
             (dict(scale=float("inf")), ssv.SSV_ERR_INVALID), (dict(v_stride=1000), ssv.SSV_ERR_INVALID),
             (dict(v_stride=1028), ssv.SSV_ERR_INVALID), (dict(k_scale=None), ssv.SSV_ERR_INVALID),
             (dict(o=9 * M + 8), ssv.SSV_ERR_INVALID), (dict(n_pages=1 << 22), ssv.SSV_ERR_INVALID),
             (dict(pages=None), ssv.SSV_ERR_INVALID), (dict(tau=None), ssv.SSV_ERR_INVALID)]
    for kw, code in cases:
        assert L.ssv_verify_attn_fp8(C.byref(_attn(**kw)), None, 0, None) == code, kw
        assert L.ssv_verify_attn_fp8_workspace(C.byref(_attn(**kw)), C.byref(n)) == code, kw
    assert L.ssv_verify_attn_fp8_workspace(C.byref(_attn()), C.byref(n)) == ssv.SSV_OK and n.value > 0
    assert L.ssv_verify_attn_fp8_workspace(C.byref(_attn()), None) == ssv.SSV_ERR_INVALID
    assert L.ssv_verify_attn_fp8(C.byref(_attn()), None, 0, None) == ssv.SSV_ERR_WORKSPACE
    assert L.ssv_verify_attn_fp8(C.byref(_attn()), 24, 1 << 30, None) == ssv.SSV_ERR_WORKSPACE   # misaligned
    assert L.ssv_verify_attn_fp8(C.byref(_attn(batch=0)), None, 0, None) == ssv.SSV_OK


def _commit(**kw):
    base = dict(k_new=M, v_new=2 * M, k_cache=3 * M, v_cache=4 * M, k_scale=5 * M, v_scale=6 * M, pages=7 * M,
                k_stride=0, v_stride=0, dtype=ssv.SSV_BF16, Hkv=2, d=128, page_size=16, n_pages=10, table_len=10,
                seqs=8 * M, batch=2, tau=9 * M, n_acc=10 * M, new_len=11 * M, total_rows=20, total_slots=10,
                max_new=0, max_block=5, dev_status=None)
    base.update(kw)
    return ssv.CommitFp8Args(**base)


def test_commit_validation(L):
    cases = [(dict(dtype=7), ssv.SSV_ERR_INVALID), (dict(d=96), ssv.SSV_ERR_UNSUPPORTED),
             (dict(Hkv=0), ssv.SSV_ERR_INVALID), (dict(page_size=24), ssv.SSV_ERR_INVALID),
             (dict(max_block=0), ssv.SSV_ERR_INVALID), (dict(max_new=-1), ssv.SSV_ERR_INVALID),
             (dict(k_new=M + 8), ssv.SSV_ERR_INVALID), (dict(v_stride=128), ssv.SSV_ERR_INVALID),
             (dict(k_stride=260), ssv.SSV_ERR_INVALID), (dict(new_len=None), ssv.SSV_ERR_INVALID),
             (dict(v_scale=None), ssv.SSV_ERR_INVALID), (dict(n_pages=1 << 28), ssv.SSV_ERR_INVALID)]
    for kw, code in cases:
        assert L.ssv_commit_fp8(C.byref(_commit(**kw)), None) == code, kw
    assert L.ssv_commit_fp8(None, None) == ssv.SSV_ERR_INVALID
    assert L.ssv_commit_fp8(C.byref(_commit(batch=0)), None) == ssv.SSV_OK


def test_binding_refuses_wrong_tensors():
    """Shapes, types and strides are checked before any address is passed on."""
    seqs = torch.zeros((2, 6), dtype=torch.int32)
    batch = ssv.Batch.from_device(seqs, 8, 4, 10, 0, 2)
    tau, acc = torch.zeros(4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    cache, scale = torch.zeros((3, 2, 16, 128), dtype=torch.uint8), torch.zeros((3, 2))
    pages = torch.zeros(6, dtype=torch.int32)
    rows, q = torch.zeros((8, 2, 128), dtype=torch.bfloat16), torch.zeros((8, 4, 128), dtype=torch.bfloat16)
    ok = dict(k_cache=cache, v_cache=cache, k_scale=scale, v_scale=scale, pages=pages)

    def refused(f, *a, **kw):
        with pytest.raises(ssv.SsvError) as e:
            f(*a, **kw)
        assert e.value.code == ssv.SSV_ERR_INVALID

    for bad in (dict(k_cache=cache.float()), dict(v_cache=cache[:2]), dict(k_scale=scale.double()),
                dict(v_scale=scale[:, :1]), dict(pages=pages.long()), dict(k_cache=cache[:, :, ::2])):
        c = {**ok, **bad}
        refused(ssv.commit_fp8, rows, rows, c["k_cache"], c["v_cache"], c["k_scale"], c["v_scale"], c["pages"], batch,
                tau, acc)
        refused(ssv.verify_attn_fp8, q, c["k_cache"], c["v_cache"], c["k_scale"], c["v_scale"], c["pages"], rows,
                rows, batch, tau)
    args = (cache, cache, scale, scale, pages)
    refused(ssv.commit_fp8, rows, rows.float(), *args, batch, tau, acc)
    refused(ssv.commit_fp8, rows, rows, *args, batch, tau, acc[:1])
    refused(ssv.verify_attn_fp8, q.float(), *args, rows, rows, batch, tau)
    refused(ssv.verify_attn_fp8, q, *args, rows[:7], rows[:7], batch, tau)
    refused(ssv.verify_attn_fp8, q, *args, rows.transpose(1, 2), rows, batch, tau)
    w = torch.ones(128, dtype=torch.bfloat16)
    refused(ssv.norm_rope_copy, q, rows, w[:64], w, batch)
    refused(ssv.norm_rope_copy, q, rows, w, w.float(), batch)
    refused(ssv.norm_rope_copy, q, rows, w, w, batch, positions=torch.zeros(7, dtype=torch.int32))
    refused(ssv.norm_rope_copy, q, rows[:, :, ::2], w, w, batch)
    i2 = torch.zeros(2, dtype=torch.int32)
    refused(ssv.page_plan, i2, i2, i2.long(), i2, torch.zeros((2, 4), dtype=torch.int32), i2, i2[:1], 16, 10)
    refused(ssv.page_plan, i2, i2, i2, i2, torch.zeros((3, 4), dtype=torch.int32), i2, i2[:1], 16, 10)
    assert np.array_equal(cache.numpy(), np.zeros_like(cache.numpy()))


def test_attn_output_over_its_inputs(L):
    """o written over rows that other CTAs still read."""
    rows, wide = 40, 3 * 8 * 128   # K and V as parts of a fused projection
    for kw in (dict(o=M), dict(o=7 * M), dict(o=M + 2 * rows * 32 * 128 - 16), dict(o=8 * M - 2 * rows * 32 * 128 + 16),
               dict(o=7 * M + 2 * (rows - 1) * wide + 2 * 8 * 128 - 16, k_stride=wide)):
        assert L.ssv_verify_attn_fp8(C.byref(_attn(**kw)), 64 * M, 1 << 40, None) == ssv.SSV_ERR_INVALID, kw


def test_binding_refuses_host_tensors():
    """Tensors that are right but for where they are: no host address reaches a kernel."""
    seqs = torch.zeros((2, 6), dtype=torch.int32)
    batch = ssv.Batch.from_device(seqs, 8, 4, 10, 0, 2)
    tau, acc = torch.zeros(4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    cache, scale = torch.zeros((3, 2, 16, 128), dtype=torch.uint8), torch.zeros((3, 2))
    pages, w = torch.zeros(6, dtype=torch.int32), torch.ones(128, dtype=torch.bfloat16)
    rows, q = torch.zeros((8, 2, 128), dtype=torch.bfloat16), torch.zeros((8, 4, 128), dtype=torch.bfloat16)
    i2 = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: ssv.commit_fp8(rows, rows, cache, cache, scale, scale, pages, batch, tau, acc),
                 lambda: ssv.verify_attn_fp8(q, cache, cache, scale, scale, pages, rows, rows, batch, tau,
                                             workspace=torch.zeros(1 << 24, dtype=torch.uint8)),
                 lambda: ssv.norm_rope_copy(q, rows, w, w, batch),
                 lambda: ssv.page_plan(i2, i2, i2, i2, torch.zeros((2, 4), dtype=torch.int32), i2, i2[:1], 16, 10)):
        with pytest.raises(ssv.SsvError, match="one CUDA device"):
            call()
