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


def test_rows_that_share_memory_are_refused():
    """One row expanded over all (row stride 0) or rows that overlap: the library would read rows that are not there."""
    seqs = torch.zeros((2, 6), dtype=torch.int32)
    batch = ssv.Batch.from_device(seqs, 8, 4, 10, 0, 2)
    tau, acc = torch.zeros(4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    cache, scale = torch.zeros((3, 2, 16, 128), dtype=torch.uint8), torch.zeros((3, 2))
    pages, w = torch.zeros(6, dtype=torch.int32), torch.ones(128, dtype=torch.bfloat16)
    rows, q = torch.zeros((8, 2, 128), dtype=torch.bfloat16), torch.zeros((8, 4, 128), dtype=torch.bfloat16)
    c = (cache, cache, scale, scale, pages)

    def shared(heads):
        yield torch.zeros((1, heads, 128), dtype=torch.bfloat16).expand(8, heads, 128)
        yield torch.zeros((4096,), dtype=torch.bfloat16).as_strided((8, heads, 128), (128, 128, 1))

    for r in shared(2):
        for f in (lambda: ssv.norm_rope_copy(q, r, w, w, batch, k_out=rows),
                  lambda: ssv.norm_rope_copy(q, r, w, w, batch),
                  lambda: ssv.norm_rope_copy(q, rows, w, w, batch, k_out=r),
                  lambda: ssv.verify_attn_fp8(q, *c, r, rows, batch, tau),
                  lambda: ssv.verify_attn_fp8(q, *c, rows, r, batch, tau),
                  lambda: ssv.commit_fp8(r, rows, *c, batch, tau, acc),
                  lambda: ssv.commit_fp8(rows, r, *c, batch, tau, acc)):
            with pytest.raises(ssv.SsvError, match="rows that do not overlap"):
                f()
    for r in shared(4):
        with pytest.raises(ssv.SsvError, match="rows that do not overlap"):
            ssv.norm_rope_copy(r, rows, w, w, batch, q_out=q)
    assert ssv._rows_strided(rows[:1].expand(1, 2, 128), "") == 0       # a single row is itself
    assert ssv._rows_strided(torch.zeros((8, 6, 128))[:, 2:4], "") == 6 * 128


def test_workspace_of_one_element_expanded_is_refused():
    q = torch.zeros((8, 4, 128), dtype=torch.bfloat16)
    with pytest.raises(ssv.SsvError, match="the workspace is contiguous"):
        ssv._launch("ssv_verify_attn_fp8", (q,), b"", None, torch.zeros(1, dtype=torch.uint8).expand(1 << 24))


def test_outputs_and_scratch_are_made_on_the_stream_of_the_call(L, monkeypatch):
    """Tensors that a call makes itself are made under the stream that it was given."""
    made, entered = [], []

    class On:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            entered.append(self.stream)

        def __exit__(self, *a):
            entered.pop()

    def spy(f):
        def g(*a, **kw):
            made.append(entered[-1] if entered else None)
            return f(*a, **kw)
        return g

    seqs = torch.zeros((2, 6), dtype=torch.int32)
    batch = ssv.Batch.from_device(seqs, 8, 4, 10, 0, 2)
    tau, acc = torch.zeros(4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    cache, scale = torch.zeros((3, 2, 16, 128), dtype=torch.uint8), torch.zeros((3, 2))
    pages, i2, table = torch.zeros(6, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros((2, 4), dtype=torch.int32)
    rows, q = torch.zeros((8, 2, 128), dtype=torch.bfloat16), torch.zeros((8, 4, 128), dtype=torch.bfloat16)
    c = (cache, cache, scale, scale, pages)
    ws = torch.zeros(1 << 16, dtype=torch.uint8)
    monkeypatch.setattr(torch.cuda, "stream", On)
    monkeypatch.setattr(torch, "empty", spy(torch.empty))
    monkeypatch.setattr(torch, "zeros", spy(torch.zeros))
    s = object()
    for call, n in ((lambda: ssv.verify_attn_fp8(q, *c, rows, rows, batch, tau, stream=s), 2),
                    (lambda: ssv.verify_attn_fp8(q, *c, rows, rows, batch, tau, stream=s, workspace=ws), 1),
                    (lambda: ssv.commit_fp8(rows, rows, *c, batch, tau, acc, stream=s), 1),
                    (lambda: ssv.page_plan(i2, i2, i2, i2, table, i2, i2[:1], 16, 10, stream=s), 1)):
        made.clear()
        with pytest.raises(ssv.SsvError, match="one CUDA device"):
            call()
        assert made == [s] * n
    made.clear()
    assert ssv.verify_attn_fp8_workspace(q, *c, rows, rows, batch, tau, stream=s).numel() and made == [s]


def test_attn_bounds_of_many_requests_and_a_long_prompt(L):
    """Units follow the rows there are, not batch times the longest: 1000 decoding requests beside a prompt of 32768."""
    n = C.c_size_t(0)
    big = dict(batch=1000, total_rows=33 * 1000 + 32768, total_slots=16000, max_cache=32768, max_new=32768, max_block=16)
    assert L.ssv_verify_attn_fp8_workspace(C.byref(_attn(**big)), C.byref(n)) == ssv.SSV_OK
    assert n.value < 2 << 30
    big.update(total_rows=1 << 28, max_cache=1 << 20)
    assert L.ssv_verify_attn_fp8_workspace(C.byref(_attn(**big)), C.byref(n)) == ssv.SSV_ERR_UNSUPPORTED
