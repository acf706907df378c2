"""One attention workspace over calls of other sizes, each of which cuts units
across CTAs: the counters of one call must not lie where another keeps its
partials or its plan.  Every output is compared, bit for bit, with a run on a
workspace of its own (units are merged in a fixed order)."""
import numpy as np
import pytest
import torch

from diffusion_speculative_verification_gb300 import ssv, io as sio, workloads as W
from gpu_common import ensure_built
from paged_common import PagedBatch
from test_gpu_attn_fp8 import call

pytestmark = pytest.mark.gpu


def setup_module():
    ensure_built()


def paged(C, N, B, hq, hkv, seed):
    return PagedBatch(C, N, B, hq, hkv, 128, 64, seed=seed).device()


def serve(shapes, run, size):
    """Each shape on a cleared workspace of its own, then all of them, three rounds and back, on one that is never
    cleared; returns that workspace."""
    want = [run(s, torch.zeros(size(s), dtype=torch.uint8, device="cuda")).clone() for s in shapes]
    ws = torch.zeros(max(size(s) for s in shapes), dtype=torch.uint8, device="cuda")
    order = list(range(len(shapes)))
    for i in order * 3 + order[::-1]:
        assert torch.equal(run(shapes[i], ws), want[i]), i
    return ws


def fp8_size(t):
    return ssv.verify_attn_fp8_workspace(t["q"], t["k_cache"], t["v_cache"], t["k_scale"], t["v_scale"], t["pages"],
                                         t["k_new"], t["v_new"], t["batch"], t["tau"]).numel()


def run_fp8(t, ws):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    o = call(t, workspace=ws, dev_status=status)
    assert ssv.get_status(status) == ssv.SSV_OK
    return o


def test_fp8_batches_of_two_and_three():
    """Two long-and-short batches: the units of both are cut over several CTAs."""
    ts = [paged([3000, 1], [0, 0], [8, 2], 4, 2, 1), paged([3000, 1, 1], [0, 0, 0], [8, 2, 2], 4, 2, 2)]
    serve(ts, run_fp8, fp8_size)


def test_fp8_batch_falls_below_the_tables_in_shared_memory():
    """65 sequences keep their plan in the workspace, 64 and 60 in shared memory."""
    r = np.random.default_rng(3)
    C = r.integers(100, 900, 65)
    ts = [paged(C[:n], [0] * n, [1 + i % 20 for i in range(n)], 8, 8, n) for n in (65, 64, 60, 61)]
    serve(ts, run_fp8, fp8_size)


def test_fp8_prompt_chunk_between_decode_passes():
    """At one batch size, more rows: 4 sequences decoding, then one of them with a prompt of 2048 rows."""
    C, B = [4000, 3500, 2000, 3900], [8, 4, 8, 2]
    ts = [paged(C, [0] * 4, B, 32, 8, 5), paged(C, [2048, 0, 0, 0], B, 32, 8, 6), paged(C, [0, 1, 0, 40], B, 32, 8, 7)]
    ws = serve(ts, run_fp8, fp8_size)
    assert not ws[: 4096].any()   # the counters, 32 bytes for each CTA, are zero again


def flat(C, N, B, hq, hkv, seed):
    return sio.attn_to_device(W.make_attn_inputs("ws", C, N, B, hq, hkv, 128, W.BF16, seed))


def flat_size(t):
    return ssv.verify_attn_workspace_bytes(ssv.attn_args(t["q"], t["k_cache"], t["v_cache"], t["k_new"], t["v_new"],
                                                         t["q"], t["batch"], t["tau"]))


def run_flat(t, ws):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    o = ssv.verify_attn(t["q"], t["k_cache"], t["v_cache"], t["k_new"], t["v_new"], t["batch"], t["tau"], workspace=ws,
                        dev_status=status)
    assert ssv.get_status(status) == ssv.SSV_OK
    return o


def test_flat_cache_over_batches_and_prompts():
    """ssv_verify_attn: batches of 2 and 3, of 130 (plan tables in the workspace), 129 and 40, and a prompt chunk between
    decode passes."""
    r = np.random.default_rng(9)
    C = [int(c) for c in r.integers(100, 900, 130)]
    B = [32 if i % 7 == 0 else 1 + i % 16 for i in range(130)]
    ts = [flat([3000, 1], [0, 0], [8, 2], 4, 2, 1), flat([3000, 1, 1], [0, 0, 0], [8, 2, 2], 4, 2, 2)]
    ts += [flat(C[:n], [0] * n, B[:n], 32, 8, n) for n in (130, 129, 40)]
    ts += [flat([4000, 3500, 2000, 3900], [n, 0, 0, 0], [8, 4, 8, 2], 32, 8, n + 1) for n in (0, 2048, 1)]
    ws = serve(ts, run_flat, flat_size)
    assert not ws[: 4096].any()


def test_flat_and_paged_calls_share_one():
    """ssv_verify_attn and ssv_verify_attn_fp8 keep their counters at the same place."""
    ts = [paged([3000, 1], [0, 0], [8, 2], 4, 2, 11), flat([3000, 1, 700], [0, 40, 0], [8, 2, 33], 4, 2, 12),
          paged([100, 2700, 60], [1, 0, 300], [8, 2, 30], 4, 2, 13), flat([5000], [0], [8], 8, 2, 14)]
    serve(ts, lambda t, ws: (run_fp8 if "pages" in t else run_flat)(t, ws),
          lambda t: (fp8_size if "pages" in t else flat_size)(t))
