"""A whole pass of the paged-cache loop captured once and replayed, its lengths and tables carried on the device; requests
that share the pages of a common prompt."""
import numpy as np
import pytest
import torch

from diffusion_speculative_verification_gb300 import ssv, io as sio, workloads as W
from gpu_common import ensure_built
from paged_common import PagedBatch
from test_gpu_attn_fp8 import check

pytestmark = pytest.mark.gpu
HQ, HKV, D, PAGE, N_PAGES, BATCH = 4, 2, 128, 32, 40, 3


def setup_module():
    ensure_built()


def state():
    r = np.random.default_rng(1)
    ints = lambda x: sio.int_tensor(np.asarray(x, np.int32), "cuda")  # noqa: E731
    return dict(C=ints([0, 0, 0]), N=ints([40, 1, 17]), B=ints([4, 8, 3]), held=ints([0] * 3),
                pages=torch.full((BATCH, N_PAGES), -1, dtype=torch.int32, device="cuda"), free=ints(r.permutation(N_PAGES)),
                n_free=ints([N_PAGES]), tau=ints(np.concatenate([W.random_tau(r, b) for b in (4, 8, 3)])),
                n_acc=ints([2, 8, 0]), status=ints([0]),
                codes=[torch.zeros((N_PAGES, HKV, PAGE, D), dtype=torch.uint8, device="cuda") for _ in range(2)],
                scale=[torch.ones((N_PAGES, HKV), device="cuda") for _ in range(2)],
                w=torch.ones(D, dtype=torch.bfloat16, device="cuda"))


def one_pass(s, qkv):
    """In place on every tensor of `s`; returns the attention's output."""
    rows = 58 + 30
    q, k, v = qkv[:, :HQ], qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:]
    seqs, _, _, held, n_free = ssv.page_plan(s["C"], s["N"], s["B"], s["held"], s["pages"], s["free"], s["n_free"], PAGE,
                                             rows, dev_status=s["status"])
    s["held"].copy_(held)
    s["n_free"].copy_(n_free)
    batch = ssv.Batch.from_device(seqs, rows, 15, PAGE * N_PAGES, 40, 8)
    q, k = ssv.norm_rope_copy(q, k, s["w"], s["w"], batch, q_out=torch.empty(q.shape, dtype=q.dtype, device="cuda"),
                              k_out=torch.empty(k.shape, dtype=k.dtype, device="cuda"), dev_status=s["status"])
    o = ssv.verify_attn_fp8(q, *s["codes"], *s["scale"], s["pages"], k, v, batch, s["tau"], dev_status=s["status"])
    ssv.commit_fp8(k, v, *s["codes"], *s["scale"], s["pages"], batch, s["tau"], s["n_acc"], new_len=s["C"],
                   cache_len=s["C"], dev_status=s["status"])
    return o


def test_a_captured_pass_goes_on_from_replay_to_replay():
    g = torch.Generator(device="cuda").manual_seed(3)
    inputs = [torch.randn((88, HQ + 2 * HKV, D), device="cuda", generator=g).bfloat16() for _ in range(20)]
    eager, replayed = state(), state()
    keep = {k: v.clone() for k, v in replayed.items() if isinstance(v, torch.Tensor)}
    one_pass(replayed, inputs[0])               # warm-up, taken back
    for k, v in keep.items():
        replayed[k].copy_(v)
    for c, y in zip(replayed["codes"] + replayed["scale"], eager["codes"] + eager["scale"]):
        c.copy_(y)
    x = inputs[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = one_pass(replayed, x)
    refused = 0
    for y in inputs:
        x.copy_(y)
        graph.replay()
        want = one_pass(eager, y)
        code = ssv.get_status(replayed["status"])
        assert code == ssv.get_status(eager["status"]) and code in (ssv.SSV_OK, ssv.SSV_ERR_NO_PAGES)
        refused += code == ssv.SSV_ERR_NO_PAGES
        if code == ssv.SSV_OK:
            assert torch.equal(o, want)
        for k in ("C", "held", "pages", "free", "n_free"):
            assert torch.equal(replayed[k], eager[k]), k
        for a, b in zip(replayed["codes"] + replayed["scale"], eager["codes"] + eager["scale"]):
            assert torch.equal(a, b)
    assert refused                              # 42, 9 and 17 tokens a pass: 1280 rows hold fewer than twenty of them


def test_requests_that_share_the_pages_of_a_prompt():
    """Reading needs no page of one's own: three requests over the same cached pages, one of them with a page more."""
    x = PagedBatch([160, 160, 200], [0, 1, 2], [8, 4, 3], 4, 2, 128, 32, seed=5)
    x.table[0, :5] = x.table[2, :5]
    x.table[1, :5] = x.table[2, :5]
    check(x)
