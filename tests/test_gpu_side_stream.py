"""Calls on a stream other than the current one that make their outputs and
their scratch themselves: nothing of them is left on the current stream, which is
kept busy meanwhile."""
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


def beside_a_busy_stream(run):
    """run(stream) while the current stream copies, over memory that holds no zeros; its results once its own stream is
    through, which has to be before the current one is."""
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for s in (side, torch.cuda.current_stream()):       # memory that both streams' pools hand out again
        with torch.cuda.stream(s):
            junk = [torch.full((n,), 0x41, dtype=torch.uint8, device="cuda") for n in (1 << 12, 1 << 20, 40 << 20)]
            del junk
    torch.cuda.synchronize()
    done = torch.cuda.Event()
    host, dev = torch.empty(1 << 30, dtype=torch.uint8, pin_memory=True), torch.empty(1 << 30, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    for _ in range(100):                                # about 0.5 s of copies, which leave the SMs free
        dev.copy_(host, non_blocking=True)
    done.record()
    out = run(side)
    side.synchronize()
    assert not done.query()
    torch.cuda.synchronize()
    return [x.cpu() for x in out]


def test_paged_calls():
    x = PagedBatch([3000, 300], [0, 1], [8, 16], 4, 2, 128, 64, seed=1)
    t, u = x.device(), x.device()
    args = (t["k_scale"], t["v_scale"], t["pages"], t["batch"], t["tau"], t["n_acc"])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    want_o = call(u).cpu()
    want_n = ssv.commit_fp8(u["k_new"], u["v_new"], u["k_cache"], u["v_cache"], u["k_scale"], u["v_scale"], u["pages"],
                            u["batch"], u["tau"], u["n_acc"]).cpu()
    out = {}

    def run(s):
        out["o"] = call(t, stream=s, dev_status=status)
        out["n"] = ssv.commit_fp8(t["k_new"], t["v_new"], t["k_cache"], t["v_cache"], *args, stream=s, dev_status=status)
        return out["o"], out["n"]

    o, n = beside_a_busy_stream(run)
    assert ssv.get_status(status) == ssv.SSV_OK
    assert torch.equal(o, want_o) and torch.equal(n, want_n)
    assert torch.equal(t["k_cache"], u["k_cache"]) and torch.equal(t["v_cache"], u["v_cache"])


@pytest.mark.parametrize("batch", [0, 5])
def test_plan(batch):
    r = np.random.default_rng(2)
    ints = lambda y: sio.int_tensor(np.asarray(y, np.int32), "cuda")  # noqa: E731
    a = [ints(r.integers(0, 60, batch)), ints(r.integers(0, 9, batch)), ints(r.integers(1, 9, batch)), ints([0] * batch)]
    free, n = ints(r.permutation(64)), ints([64])

    def plan(s):
        return ssv.page_plan(*a, torch.full((batch, 16), -1, dtype=torch.int32, device="cuda") if s is None else table,
                             free.clone() if s is None else free, n, 16, 200, stream=s)

    want = [y.cpu() for y in plan(None)]
    table = torch.full((batch, 16), -1, dtype=torch.int32, device="cuda")
    for g, w in zip(beside_a_busy_stream(plan), want):
        assert torch.equal(g, w)


def test_flat_calls():
    t = sio.attn_to_device(W.make_attn_inputs("ws", [3000, 1], [0, 0], [8, 2], 4, 2, 128, W.BF16, 3))
    args = (t["q"], t["k_cache"], t["v_cache"], t["k_new"], t["v_new"], t["batch"], t["tau"])
    want = ssv.verify_attn(*args).cpu()
    x = sio.accept_to_device(W.make_accept_inputs("ss", W.MODE_ARGMAX, 0.0, 20000, np.array([4, 8]), np.array([4, 8]),
                                                  seed=4))
    acc = (x["mode"], x["T"], x["logits"], x["draft_tokens"], x["tau"], x["block"], x["gamma"], x["slot_off"])
    want_acc = [y.cpu() for y in ssv.accept(*acc)]
    got = beside_a_busy_stream(lambda s: (ssv.verify_attn(*args, stream=s), *ssv.accept(*acc, stream=s)))
    assert torch.equal(got[0], want) and all(torch.equal(g, w) for g, w in zip(got[1:], want_acc))
