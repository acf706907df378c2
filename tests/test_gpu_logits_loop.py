"""The logits operators as a server and a training step use them: the acceptance's tokens scored, the target's
alternatives kept, a drafter's loss and gradient against them; the same captured and replayed over other logits."""
import numpy as np
import pytest
import torch

from diffusion_speculative_verification_gb300 import ssv, io as sio, workloads as W
import oracle.accept as oacc
import oracle.distill as odist
import oracle.logprobs as olp
from gpu_common import ensure_built
from logits_common import EPS, LN, near
from test_gpu_distill import half_step, tolerances

pytestmark = pytest.mark.gpu
BLOCKS, V, K, T = [8, 4, 16, 1], 9001, 20, 1.5


def setup_module():
    ensure_built()


def inputs(seed):
    x = W.make_accept_inputs("logits_loop", W.MODE_ARGMAX, 0.0, V, BLOCKS, [b - b // 4 for b in BLOCKS], seed=seed)
    r = np.random.default_rng(seed)
    draft = (x.logits.astype(np.float64) + 0.5 * r.standard_normal(x.logits.shape)).astype(np.float32)
    return x, draft


def stage_rows(tau, block, slot_off):
    """Row (slot) of every token of the acceptance's output, which is in the order of the stages."""
    slot = torch.arange(tau.numel(), device=tau.device)
    b = torch.searchsorted(slot_off, slot.int(), right=True) - 1
    rows = torch.empty_like(tau)
    rows[slot_off[b].long() + tau.long() - 1] = slot.int()
    return rows


def weights(tau):
    """exp(-(stage - 1) / 7) of every slot."""
    return torch.exp(-(tau.float() - 1) / 7)


def step(d, draft, status):
    """One pass: tokens, their log-probabilities, the target's alternatives per slot, the drafter's loss and gradient."""
    n_acc, n_out, tokens = ssv.accept(d["mode"], d["T"], d["logits"], d["draft_tokens"], d["tau"], d["block"], d["gamma"],
                                      d["slot_off"], max_block=d["max_block"], dev_status=status)
    rows = stage_rows(d["tau"], d["block"], d["slot_off"])
    scored = ssv.logprobs(d["logits"], tokens, 5, rows=rows, dev_status=status)
    _, _, _, _, top_logprob, top_token = ssv.logprobs(d["logits"], None, K, T, dev_status=status)
    w = weights(d["tau"])
    loss, stats, grad = ssv.distill(draft, top_token, top_logprob, T, ssv.REST, w, grad=True, dev_status=status)
    up = loss / loss.sum()
    again = ssv.distill_backward(draft, top_token, top_logprob, stats, up, T, ssv.REST, w, dev_status=status)
    return (tokens, *scored, top_logprob, top_token, loss, stats, grad, up, again)


def check(x, draft, out):
    tokens, lp, rank, ent, lse, tl, tt, top_logprob, top_token, loss, stats, grad, up, again = (
        None if o is None else o.cpu().numpy() for o in out)
    ref = oacc.accept_batch(x)
    assert tokens.tolist() == ref["tokens"].tolist()
    z = x.logits.astype(np.float64)
    rows = np.empty(len(x.tau), np.int64)
    for b, off in enumerate(x.slot_off):
        for k in range(x.blocks[b]):
            rows[off + x.tau[off + k] - 1] = off + k
    want = olp.logprobs_batch(z, tokens, rows, 5, 1.0)
    near(lp, want["logprob"], LN + EPS * np.abs(want["logprob"]))
    near(ent, want["entropy"], 2 * LN * (1 + want["entropy"]))
    near(lse, want["lse"], LN + EPS * np.abs(want["lse"]))
    assert np.array_equal(rank, want["rank"]) and np.array_equal(tt, want["top_token"])
    assert (rank[tokens >= 0] == 1).all()                      # greedy: what is emitted is the most likely
    want = olp.logprobs_batch(z, None, None, K, T)
    assert np.array_equal(top_token, want["top_token"])
    near(top_logprob, want["top_logprob"], LN + 4 * EPS * np.abs(want["top_logprob"]))
    # the loss on the alternatives that were kept
    d = draft.astype(np.float64)
    w = weights(torch.tensor(x.tau)).numpy().astype(np.float64)
    wl, wg, ws = odist.distill_batch(d, top_token, top_logprob, T, odist.REST, w)
    tol, tg = tolerances(d, top_token, top_logprob, T, odist.REST, w)
    near(loss, wl, tol + EPS * np.abs(wl) + 2 * EPS * w)        # exp rounds the weights
    near(grad, wg, tg + half_step(wg, W.F32) + 4 * EPS * np.abs(wg))
    wb = wg * up.astype(np.float64)[:, None]
    near(again, wb, tg * np.abs(up)[:, None] + half_step(wb, W.F32) + 4 * EPS * np.abs(wb))


def test_a_pass_and_a_training_step():
    for seed in (1, 2):
        x, draft = inputs(seed)
        d = sio.accept_to_device(x)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = step(d, torch.tensor(draft, device="cuda"), status)
        assert ssv.get_status(status) == ssv.SSV_OK
        check(x, draft, out)


def test_captured():
    """One capture replayed over the logits of other passes; the results of eager calls made meanwhile stay theirs."""
    data = [inputs(seed) for seed in (3, 4)]
    d = sio.accept_to_device(data[0][0])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    draft = torch.tensor(data[0][1], device="cuda")
    want = []
    for x, z in data:
        e = sio.accept_to_device(x)
        want.append([o for o in step(e, torch.tensor(z, device="cuda"), status)])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step(d, draft, status)
    for k in (1, 0, 1):
        e = sio.accept_to_device(data[k][0])
        for name in ("logits", "draft_tokens", "tau"):
            d[name].copy_(e[name])
        draft.copy_(torch.tensor(data[k][1], device="cuda"))
        g.replay()
        torch.cuda.synchronize()
        assert ssv.get_status(status) == ssv.SSV_OK
        assert all(torch.equal(a, b) for a, b in zip(out, want[k]))
        check(*data[k], out)


def test_beside_a_busy_stream():
    """Outputs made by the calls on a stream of their own."""
    from test_gpu_side_stream import beside_a_busy_stream
    x, draft = inputs(5)
    d, z = sio.accept_to_device(x), torch.tensor(draft, device="cuda")
    top = ssv.logprobs(d["logits"], None, K, T)
    want = [o.cpu() for o in top[2:]]
    ref = ssv.distill(z, top[5], top[4], T, grad=True)
    want += [o.cpu() for o in ref] + [ssv.distill_backward(z, top[5], top[4], ref[1], None, T).cpu()]

    def run(s):
        _, _, ent, lse, tl, tt = ssv.logprobs(d["logits"], None, K, T, stream=s)
        out = ssv.distill(z, tt, tl, T, grad=True, stream=s)
        return (ent, lse, tl, tt, *out, ssv.distill_backward(z, tt, tl, out[1], None, T, stream=s))

    for a, b in zip(beside_a_busy_stream(run), want):
        assert torch.equal(a, b)
