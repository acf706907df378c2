"""The operators on logits as a program uses them: the map of accepted tokens' rows, and a gradient that goes on into the
drafter's own graph."""
import numpy as np
import pytest
import torch

from diffusion_speculative_verification_gb300 import ssv
from gpu_common import ensure_built
from logits_common import EPS, LN

pytestmark = pytest.mark.gpu


def setup_module():
    ensure_built()


def test_rows_of_accepted_tokens():
    r = np.random.default_rng(50)
    blocks = [8, 1, 4, 16]
    off = np.concatenate([[0], np.cumsum(blocks)[:-1]])
    stage = np.concatenate([r.permutation(b) + 1 for b in blocks])
    tau = torch.tensor(stage, dtype=torch.int32, device="cuda")
    slot_off = torch.tensor(off, dtype=torch.int32, device="cuda")
    slot = torch.arange(tau.numel(), dtype=torch.int32, device="cuda")
    start = slot_off[torch.searchsorted(slot_off, slot, right=True) - 1]
    rows = torch.empty_like(tau)
    rows[(start + tau - 1).long()] = slot
    for b, o in zip(blocks, off):
        for k in range(b):
            assert rows[o + stage[o + k] - 1] == o + k
    x = torch.randn(int(tau.numel()), 900, device="cuda")
    tokens = torch.randint(0, 900, (int(tau.numel()),), device="cuda").int()
    lp = ssv.logprobs(x, tokens, rows=rows)[0]
    want = torch.log_softmax(x.double(), 1)[rows.long(), tokens.long()]
    assert float(((lp - want).abs() - LN - EPS * want.abs()).max()) <= 0


@pytest.mark.parametrize("v", [1000, 9001])      # gradient rows that are packed, and that lie as the logits' do
@pytest.mark.parametrize("mode", [ssv.RENORM, ssv.REST])
def test_gradient_into_a_drafter(mode, v):
    """Logits of a linear head: its weight's gradient through the operators and through autograd in 64 bits.  The gradient of
    the logits is within 2^-14 of its terms P q + p (test_gpu_distill: 2 LN of each, LN for r), and a head's weight sums its
    products with the hidden states in fp32: 2^-12 of the sum of their magnitudes is more than both."""
    g = torch.Generator(device="cuda").manual_seed(51)
    T, n, h, K = 2.0, 24, 32, 12
    hidden = torch.randn(n, h, generator=g, device="cuda")
    w = (torch.randn(v, h, generator=g, device="cuda") / 4).requires_grad_()
    *_, value, token = ssv.logprobs(torch.randn(n, v, generator=g, device="cuda") * 3, None, K, T)
    wide = torch.zeros(n, v + 7, device="cuda")
    logits = torch.addmm(wide[:, :v] if v == 9001 else torch.zeros(n, v, device="cuda"), hidden, w.t())
    weight = torch.rand(n, generator=g, device="cuda")
    loss, stats, grad = ssv.distill(logits, token, value, T, mode, weight, grad=True)
    assert loss.grad_fn is None and grad.grad_fn is None
    logits.backward(grad)
    back = ssv.distill_backward(logits, token, value, stats, None, T, mode, weight)
    assert float((back - grad).abs().max()) <= 2.0 ** -20

    d = w.detach().double().requires_grad_()
    q = torch.log_softmax(hidden.double() @ d.t() / T, 1)
    t = value.double()
    p = t.exp() if mode == ssv.REST else torch.softmax(t, 1)
    at = token.long()
    total = (p * (p.log() - q.gather(1, at))).sum(1)
    if mode == ssv.REST:
        r = 1 - p.sum(1)
        u = torch.zeros_like(q, dtype=torch.bool).scatter_(1, at, True)
        total = total + r * (r.log() - torch.logsumexp(q.masked_fill(u, float("-inf")), 1))
    (total * weight.double()).sum().backward()
    size = (q.exp() + torch.zeros_like(q).scatter_(1, at, p)).detach() * (weight.double() / T)[:, None]
    tol = 2.0 ** -12 * (size.t() @ hidden.double().abs()) + 2.0 ** -30
    assert (loss - total * weight).abs().max() <= 2.0 ** -12
    assert float(((w.grad - d.grad).abs() - tol).max()) <= 0
