"""The loss and gradient of whole training steps: more long rows than SMs, at every number of CTAs per row (1, 2, 4, 8) with
blocks of 512 threads and with the target brought by one warp and by two, in place and beside the logits, against torch in 64
bits (tolerances: test_gpu_distill)."""
import pytest
import torch

from diffusion_speculative_verification_gb300 import ssv, workloads as W
from gpu_common import ensure_built
from logits_common import EPS, LN, placed

pytestmark = pytest.mark.gpu


def setup_module():
    ensure_built()


def reference(x, token, value, T, mode, w):
    """(loss, its tolerance, gradient, its tolerance before the last rounding, statistics) of rows x, in 64 bits."""
    z, t, there = x.double(), value.double(), token >= 0
    n, v = z.shape
    at = torch.where(there, token, 0).long()
    if mode == ssv.REST:
        p = torch.where(there, t.exp(), 0.0)
        r = (1 - p.sum(1, keepdim=True)).clamp(min=0)
    else:
        p = torch.softmax(torch.where(there, t, float("-inf")), 1)
        r = torch.zeros_like(p[:, :1])
    listed = torch.zeros_like(z).scatter_add_(1, at, there.double()) > 0
    dense = torch.zeros_like(z).scatter_add_(1, at, p)
    P = p.sum(1, keepdim=True) + r
    logq = torch.log_softmax(z / T, 1)
    m = z.amax(1, keepdim=True)
    mo = z.masked_fill(listed, float("-inf")).amax(1, keepdim=True)
    So = ((z - mo) / T).exp().masked_fill(listed, 0.0).sum(1, keepdim=True)
    S = ((z - m) / T).exp().sum(1, keepdim=True)
    ln_u = (mo - m) / T + So.log() - S.log()
    gap = torch.where(p > 0, p.clamp(min=1e-300).log() - logq.gather(1, at), 0.0)
    gap_r = torch.where(r > 0, r.clamp(min=1e-300).log() - ln_u, 0.0)
    loss = (p * gap).sum(1, keepdim=True) + r * gap_r
    dr = (token.shape[1] + 4) * 2 * EPS if mode == ssv.REST else 0.0
    tl = 2 * LN * P + LN * (p * gap.abs()).sum(1, keepdim=True) + dr * (gap_r.abs() + 1)
    share = ((z - mo) / T).exp().masked_fill_(listed, 0.0) / So
    q = logq.exp()
    grad = torch.where(listed, P * q - dense, share * (P * ln_u.exp() - r))
    tg = torch.where(listed, 2 * LN * P * q + LN * dense, share * (2 * LN * (P * ln_u.exp() + r) + dr) + dr * q)
    w = w.double()[:, None]
    live = w != 0
    stats = torch.where(live, torch.cat([m, S, mo, So], 1), 0.0)
    return (loss * w)[:, 0], (tl * w.abs() + EPS * (loss * w).abs())[:, 0], grad * (w / T), tg * (w / T).abs(), stats


def within(got, want, tol):
    d = (got.double() - want).abs() - tol
    assert not d.isnan().any() and float(d.max()) <= 0, (float(d.max()), divmod(int(d.argmax()), d.shape[-1]))


def rows(n, v, K, dtype, T, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(n, v, generator=g, device="cuda") * 2
    x.scatter_add_(1, torch.randint(0, v, (n, 30), generator=g, device="cuda"),
                   torch.empty(n, 30, device="cuda").exponential_(0.3, generator=g))
    x = x.to(dtype)
    target = (x.float() + 0.7 * torch.randn(n, v, generator=g, device="cuda")) / T
    top, at = target.topk(K, 1)
    value = top - torch.logsumexp(target, 1, keepdim=True)
    token = torch.where(torch.rand(n, K, generator=g, device="cuda") < 0.1, -1, at).int()
    w = torch.rand(n, generator=g, device="cuda") / n
    w[torch.rand(n, generator=g, device="cuda") < 0.1] = 0
    return x, token, value, w


# rows of 128 .. 160 KB per CTA: of one, two, four and eight CTAs, as many as leave none for more
STEPS = [(310, 70001, torch.bfloat16), (160, 151936, torch.bfloat16), (160, 151937, torch.bfloat16),
         (310, 37000, torch.float32), (160, 75001, torch.float32), (80, 151936, torch.float32), (40, 300003, torch.float32)]


@pytest.mark.parametrize("mode", [ssv.RENORM, ssv.REST])
@pytest.mark.parametrize("K", [20, 128])
@pytest.mark.parametrize("n,v,dtype", STEPS)
def test_steps(n, v, dtype, K, mode):
    T = 1.5
    x, token, value, w = rows(n, v, K, dtype, T, v + K)
    loss, tl, grad, tg, stats = reference(x, token, value, T, mode, w)
    tg += grad.abs() * (2.0 ** -8 if dtype == torch.bfloat16 else EPS) * (1 + 2.0 ** -6) + 2.0 ** -126
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def check(got, kept):
        assert ssv.get_status(status) == ssv.SSV_OK
        if kept is not None:     # the loss alone and with its gradient
            within(got[0], loss, tl)
            assert torch.equal(got[1][:, ::2].double(), stats[:, ::2])
            within(got[1][:, 1::2], stats[:, 1::2], LN * stats[:, 1::2])
        if got[2] is not None:
            within(got[2], grad, tg)

    check(ssv.distill(x, token, value, T, mode, w, dev_status=status), True)
    kept = None
    for lead, pad in ((0, 0), (3, 5)):
        # in place: every CTA reads its part again while others write theirs
        y, buf = placed(x, lead, pad, 3.0)
        got = ssv.distill(y, token, value, T, mode, w, grad=y, dev_status=status)
        check(got, True)
        kept = got[1].clone()
        y.copy_(x)
        check((None, None, ssv.distill_backward(y, token, value, kept, None, T, mode, w, grad=y, dev_status=status)), None)
        y.fill_(3.0)
        assert (buf == 3.0).all()
    # beside the logits: as they lie to 16-byte boundaries, and otherwise
    check(ssv.distill(x, token, value, T, mode, w, grad=True, dev_status=status), True)
    g, buf = placed(torch.zeros_like(x), 1, 2, 3.0)
    check(ssv.distill(x, token, value, T, mode, w, grad=g, dev_status=status), True)
    check((None, None, ssv.distill_backward(x, token, value, kept, None, T, mode, w, grad=g, dev_status=status)), None)
    g.fill_(3.0)
    assert (buf == 3.0).all()
