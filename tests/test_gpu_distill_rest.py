"""The rest of a distillation target to its own digits: r and u far below 1 and next to each other, where the other tokens'
gradient is a multiple of their small difference.

Tolerances of that gradient, (w / T) (q_v / u) (P u - r), derived before any run (logits_common: a sum is within LN of itself,
so that the share q_v / u and u are within 2 LN of themselves).  r = 1 - sum p, from exponentials that are off by what their
logarithms are: below 2^-30, and below 2^-23 of the logarithm itself where that is small (log_sum's series starts with it);
the pairs' additions by 2^-46; then r is rounded to fp32 and enters a difference that is rounded once."""
import numpy as np
import pytest
import torch

from diffusion_speculative_verification_gb300 import ssv, workloads as W
import oracle.distill as odist
from gpu_common import ensure_built
from logits_common import EPS, LN, near, store
from test_gpu_distill import half_step

pytestmark = pytest.mark.gpu


def setup_module():
    ensure_built()


def rest_error(value):
    """What the kernel's r is off by, before it is rounded, for a row's fp32 log-probabilities."""
    t = np.asarray(value, np.float64)
    t = t[t > -np.inf]
    return float(np.sum(np.exp(t) * np.minimum(2.0 ** -30, 2.0 ** -23 * np.abs(t))) + 2.0 ** -46)


def sharp(r, n, v, K, rest, factor, dtype, T, spread):
    """Drafter rows whose unlisted tokens have about factor * rest together, and targets that leave them `rest`; `spread`:
    the listed probability over the first three tokens, else nearly all on the first.  (logits as the dtype has them,
    token, value)"""
    z = r.standard_normal((n, v))
    token = np.stack([r.permutation(v)[:K] for _ in range(n)]).astype(np.int32)
    p = np.full((n, K), rest / 4 / K)
    head = min(K, 3) if spread else 1
    share = np.array([0.5, 0.3, 0.2])[:head] if spread else np.ones(1)
    p[:, :head] = (1 - rest - p[:, head:].sum(1, keepdims=True)) * (share / share.sum())
    others = np.ones((n, v), bool)
    np.put_along_axis(others, token.astype(np.int64), False, 1)
    s = np.where(others, np.exp(z / T), 0).sum(1)
    c = T * np.log(s * (1 - factor * rest) / (factor * rest))
    np.put_along_axis(z, token.astype(np.int64), T * np.log(p) + c[:, None] + 0.01 * r.standard_normal((n, K)), 1)
    ref, t = store(z, dtype)
    # the target again, so that u is `factor` times its rest with the logits as they have been rounded
    for i in range(n):
        x = (ref[i] - ref[i].max()) / T
        u = np.exp(x[others[i]]).sum() / np.exp(x).sum()
        p[i, head:] = u / factor / 4 / K
        p[i, :head] *= (1 - u / factor - p[i, head:].sum()) / p[i, :head].sum()
    return ref, t, token, np.log(p).astype(np.float32)


def other_gradient(ref, token, value, T, w):
    """(gradient [n, V] in 64 bits; of the unlisted tokens its tolerance before the last rounding; how far it may move with
    the order in which the target's sum is formed; unlisted [n, V])."""
    n, v = ref.shape
    grad, tol, same, unlisted = np.zeros((n, v)), np.zeros((n, v)), np.zeros((n, v)), np.ones((n, v), bool)
    for i in range(n):
        _, grad[i], stats = odist.row_distill(ref[i], token[i], value[i], T, odist.REST, w)
        p, listed, r = odist.target(token[i], value[i], odist.REST, v)
        unlisted[i] = ~listed
        u, P = np.exp(odist.log_rest(stats, T)), p.sum() + r
        share = np.exp((ref[i] - stats[2]) / T) / stats[3]
        tol[i] = share * abs(w / T) * (2 * LN * abs(P * u - r) + 2 * LN * P * u + rest_error(value[i]) + 4 * EPS * (r + u))
        q = np.exp((ref[i] - stats[0]) / T) / stats[1]
        same[i] = abs(w / T) * np.where(listed, 4 * EPS * (P * q + p), share * (2.0 ** -45 + 4 * EPS * (r + u)))
    return grad, tol, same, unlisted


@pytest.mark.parametrize("dtype", [W.F32, W.BF16])
@pytest.mark.parametrize("spread", [False, True])
@pytest.mark.parametrize("rest", [1e-3, 1e-5, 1e-6])
def test_gradient_of_a_small_rest(rest, spread, dtype):
    """Target and drafter leave the others little, one a fifth more than the other: both entry points give the gradient of
    the difference, and the same one."""
    r = np.random.default_rng(40)
    T, w = 1.5, 0.25
    for v, K, factor in ((500, 2, 1.2), (3001, 20, 0.8), (20000, 100, 1.2), (60000, 128, 2.0)):
        ref, t, token, value = sharp(r, 4, v, K, rest, factor, dtype, T, spread)
        want, tol, same, others = other_gradient(ref, token, value.astype(np.float64), T, w)
        a = [torch.tensor(token, device="cuda"), torch.tensor(value, device="cuda"), T, ssv.REST]
        wt = torch.full((4,), w, device="cuda")
        _, stats, fused = ssv.distill(t, *a, wt, grad=True)
        back = ssv.distill_backward(t, *a[:2], stats, None, *a[2:], wt)
        for g in (fused, back):
            g = g.float().cpu().numpy().astype(np.float64)
            near(g[others], want[others], (tol + half_step(want, dtype))[others])
        # the same formula on the same statistics
        near(back.float().cpu().numpy(), fused.float().cpu().numpy().astype(np.float64), same + 2 * half_step(want, dtype))


@pytest.mark.parametrize("dtype", [W.F32, W.BF16])
@pytest.mark.parametrize("T", [0.3, 0.7, 1.0, 1.5, 3.0])
def test_gradient_next_to_the_target(T, dtype):
    """One listed token and others that are all equal, 26 T .. 85 T below: sums are whole numbers and probabilities their
    logarithms' exponentials, so that u = S' e^-gap / S is off by the exponential (2 eps), its low part, S, the quotient, the
    product and P alone, r = -expm1(t) by its rounding.  They are next to each other, and the gradient is their difference.
    The exponent is a difference of fp32 numbers times 1 / T: as one product in fp32 it would be off by up to 85 eps."""
    r = np.random.default_rng(41)
    n, v, K = 48, 3001, 20
    T = float(np.float32(T))
    m = r.standard_normal(n) * 3
    z = np.repeat((m - T * np.linspace(26, 85, n))[:, None], v, 1)
    token = np.full((n, K), -1, np.int32)
    token[:, 7] = r.integers(0, v, n)
    at = (np.arange(n), token[:, 7])
    z[at] = m
    ref, t = store(z, dtype)
    low = ref[np.arange(n), (token[:, 7] + 1) % v]
    s = (v - 1) * np.exp((low - ref[at]) / T)
    u = s / (1 + s)
    value = np.full((n, K), -1.0, np.float32)
    apart = 1.001 if dtype == W.F32 else 1.00003        # bf16 shows an error only where it is multiplied by more
    value[:, 7] = np.log1p(-u / apart)
    rest = -np.expm1(value[:, 7].astype(np.float64))
    w = 2.0 ** 60                                       # brings the smallest back into fp32's range
    want = (u - rest) / (v - 1) * (w / T)
    tol = ((2 + 5) * EPS * u + 2 * EPS * rest + 4 * EPS * np.abs(u - rest)) / (v - 1) * (w / T) + half_step(want, dtype)
    a = [torch.tensor(token, device="cuda"), torch.tensor(value, device="cuda")]
    wt = torch.full((n,), w, device="cuda")
    _, stats, fused = ssv.distill(t, *a, T, ssv.REST, wt, grad=True)
    assert (stats[:, 3] == v - 1).all()
    back = ssv.distill_backward(t, *a, stats, None, T, ssv.REST, wt)
    for g in (fused, back):
        near(g.float().cpu().numpy()[np.arange(n), (token[:, 7] + 1) % v], want, tol)


@pytest.mark.parametrize("dtype", [W.F32, W.BF16])
@pytest.mark.parametrize("T", [0.7, 2.0])
def test_finite_masks(T, dtype):
    """Tokens masked with a number instead of -inf, on both sides: what the roundings of the target's log-probabilities leave
    of 1 is nobody's, and loss and gradient are those of the same rows masked with -inf."""
    r = np.random.default_rng(43)
    n, v, K = 8, 3001, 6
    for mask in (-1e3, -1e4, -1e9, -3.3895314e38):
        z = np.full((n, v), mask)
        legal = np.stack([r.permutation(v)[:3] for _ in range(n)])
        np.put_along_axis(z, legal, r.standard_normal((n, 3)) * 2, 1)
        target = z.copy()
        np.put_along_axis(target, legal, np.take_along_axis(z, legal, 1) + 0.3 * r.standard_normal((n, 3)), 1)
        ref, x = store(z, dtype)
        *_, value, token = ssv.logprobs(store(target, dtype)[1], None, K, T)
        value[:, :3] += torch.tensor(np.log1p(-5e-7) * r.random((n, 1)), dtype=torch.float32, device="cuda")
        assert (value.double().exp().sum(1) < 1).any()
        hidden = torch.where(x < -900, float("-inf"), x)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        want = ssv.distill(hidden, token, value, T, ssv.REST, grad=True, dev_status=status)
        loss, stats, grad = ssv.distill(x, token, value, T, ssv.REST, grad=True, dev_status=status)
        back = ssv.distill_backward(x, token, value, stats, None, T, ssv.REST, dev_status=status)
        assert ssv.get_status(status) == ssv.SSV_OK
        assert want[0].isfinite().all() and torch.equal(loss, want[0])
        assert torch.equal(grad, want[2])
        near(back.float().cpu().numpy(), grad.float().cpu().numpy().astype(np.float64),
             2 * half_step(grad.float().cpu().numpy().astype(np.float64), dtype) + 2.0 ** -21)
        own, _, _ = odist.distill_batch(ref, token.cpu().numpy(), value.double().cpu().numpy(), T, odist.REST)
        near(loss.cpu().numpy(), own, 4 * LN * (1 + np.abs(own)))
