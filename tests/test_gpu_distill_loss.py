"""Losses next to 0 to their own digits: a drafter that has nearly learnt its target.

Tolerances, derived before any run.  A loss is the sum of p (ln p - ln q) and r (ln r - ln u).  Logarithms of sums are within
2^-30 of what their sums give (log_sum's series), and relatively within 2^-23 where the sum is 1 and a little; each difference
is rounded once to fp32.  What the sums are off by: a listed token's exponential by 2 eps unless it is 1, the others' share by
LN of itself (logits_common), or, where they are all equal and their sum a whole number, by the one factor that brings them to
the row's maximum (2^-22 and 3 eps of its exponent)."""
import numpy as np
import pytest
import torch

from diffusion_speculative_verification_gb300 import ssv, workloads as W
import oracle.distill as odist
from gpu_common import ensure_built
from logits_common import EPS, LN, near, store
from test_gpu_distill_rest import rest_error, sharp

pytestmark = pytest.mark.gpu


def setup_module():
    ensure_built()


def on_gpu(token, value):
    return torch.tensor(token, device="cuda"), torch.tensor(np.asarray(value, np.float32), device="cuda")


@pytest.mark.parametrize("dtype", [W.F32, W.BF16])
@pytest.mark.parametrize("mode", [ssv.RENORM, ssv.REST])
def test_equal_probabilities(mode, dtype):
    """K tokens of equal probability, as many of equal logits: every exponential is 1, and p as q K times 1 / K but for the
    little u that the others take.  RENORM: loss = -ln(1 - u)."""
    T = float(np.float32(0.7))
    for K in (2, 3, 60, 100, 127, 128):
        n, v = 10, 3001
        r = np.random.default_rng(K)
        # the others: -inf (where the target leaves them nothing), then more and more of them
        gap = np.array([np.inf if mode == ssv.RENORM else 45.0, 40.0, 25, 20, 17, 15, 13, 12, 11, 10]) * T
        z = np.repeat(-gap[:, None], v, 1)
        token = np.stack([r.permutation(v)[:K] for _ in range(n)]).astype(np.int32)
        np.put_along_axis(z, token.astype(np.int64), 0.0, 1)
        ref, t = store(z, dtype)
        value = np.full((n, K), -np.log(K), np.float32) + (0.0 if mode == ssv.REST else np.float32(3.7))
        if mode == ssv.REST:
            value = value * np.float32(1 + 2.0 ** -12)                                  # a rest of 2^-12 ln K
        loss = ssv.distill(t, *on_gpu(token, value), T, mode)[0].cpu().numpy()
        want, _, stats = odist.distill_batch(ref, token, value.astype(np.float64), T, mode)
        ln_u = np.array([odist.log_rest(s, T) for s in stats])
        if mode == ssv.RENORM:
            others = (v - K) * np.exp(-np.where(np.isinf(ref.min(1)), np.inf, -ref.min(1)) / T)
            want = np.log1p(others / K)                  # the oracle's own difference would be off by 2^-52 ln K
        u = np.exp(ln_u)
        y = np.where(u > 0, -ref.min(1) / T, 0.0)
        tol = 2.0 ** -29 + u * (2.0 ** -22 + 3 * EPS * y) + 2 * EPS * np.abs(want)
        if mode == ssv.REST:
            for i in range(n):
                p = np.exp(value[i].astype(np.float64))
                rest = max(0.0, 1 - p.sum())
                g = abs(np.log(rest) - ln_u[i]) if rest > 0 else 0.0
                d = rest_error(value[i]) + EPS * rest
                # each p (rounded to fp32) and its difference; the rest's logarithms
                tol[i] += 2 * EPS * np.sum(p * np.abs(value[i] + np.log(K))) + rest * (2.0 ** -28 + EPS * g) + d * (g + 1)
                tol[i] += 2 * EPS * np.sum(p * u[i])     # ln q = -ln K - u
        near(loss, want, tol)


@pytest.mark.parametrize("dtype", [W.F32, W.BF16])
@pytest.mark.parametrize("rest", [1e-2, 1e-4, 1e-5, 1e-6])
def test_sharp_targets(rest, dtype):
    """Nearly all on one token on both sides, the others' small shares a fifth apart: a loss of about rest / 50."""
    r = np.random.default_rng(42)
    T = 1.5
    for v, K, factor in ((500, 2, 1.2), (3001, 20, 0.8), (60000, 128, 1.2)):
        ref, t, token, value = sharp(r, 4, v, K, rest, factor, dtype, T, False)
        loss = ssv.distill(t, *on_gpu(token, value), T, ssv.REST)[0].cpu().numpy()
        for i in range(4):
            want, _, stats = odist.row_distill(ref[i], token[i], value[i].astype(np.float64), T, odist.REST)
            m, S, mo, So = stats
            t64 = value[i].astype(np.float64)
            p = np.exp(t64)
            logq = (ref[i, token[i]] - m) / T - np.log(S)
            little = np.exp(logq[1:]).sum()
            ln_u = odist.log_rest(stats, T)
            u, rr = np.exp(ln_u), max(0.0, 1 - p.sum())
            g = abs(np.log(rr) - ln_u)
            d = rest_error(value[i]) + EPS * rr
            lnS = np.log(S)
            tol = (2 * EPS * little + 2 * LN * u + 2 * EPS * lnS + 2.0 ** -44      # ln S, of 1 and a little
                   + 3 * EPS * np.sum(p * np.abs(t64 - logq))                      # p and its difference, each rounded
                   + rr * (2 * LN + 2.0 ** -29 + EPS * g) + d * (g + 1) + EPS * abs(want) + 2.0 ** -50)
            assert tol < 0.1 * want                                                # a test of the loss's own digits
            near(loss[i], want, tol)
