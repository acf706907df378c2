"""Inputs and tolerances of the logits operators' GPU tests.

Tolerances, derived before any run, eps = 2^-24 half a step of fp32.  An exponent's argument (l - m) log2(e) / T takes
three roundings, so a term 2^y is off by 3 ln(2) |y| eps and the exponential's own 2^-22; weighted by the terms, |y| ln 2
is at most the row's entropy, below ln V <= 13.2.  A thread adds at most V / (32 threads * 1) terms in pairs and
batches; for the sizes here (at most 2400 terms per accumulator, growing sums) and the joins (warp, CTA, cluster) the
relative error of a sum of positive terms is below (number of additions in a row) eps <= 160 eps with the batches of 32
and 75 batches.  In all a sum is within (40 + 4 + 160) eps < 2^-16 of itself, and so is a logarithm of a sum, absolutely.
Rounding a result v adds eps |v|; alternatives are formed in fp32, three roundings of parts no larger than it."""
import numpy as np
import torch

from diffusion_speculative_verification_gb300 import workloads as W

LN = 2.0 ** -16      # a logarithm of a sum, absolutely; a sum, relatively
EPS = 2.0 ** -24


def store(x, dtype):
    """(tensor values as float64, torch tensor on the GPU) of x rounded to dtype."""
    t = torch.from_numpy(np.ascontiguousarray(x, np.float32))
    t = t.bfloat16() if dtype == W.BF16 else t
    return t.double().numpy(), t.cuda()


def placed(t, lead, pad, fill=float("nan")):
    """t's rows inside a wider buffer: `lead` elements before the first, `pad` between rows; the rest holds `fill`."""
    n, v = t.shape
    buf = torch.full((lead + max(n, 1) * (v + pad),), fill, dtype=t.dtype, device=t.device)
    out = buf[lead:].as_strided((n, v), (v + pad, 1), lead)
    out.copy_(t)
    return out, buf


def near(got, want, tol):
    """got within tol of want, infinities and NaN in the same places (a value beyond fp32's range is infinite in fp32)."""
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        want = np.where(np.isinf(want.astype(np.float32)), want.astype(np.float32), want)
    odd = ~np.isfinite(want)
    assert np.array_equal(got[odd], want[odd], equal_nan=True), (got[odd][:5], want[odd][:5])
    with np.errstate(invalid="ignore"):
        d = np.where(odd, 0.0, np.abs(got - want)) - np.where(odd, 0.0, np.broadcast_to(tol, want.shape))
    assert np.isfinite(got[~odd]).all() and (d <= 0).all(), (float(d.max()), np.unravel_index(d.argmax(), d.shape))
