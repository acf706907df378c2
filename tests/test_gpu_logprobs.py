"""ssv_logprobs against the float64 oracle (tolerances: logits_common)."""
import numpy as np
import pytest
import torch

from diffusion_speculative_verification_gb300 import ssv, workloads as W
import oracle.logprobs as olp
from gpu_common import ensure_built
from logits_common import EPS, LN, near, placed, store

pytestmark = pytest.mark.gpu


def setup_module():
    ensure_built()


def check(x, dtype, tokens=None, rows=None, top_k=0, T=1.0, lead=0, pad=0, code=ssv.SSV_OK):
    """x [rows, V] float; tokens and rows as the call gets them (entries that it has to refuse: -2 in `code` cases)."""
    T = float(np.float32(T))                      # the call's T is fp32
    ref, t = store(x, dtype)
    t, buf = placed(t, lead, pad)
    was = buf.clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dev = lambda a: None if a is None else torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")  # noqa: E731
    got = ssv.logprobs(t, dev(tokens), top_k, T, dev(rows), dev_status=status)
    assert ssv.get_status(status) == code
    assert torch.equal(buf.view(torch.uint8), was.view(torch.uint8))
    v = x.shape[1]
    if code != ssv.SSV_OK:     # refused entries are idle
        tokens = [-1 if not -1 <= a < v else a for a in tokens]
        rows = None if rows is None else [-1 if not -1 <= a < len(x) else a for a in rows]
    want = olp.logprobs_batch(ref, tokens, rows, top_k, T)
    names = ("logprob", "rank", "entropy", "lse", "top_logprob", "top_token")
    g = {k: None if a is None else a.cpu().numpy() for k, a in zip(names, got)}
    near(g["lse"], want["lse"], LN + EPS * np.abs(want["lse"]))
    # ln S - W / S: the sum W is off by 2^-16 of itself as well
    near(g["entropy"], want["entropy"], 2 * LN * (1 + np.abs(want["entropy"])))
    if tokens is None:
        assert g["logprob"] is None and g["rank"] is None
    else:
        near(g["logprob"], want["logprob"], LN + EPS * np.abs(want["logprob"]))
        assert np.array_equal(g["rank"], want["rank"])
    if top_k:
        assert np.array_equal(g["top_token"], want["top_token"])
        near(g["top_logprob"], want["top_logprob"], LN + 4 * EPS * np.abs(want["top_logprob"]))
    else:
        assert g["top_token"] is None and g["top_logprob"] is None
    return got


def spread(r, n, v):
    """Logits with a few tokens that stand out."""
    x = r.standard_normal((n, v)) * 2
    for i in range(n):
        x[i, r.integers(0, v, 6)] += r.exponential(4.0, 6)
    return x


@pytest.mark.parametrize("dtype", [W.F32, W.BF16])
@pytest.mark.parametrize("v", [1, 2, 7, 8, 9, 16, 17, 31, 33, 63, 256, 257, 1000])
def test_small_vocabularies(v, dtype):
    r = np.random.default_rng(v)
    for top_k in (0, 1, 5, 128):
        check(spread(r, 5, v), dtype, r.integers(0, v, 5), top_k=top_k)


@pytest.mark.parametrize("dtype", [W.F32, W.BF16])
@pytest.mark.parametrize("v,n", [(9001, 3), (32003, 2), (151936, 2), (151937, 1), (40000, 130)])
@pytest.mark.parametrize("top_k", [0, 20, 128])
def test_large_vocabularies(v, n, top_k, dtype):
    r = np.random.default_rng(v + n)
    check(spread(r, n, v), dtype, r.integers(0, v, n), top_k=top_k, T=0.8)


def test_largest_vocabulary():
    r = np.random.default_rng(5)
    for dtype in (W.F32, W.BF16):
        check(spread(r, 1, 1 << 19), dtype, [12345], top_k=128)


@pytest.mark.parametrize("n", [700, 1300])
def test_many_rows(n):
    """One CTA per row, or two."""
    r = np.random.default_rng(n)
    check(spread(r, n, 3000), W.BF16, r.integers(0, 3000, n), top_k=10)
    check(spread(r, n, 500), W.F32, r.integers(0, 500, n), top_k=64)


@pytest.mark.parametrize("dtype", [W.F32, W.BF16])
@pytest.mark.parametrize("lead,pad", [(1, 0), (3, 1), (0, 5), (7, 9), (16, 16), (15, 2)])
def test_strides_and_alignment(lead, pad, dtype):
    """Rows at every offset from a 32-byte boundary, NaN in front of, between and behind them."""
    r = np.random.default_rng(lead * 31 + pad)
    for v in (1, 5, 40, 1001, 5000):
        check(spread(r, 4, v), dtype, r.integers(0, v, 4), top_k=7, lead=lead, pad=pad)


@pytest.mark.parametrize("T", [1e-3, 0.3, 1.5, 100.0, 1e30])
def test_temperatures(T):
    """A logarithm of a sum, times nothing; l_t / T of 2000 at T = 1e-3 rounds by 2^-24 of it."""
    r = np.random.default_rng(6)
    check(spread(r, 3, 700), W.F32, [3, 500, 699], top_k=12, T=T)


def test_rows_and_idle_entries():
    r = np.random.default_rng(7)
    x = spread(r, 6, 300)
    check(x, W.BF16, [4, -1, 299, 0, 5, 17, 9], rows=[5, 0, 0, -1, 2, 2, 2], top_k=6)
    check(x, W.BF16, [4, -1, 299], top_k=6)
    check(x, W.F32, None, rows=[3, 3, -1], top_k=4)
    check(x, W.F32, None, top_k=4)
    check(x, W.F32, None)
    check(x[:0], W.F32, [], top_k=3)


def test_refused_entries():
    r = np.random.default_rng(8)
    x = spread(r, 3, 50)
    for tokens, rows in (([50, 1], [0, 1]), ([-2, 1], [0, 1]), ([1 << 30, 1], [0, 1]), ([3, 1], [3, 1]),
                         ([3, 1], [-2, 1]), ([3, 1], [-(1 << 31), 0]), ([50, -1], [7, -1])):
        check(x, W.F32, tokens, rows=rows, top_k=3, code=ssv.SSV_ERR_INVALID)


@pytest.mark.parametrize("dtype", [W.F32, W.BF16])
def test_masked_tokens(dtype):
    """-inf, the type's lowest number, rows with one token left and with none."""
    r = np.random.default_rng(9)
    for v in (40, 3001, 70000):
        x = spread(r, 8, v)
        x[0, r.random(v) < 0.95] = -np.inf
        x[1] = -np.inf
        x[2] = -np.inf
        x[2, v // 3] = -4.0
        low = -3.3895314e38                       # bf16's lowest, a number of fp32 too
        x[3, r.random(v) < 0.9] = low
        x[4] = low
        x[5, : v - 1] = -np.inf
        x[6, 1:] = -np.inf
        x[7] = -np.inf
        x[7, ::5] = low
        tok = r.integers(0, v, 8)
        check(x, dtype, tok, top_k=9)
        check(x, dtype, np.full(8, v // 3), top_k=128, T=0.5)


@pytest.mark.parametrize("dtype", [W.F32, W.BF16])
def test_equal_logits(dtype):
    """Ties go to the lowest index, also where far more elements are equal than a list holds."""
    r = np.random.default_rng(10)
    for v in (30, 700, 9000, 60000):
        x = np.zeros((6, v))
        x[1] = r.integers(0, 2, v)
        x[2] = r.integers(0, 6, v)
        x[3, ::3] = -0.0
        x[4] = -1.5
        x[4, v - 3:] = 2.0
        x[5] = np.floor(r.standard_normal(v) * 4) / 4
        for top_k in (1, 20, 128):
            check(x, dtype, r.integers(0, v, 6), top_k=top_k)


def test_sorted_logits():
    """The greatest elements next to one another, in one part of the row."""
    v = 50000
    x = np.stack([np.linspace(-9, 9, v), np.linspace(9, -9, v), np.roll(np.linspace(-9, 9, v), 777)])
    for dtype in (W.F32, W.BF16):
        check(x, dtype, [0, v - 1, 40], top_k=128)
        check(x, dtype, [0, v - 1, 40], top_k=17)


@pytest.mark.parametrize("dtype", [W.F32, W.BF16])
def test_not_finite(dtype):
    r = np.random.default_rng(11)
    for v in (20, 4000):
        x = spread(r, 6, v)
        x[0, 3] = np.nan
        x[1, v - 1] = np.inf
        x[2] = np.nan
        x[3] = -np.inf
        x[3, 7] = np.nan
        x[4, 2], x[4, 9] = np.inf, np.nan
        check(x, dtype, [3, v - 1, 0, 7, 1, 5], top_k=11)


def test_certain_rows():
    """One token of nearly all the probability, one of all of it."""
    x = np.zeros((2, 1000))
    x[0, 5], x[1, 6] = 12.0, 300.0
    check(x, W.F32, [5, 6], top_k=3)
    check(x, W.F32, [0, 0], top_k=3)


@pytest.mark.parametrize("dtype", [W.F32, W.BF16])
@pytest.mark.parametrize("v", [3, 60, 700, 9001, 100000])
def test_nearly_certain_rows(v, dtype):
    """One token of nearly all the probability: what the others have, not what is left of 1.  Each of their terms is within
    3 eps |y| ln 2 + 2^-22 of itself (|y| < 30), their sum within 2^-16 with the additions (logits_common), and so are
    entropy, its two parts both of that sum, and the log-probability of the token, relatively."""
    r = np.random.default_rng(v)
    x = r.standard_normal((12, v)) * 0.5
    top = r.integers(0, v, 12)
    x[np.arange(12), top] = np.linspace(5, 19, 12) + np.log(v)
    x[5, (top[5] + 1) % v] = x[5, top[5]] - 4.0
    ref, t = store(x, dtype)
    tok = torch.tensor(top, dtype=torch.int32, device="cuda")
    lp, rank, ent, lse, tl, tt = (o.cpu().numpy().astype(np.float64) for o in ssv.logprobs(t, tok, 2))
    for i in range(12):
        y = ref[i] - ref[i].max()
        rest = np.exp(np.delete(y, top[i]))
        small = rest.sum()
        want = np.log1p(small)
        h = want - (rest * np.delete(y, top[i])).sum() / (1 + small)
        assert abs(lp[i] + want) <= LN * want and abs(tl[i, 0] + want) <= LN * want
        assert abs(ent[i] - h) <= 2 * LN * h and rank[i] == 1 and tt[i, 0] == top[i]


def test_long_offsets():
    """A row that starts beyond 2^31 elements."""
    r = np.random.default_rng(12)
    v, stride = 2000, 1 << 30
    buf = torch.empty(2 * stride + v + 8, dtype=torch.bfloat16, device="cuda")
    t = buf.as_strided((3, v), (stride, 1), 0)
    ref, x = store(spread(r, 3, v), W.BF16)
    for i in range(3):
        t[i] = x[i]
    lp, rank, ent, lse, tl, tt = ssv.logprobs(t, torch.tensor([1, 2, 3], dtype=torch.int32, device="cuda"), 5)
    want = olp.logprobs_batch(ref, [1, 2, 3], None, 5, 1.0)
    near(lp.cpu().numpy(), want["logprob"], LN + EPS * np.abs(want["logprob"]))
    assert np.array_equal(tt.cpu().numpy(), want["top_token"]) and np.array_equal(rank.cpu().numpy(), want["rank"])


@pytest.mark.parametrize("dtype", [W.F32, W.BF16])
def test_zeros_and_subnormal_logits(dtype):
    """The order of numbers next to 0, of both signs: zeros are equal, subnormal numbers are not zeros."""
    r = np.random.default_rng(17)
    near_zero = np.array([0.0, -0.0] + [s * 2.0 ** e for s in (1, -1) for e in (-133, -132, -130, -127, -126, -120)])
    for v, top_k in ((40, 20), (900, 128), (20000, 64)):
        x = near_zero[r.integers(0, len(near_zero), (8, v))]
        x[4:] -= (r.random((4, v)) < 0.98) * r.integers(1, 50, (4, v))   # few of them among others, below
        t = r.integers(0, v, 8)
        t[6:] = x[6:].argmax(1)
        check(x, dtype, t, top_k=top_k)


def test_given_outputs_and_repeats():
    r = np.random.default_rng(13)
    _, t = store(spread(r, 9, 20000), W.BF16)
    tok = torch.tensor(r.integers(0, 20000, 9), dtype=torch.int32, device="cuda")
    first = ssv.logprobs(t, tok, 30)
    out = tuple(torch.full_like(x, 7) for x in first)
    assert ssv.logprobs(t, tok, 30, out=out)[4] is out[4]
    for a, b in zip(first, out):
        assert torch.equal(a, b)
    assert ssv.logprobs(t, tok, 30, out=list(out))[5] is out[5]
    with pytest.raises(ssv.SsvError):
        ssv.logprobs(t, tok, 30, out=out[:4])
    only = (out[0].fill_(0), None, None, None, None, None)
    ssv.logprobs(t, tok, out=only)
    assert torch.equal(out[0], first[0])


def test_graph_on_a_side_stream():
    r = np.random.default_rng(14)
    _, t = store(spread(r, 12, 30000), W.BF16)
    tok = torch.tensor(r.integers(0, 30000, 12), dtype=torch.int32, device="cuda")
    want = ssv.logprobs(t, tok, 20)
    out = tuple(torch.zeros_like(x) for x in want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=torch.cuda.Stream()):
        ssv.logprobs(t, tok, 20, out=out)
    for _ in range(2):
        for x in out:
            x.zero_()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, out):
            assert torch.equal(a, b)


def test_two_streams_at_once():
    r = np.random.default_rng(15)
    data = [store(spread(r, n, 40000), W.BF16)[1] for n in (40, 7)]
    want = [ssv.logprobs(t, None, 20) for t in data]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in data]
    got = [[ssv.logprobs(t, None, 20, stream=s) for _ in range(20)] for t, s in zip(data, streams)]
    torch.cuda.synchronize()
    for w, many in zip(want, got):
        for o in many:
            assert all(torch.equal(a, b) for a, b in zip(w[2:], o[2:]))
