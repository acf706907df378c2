"""ssv_distill and ssv_distill_backward against the float64 oracle, and the gradient against differences.

Tolerances (logits_common: a sum is within 2^-16 of itself, a logarithm of one absolutely): a probability p_j takes an
exponential (2^-22), the sum of K of them and a division: below 2^-16 of itself; r = 1 - sum p is off by (K + 4) eps of 1.
  loss: each ln p - ln q is off by 2 LN and is multiplied by p; the rest by r; p's own error meets |ln p - ln q|
  gradient: q, and the share of the others, are within 2^-15 (2 LN) of themselves; p and r as above; the last rounding
is half a step of the type."""
import numpy as np
import pytest
import torch

from diffusion_speculative_verification_gb300 import ssv, workloads as W
import oracle.distill as odist
from gpu_common import ensure_built
from logits_common import EPS, LN, near, placed, store

pytestmark = pytest.mark.gpu

MODES = [ssv.RENORM, ssv.REST]


def setup_module():
    ensure_built()


def tolerances(ref, token, value, T, mode, w, grad_loss=None):
    """(loss [n], gradient [n, V] before its last rounding)."""
    n, v = ref.shape
    tl, tg = np.zeros(n), np.zeros((n, v))
    for i in range(n):
        loss, grad, stats = odist.row_distill(ref[i], token[i], value[i], T, mode, 1.0)
        if w[i] == 0 or not np.isfinite(stats[0]):
            continue
        ln_u = odist.log_rest(stats, T)
        logq = (ref[i] - stats[0]) / T - np.log(stats[1])
        p, listed, r = odist.target(token[i], value[i], mode, v)
        if ln_u == -np.inf and r < 2.0 ** -20:
            r = 0.0
        with np.errstate(divide="ignore", invalid="ignore"):
            gap = np.where(p > 0, np.abs(np.log(np.where(p > 0, p, 1)) - logq), 0.0)
            gap_r = abs(np.log(r) - ln_u) if r > 0 else 0.0
        dr = (token.shape[1] + 4) * 2 * EPS if mode == odist.REST else 0.0
        P = p.sum() + r
        with np.errstate(invalid="ignore"):
            tl[i] = abs(w[i]) * (2 * LN * P + LN * np.sum(np.where(p > 0, p * gap, 0)) + dr * (gap_r + 1))
        q = np.exp(logq)
        with np.errstate(over="ignore"):
            share = np.where(listed, 0.0, np.exp((ref[i] - stats[2]) / T) / stats[3]) if stats[3] > 0 else np.zeros(v)
        e = np.where(listed, 2 * LN * P * q + LN * p, share * (2 * LN * (P * np.exp(ln_u) + r) + dr) + dr * q)
        tg[i] = e * abs(w[i] / T) * (1 if grad_loss is None else abs(grad_loss[i]))
    return tl, tg


def half_step(want, dtype):
    return np.abs(want) * (2.0 ** -8 if dtype == W.BF16 else EPS) * (1 + 2.0 ** -6) + 2.0 ** -126


def make(r, n, v, K, T=1.0, absent=0.0):
    z = r.standard_normal((n, v)) * 2
    for i in range(n):
        z[i, r.integers(0, v, 5)] += r.exponential(4.0, 5)
    t = z + 0.7 * r.standard_normal((n, v))
    lp = t / T - np.log(np.exp(t / T).sum(1, keepdims=True))
    k = min(K, v)
    token = np.full((n, K), -1, np.int32)
    value = np.full((n, K), -np.inf, np.float32)
    token[:, :k] = np.argsort(-t, 1, kind="stable")[:, :k]
    value[:, :k] = np.take_along_axis(lp, token[:, :k].astype(np.int64), 1)
    token[r.random((n, K)) < absent] = -1
    return z, token, value


def check(z, token, value, dtype, mode, T=1.0, weight=None, lead=0, pad=0, grad_lead=None, grad_pad=None, in_place=False,
          grad_loss=None, code=ssv.SSV_OK):
    T = float(np.float32(T))                      # the call's T is fp32
    ref, t = store(z, dtype)
    n, v = ref.shape
    w = np.ones(n) if weight is None else np.asarray(weight, np.float32).astype(np.float64)
    f = lambda a, d=torch.float32: None if a is None else torch.tensor(np.asarray(a), dtype=d, device="cuda")  # noqa: E731
    tok, val, wt, gl = f(token, torch.int32), f(value), f(weight), f(grad_loss)
    seen = np.where((token >= 0) & (token < v), token, -1)
    value = np.asarray(value, np.float32)
    want = odist.distill_batch(ref, seen, value, T, mode, w)
    tl, tg = tolerances(ref, seen, value, T, mode, w)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def rows():
        return placed(t, lead, pad)

    def space():
        if grad_lead is None:
            return True, None
        return placed(torch.full_like(t, 5.0), grad_lead, grad_pad, 3.0)

    # the loss alone, with its statistics
    x, buf = rows()
    loss, stats, none = ssv.distill(x, tok, val, T, mode, wt, dev_status=status)
    assert none is None and ssv.get_status(status) == code
    _forward(loss, stats, want, tl)
    # loss and gradient
    g, gbuf = (x, buf) if in_place else space()
    loss, stats, grad = ssv.distill(x, tok, val, T, mode, wt, grad=g, dev_status=status)
    assert ssv.get_status(status) == code
    _forward(loss, stats, want, tl)
    near(grad.float().cpu().numpy(), want[1], tg + half_step(np.where(np.isfinite(want[1]), want[1], 0), dtype))
    _between(gbuf, grad)
    # backward from the statistics, which are the ones that the gradient above was formed from
    x, buf = rows()
    g, gbuf = (x, buf) if in_place else space()
    grad = ssv.distill_backward(x, tok, val, stats, gl, T, mode, wt, None if g is True else g, dev_status=status)
    assert ssv.get_status(status) == code
    up = np.ones((n, 1)) if grad_loss is None else np.asarray(grad_loss, np.float32).astype(np.float64)[:, None]
    up = np.where(w[:, None] == 0, 0.0, up)              # a row of weight 0 has the gradient 0, whatever comes from upstream
    near(grad.float().cpu().numpy(), want[1] * up, tg * np.abs(up) + half_step(want[1] * up, dtype))
    _between(gbuf, grad)


def _forward(loss, stats, want, tol):
    near(loss.cpu().numpy(), want[0], tol + EPS * np.abs(np.where(np.isfinite(want[0]), want[0], 0)))
    got = stats.cpu().numpy()
    near(got[:, ::2], want[2][:, ::2], 0)
    near(got[:, 1::2], want[2][:, 1::2], LN * want[2][:, 1::2])


def _between(buf, rows):
    """What is not a row of the gradient is as it was (3, or the NaN around the logits)."""
    if buf is None:
        return
    keep = torch.ones(buf.shape, dtype=torch.bool, device="cuda")
    keep.as_strided(rows.shape, rows.stride(), rows.storage_offset()).fill_(False)
    left = buf[keep]
    assert left.isnan().all() or (left == 3.0).all()


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("dtype", [W.F32, W.BF16])
@pytest.mark.parametrize("v", [1, 2, 7, 16, 17, 33, 256, 1001])
def test_small_vocabularies(v, dtype, mode):
    r = np.random.default_rng(v)
    for K in (1, 3, 40, 128):
        check(*make(r, 4, v, K), dtype, mode)


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("dtype", [W.F32, W.BF16])
@pytest.mark.parametrize("v,n,K", [(9001, 3, 32), (32003, 2, 128), (151936, 2, 64), (151937, 1, 1), (1 << 19, 1, 128)])
def test_large_vocabularies(v, n, K, dtype, mode):
    r = np.random.default_rng(v)
    check(*make(r, n, v, K, T=2.0, absent=0.1), dtype, mode, T=2.0)


@pytest.mark.parametrize("T", [0.3, 0.7, 1.1, 1.5, 3.0, 50.0])
def test_temperatures(T):
    """Scales that are rounded up and down, beside the -inf around a row and in it."""
    r = np.random.default_rng(33)
    for v in (50, 3001):
        z, token, value = make(r, 3, v, 9, T)
        z[1, v // 2] = -np.inf
        for dtype in (W.F32, W.BF16):
            check(z, token, value, dtype, ssv.REST, T=T, lead=3, pad=2)


@pytest.mark.parametrize("T", [1e30, 3e37])
def test_temperatures_near_the_largest(T):
    """Logits of the type's lowest number, about -11 on the scale of the larger T: what 1 / T has beyond 24 bits is next to
    fp32's smallest numbers there.  The weights bring loss and gradient back to its range."""
    r = np.random.default_rng(34)
    for v in (100, 3001):
        z, token, value = make(r, 3, v, 9)
        z[1][r.random(v) < 0.5] = -3.3895314e38
        z[2] = -3.3895314e38 * r.random(v)
        value = value - 1
        for dtype in (W.F32, W.BF16):
            for mode in MODES:
                check(z, token, value, dtype, mode, T=T, weight=[T / 8] * 3)


@pytest.mark.parametrize("n", [700, 1300])
def test_many_rows(n):
    r = np.random.default_rng(n)
    w = r.random(n) * (r.random(n) < 0.8)
    check(*make(r, n, 2000, 20), W.BF16, ssv.REST, weight=w, grad_loss=r.standard_normal(n))
    check(*make(r, n, 300, 128), W.F32, ssv.RENORM, weight=w)


@pytest.mark.parametrize("dtype", [W.F32, W.BF16])
@pytest.mark.parametrize("lead,pad,grad_lead,grad_pad", [(1, 0, 1, 0), (3, 1, 0, 0), (0, 5, 0, 5), (7, 9, 7, 25), (0, 0, 1, 0),
                                                         (15, 2, None, None), (0, 7, None, None)])
def test_strides_and_alignment(lead, pad, grad_lead, grad_pad, dtype):
    """Rows at every offset from a 32-byte boundary, the gradient's at the same and at other ones."""
    r = np.random.default_rng(lead * 31 + pad)
    for v in (1, 5, 40, 1001, 5000):
        check(*make(r, 4, v, 9), dtype, ssv.REST, lead=lead, pad=pad, grad_lead=grad_lead, grad_pad=grad_pad)


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("dtype", [W.F32, W.BF16])
def test_in_place(dtype, mode):
    r = np.random.default_rng(20)
    for v, n in ((40, 3), (5001, 4), (60000, 2)):
        check(*make(r, n, v, 100), dtype, mode, lead=3, pad=2, in_place=True)


def test_gradient_beside_the_logits():
    """Two halves of one wider buffer."""
    r = np.random.default_rng(21)
    z, token, value = make(r, 5, 64, 8)
    ref, t = store(z, W.F32)
    buf = torch.zeros((5, 160), device="cuda")
    buf[:, :64] = t
    a = [torch.tensor(token, device="cuda"), torch.tensor(value, device="cuda")]
    _, _, want = ssv.distill(t, *a, grad=True)
    ssv.distill(buf[:, :64], *a, grad=buf[:, 64:128])
    assert torch.equal(buf[:, 64:128], want) and torch.equal(buf[:, :64], t) and (buf[:, 128:] == 0).all()
    with pytest.raises(ssv.SsvError):
        ssv.distill(buf[:, :64], *a, grad=buf[:, 60:124])


def test_weights():
    """Rows of weight 0 are not read; others scale; negative ones too."""
    r = np.random.default_rng(22)
    z, token, value = make(r, 6, 3000, 16)
    z[1], z[4] = np.nan, np.nan
    check(z, token, value, W.F32, ssv.REST, weight=[0.5, 0, -2, 1e-6, 0, 3], grad_loss=[1, 5, -1, 2, np.nan, 0])
    check(z, token, value, W.BF16, ssv.RENORM, weight=[0.5, 0, -2, 1e-6, 0, 3])


@pytest.mark.parametrize("mode", MODES)
def test_listed_more_than_once(mode):
    r = np.random.default_rng(23)
    z, token, value = make(r, 4, 500, 40)
    token[:, 5] = token[:, 2]
    token[:, 39] = token[:, 2]
    token[1] = token[1, 0]
    value[:, 20] = value[:, 21]
    value -= np.log(4.0).astype(np.float32)      # every row's probabilities stay below 1
    check(z, token, value, W.F32, mode)


@pytest.mark.parametrize("dtype", [W.F32, W.BF16])
@pytest.mark.parametrize("K", [20, 128])
def test_long_parts(K, dtype):
    """Parts above 128 KB: blocks of 512 threads, apart from the logits and in place."""
    r = np.random.default_rng(K)
    for v, lead in (((1 << 19) - 3, 3), (1 << 19, 0)):
        check(*make(r, 1, v, K), dtype, ssv.REST, lead=lead, in_place=True)
        check(*make(r, 1, v, K), dtype, ssv.RENORM, lead=lead, grad_lead=5, grad_pad=2)


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("dtype", [W.F32, W.BF16])
@pytest.mark.parametrize("K", [64, 65, 96, 97, 127, 128])
def test_long_lists(K, dtype, mode):
    """Tokens that are listed far apart, more than once, and absent ones among them, in rows of one and of several CTAs."""
    r = np.random.default_rng(K)
    for v in (300, 3001, 60000):
        z, token, value = make(r, 4, v, K)
        token[0, K - 1] = token[0, 0]
        token[0, 33:60] = token[0, 1]
        token[1, K // 2:] = token[1, :K - K // 2]
        token[2, r.random(K) < 0.5] = -1
        token[3] = token[3, 63]
        value -= np.log(8.0 if mode == ssv.RENORM else 2.0 * K).astype(np.float32)
        check(z, token, value, dtype, mode, lead=1)


@pytest.mark.parametrize("mode", MODES)
def test_absent_and_refused_tokens(mode):
    r = np.random.default_rng(24)
    z, token, value = make(r, 5, 200, 12)
    token[0] = -1
    token[1, 3:] = -1
    value[2, :6] = -np.inf
    value[3] = -np.inf
    check(z, token, value, W.F32, mode)
    for bad in (200, -2, 1 << 30, -(1 << 31)):
        t = token.copy()
        t[4, 2] = bad
        check(z, t, value, W.F32, mode, code=ssv.SSV_ERR_INVALID)


@pytest.mark.parametrize("mode", MODES)
def test_every_token_listed(mode):
    """No other tokens: nothing is left for them on either side."""
    r = np.random.default_rng(25)
    z, token, value = make(r, 4, 60, 128)
    check(z, token, value, W.F32, mode)
    value[:, :60] -= 0.5                          # the target leaves a share to tokens that are not there
    loss, stats, grad = ssv.distill(store(z, W.F32)[1], torch.tensor(token, device="cuda"), torch.tensor(value, device="cuda"),
                                    mode=mode, grad=True)
    assert (stats[:, 2] == -np.inf).all() and (stats[:, 3] == 0).all() and grad.isfinite().all()
    assert (loss == np.inf).all() if mode == ssv.REST else loss.isfinite().all()


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("dtype", [W.F32, W.BF16])
def test_masked_drafter(dtype, mode):
    """-inf and the type's lowest number in the drafter's logits; rows of which nothing is left."""
    r = np.random.default_rng(26)
    for v in (100, 20000):
        z, token, value = make(r, 7, v, 10)
        others = np.ones((7, v), bool)
        np.put_along_axis(others, token.astype(np.int64), False, 1)
        z[0][others[0] & (r.random(v) < 0.9)] = -np.inf
        z[1][others[1]] = -np.inf                # only listed tokens are left
        z[2, token[2, 3]] = -np.inf              # a listed token that cannot be
        z[3] = -np.inf
        z[4][others[4] & (r.random(v) < 0.9)] = -3.3895314e38
        z[5] = -3.3895314e38
        z[6] = -np.inf
        z[6, token[6]] = 0.0
        check(z, token, value, dtype, mode)


def test_rest_of_little_and_of_nearly_all():
    """The others' share far below what 1 - (listed) could hold, and nearly 1."""
    r = np.random.default_rng(27)
    z, token, value = make(r, 4, 5000, 8)
    z = z - 10
    np.put_along_axis(z[:2], token[:2].astype(np.int64), 40.0 + r.random((2, 8)), 1)   # u about e^-45
    np.put_along_axis(z[2:], token[2:].astype(np.int64), -30.0, 1)
    value[0] = np.log(0.1)
    value[1] = np.log(0.125) + np.float32(1e-7)
    check(z, token, value, W.F32, ssv.REST)


def test_not_finite():
    r = np.random.default_rng(28)
    z, token, value = make(r, 5, 900, 6)
    z[0, 3], z[1, token[1, 0]], z[2, 5] = np.nan, np.nan, np.inf
    value[3, 2] = np.nan
    a = [torch.tensor(token, device="cuda"), torch.tensor(value, device="cuda")]
    for dtype in (W.F32, W.BF16):
        t = store(z, dtype)[1]
        for mode in MODES:
            loss, stats, grad = ssv.distill(t, *a, mode=mode, grad=True)
            back = ssv.distill_backward(t, *a, stats, mode=mode)
            assert loss[:4].isnan().all() and loss[4].isfinite()
            for g in (grad, back):
                assert g[:3].isnan().all() and g[3].isnan().any() and g[4].isfinite().all()


@pytest.mark.parametrize("mode", MODES)
def test_gradient_against_differences(mode):
    """A central difference of the summed losses, in steps h of single logits: the loss is within its tolerance t, so the
    difference is within t / h; its second-order term is h^2 / 6 times a third derivative below 2 / T^3."""
    r = np.random.default_rng(29)
    T = float(np.float32(0.9))
    z, token, value = make(r, 3, 50, 7, T)
    a = [torch.tensor(token, device="cuda"), torch.tensor(value, device="cuda")]
    ref, t = store(z, W.F32)
    _, stats, grad = ssv.distill(t, *a, T, mode, grad=True)
    tl, _ = tolerances(ref, token, value.astype(np.float64), T, mode, np.ones(3))
    h = 2.0 ** -4
    for i in range(3):
        both = []
        for s in (h, -h):
            x = t[i].repeat(50, 1) + s * torch.eye(50, device="cuda")
            both.append(ssv.distill(x, a[0][i:i + 1].repeat(50, 1), a[1][i:i + 1].repeat(50, 1), T, mode)[0])
        d = ((both[0].double() - both[1].double()) / (2 * h)).cpu().numpy()
        near(grad[i].cpu().numpy(), d, 2 * tl[i] / h + h * h / 3 / T ** 3)


def test_long_offsets():
    """Rows, of logits and gradient, that start beyond 2^31 elements."""
    r = np.random.default_rng(30)
    z, token, value = make(r, 3, 2000, 10)
    ref, t = store(z, W.BF16)
    stride = 1 << 30
    buf = torch.empty(2 * stride + 2000, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((3, 2000), (stride, 1), 0)
    for i in range(3):
        x[i] = t[i]
    a = [torch.tensor(token, device="cuda"), torch.tensor(value, device="cuda")]
    loss, stats, want = ssv.distill(t, *a, grad=True)
    got = ssv.distill(x, *a, grad=x)
    assert torch.equal(got[0], loss) and all(torch.equal(x[i], want[i]) for i in range(3))


def test_graph_on_a_side_stream():
    """A captured step, replayed over new logits."""
    r = np.random.default_rng(31)
    data = [make(r, 6, 20000, 32) for _ in range(2)]
    t = [store(d[0], W.BF16)[1] for d in data]
    a = [torch.tensor(data[0][1], device="cuda"), torch.tensor(data[0][2], device="cuda")]
    want = []
    for x in t:
        loss, stats, grad = ssv.distill(x, *a, mode=ssv.REST, grad=True)
        want.append((loss, stats, grad, ssv.distill_backward(x, *a, stats, loss, mode=ssv.REST)))
    x = torch.zeros_like(t[0])
    out = [torch.zeros_like(y) for y in want[0]]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=torch.cuda.Stream()):
        ssv.distill(x, *a, mode=ssv.REST, grad=out[2], loss=out[0], stats=out[1])
        ssv.distill_backward(x, *a, out[1], out[0], mode=ssv.REST, grad=out[3])
    for k in (0, 1, 0):
        x.copy_(t[k])
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, want[k]))


def test_empty():
    e = torch.empty
    t, v = e((0, 4), dtype=torch.int32, device="cuda"), e((0, 4), device="cuda")
    loss, stats, grad = ssv.distill(e((0, 50), device="cuda"), t, v, grad=True)
    assert loss.shape == (0,) and stats.shape == (0, 4) and grad.shape == (0, 50)
    assert ssv.distill_backward(e((0, 50), device="cuda"), t, v, stats).shape == (0, 50)
