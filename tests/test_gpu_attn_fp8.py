"""ssv_verify_attn_fp8 against the float64 oracle on the same codes.

Tolerance per output element, before any run.  With weights w_j (their sum is
1), A = sum_j w_j |v_j| and S = scale * max_j sum_i |q_i k_ji|:
  * the output rounds to bf16: 2^-8 |o|; what it is merged from may have been
    rounded to bf16 once before: again 2^-8 of a part that A bounds;
  * each weight may be rounded to 16 bits (bf16: 2^-8) before it meets v, and
    the sum it is divided by is not: 2^-8 A;
  * a score is off by the fp32 accumulation of d = 128 products and by the
    query's split (2^-17 of the row's largest element per element): 2^-15 S,
    and moves o by at most twice that times A.
In all 2^-8 |o| + (2^-7 + 2^-14 S) A."""
import numpy as np
import pytest
import torch

from diffusion_speculative_verification_gb300 import ssv, io as sio, workloads as W
import oracle.attention as oattn
import oracle.mask as omask
from gpu_common import ensure_built
from paged_common import PagedBatch

pytestmark = pytest.mark.gpu


def setup_module():
    ensure_built()


def call(t, out=None, **kw):
    return ssv.verify_attn_fp8(t["q"], t["k_cache"], t["v_cache"], t["k_scale"], t["v_scale"], t["pages"], t["k_new"],
                               t["v_new"], t["batch"], t["tau"], out=out, **kw)


def reference(x, scale=None):
    """(o, tolerance) float64 [rows, Hq, d]; NaN rows where a record is idle."""
    kc, vc, seqs = x.caches()
    q, kn, vn = x.values(x.q), x.values(x.k_new), x.values(x.v_new)
    G = x.Hq // x.Hkv
    sc = 1 / np.sqrt(x.d) if scale is None else scale
    o = np.full((x.rows, x.Hq, x.d), np.nan)
    tol = np.full_like(o, np.nan)
    for b in x.live():
        C, N, B, off, _, t_off = (int(v) for v in seqs[b])
        see = omask.verify_mask(C, N, B, x.tau[t_off:t_off + B])
        for g in range(x.Hkv):
            k, v = oattn.sequence_keys(seqs[b], kc, vc, kn, vn, g)
            for h in range(g * G, g * G + G):
                qh = q[off:off + N + 2 * B, h]
                ref = oattn.masked_softmax_attention(qh, k, v, see, sc)
                a = oattn.masked_softmax_attention(qh, k, np.abs(v), see, sc)
                s = sc * ((np.abs(qh) @ np.abs(k).T) * see).max(1, keepdims=True)
                o[off:off + len(qh), h] = ref
                tol[off:off + len(qh), h] = 2.0 ** -8 * np.abs(ref) + (2.0 ** -7 + 2.0 ** -14 * s) * a + 1e-30
    return o, tol


def check(x, strided=False, scale=None, status_code=ssv.SSV_OK, t=None):
    t = x.device(strided) if t is None else t
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((x.q.shape[0], x.Hq, x.d), 3.0, dtype=torch.bfloat16, device="cuda")
    call(t, out, dev_status=status, **({} if scale is None else dict(scale=scale)))
    assert ssv.get_status(status) == status_code
    o, tol = reference(x, scale)
    got = out.double().cpu().numpy()
    live = ~np.isnan(o)
    err = np.abs(got[:x.rows] - o)
    assert np.isfinite(got[:x.rows][live]).all()
    assert (err[live] <= tol[live]).all(), float((err[live] / tol[live]).max())
    assert (got[:x.rows][~live] == 3.0).all() and (got[x.rows:] == 3.0).all()   # rows of no sequence are not touched
    return got


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 2), (7, 1), (16, 1), (10, 2)])
def test_parity_over_lengths(hq, hkv, page):
    """Cached lengths around pages and key blocks, none at all, one token."""
    check(PagedBatch([0, 1, page - 1, page, page + 1, 127, 128, 129, 400], [0, 0, 1, 0, 5, 0, 1, 0, 2],
                     [1, 3, 8, 4, 2, 5, 16, 7, 9], hq, hkv, 128, page, seed=hq * page, pad=4), strided=page == 32)


@pytest.mark.parametrize("blocks", [[64, 33], [1, 1], [32, 16]])
@pytest.mark.parametrize("G", [1, 4, 5, 8, 128])
def test_row_tiles(blocks, G):
    """One to many tiles of packed query rows."""
    check(PagedBatch([300, 37], [0, 1], blocks, G, 1, 128, 64, seed=G + blocks[0]))


def test_prompt_chunks():
    check(PagedBatch([0, 260, 50], [300, 130, 1], [4, 9, 2], 4, 2, 128, 32, seed=3), strided=True)
    check(PagedBatch([150], [513], [16], 2, 1, 128, 16, seed=4))


def test_long_cache_split_over_ctas():
    """Few sequences, many key blocks: their parts are merged."""
    check(PagedBatch([9001, 40], [1, 0], [4, 2], 2, 1, 128, 16, seed=5))
    check(PagedBatch([6000], [0], [40], 4, 1, 128, 128, seed=6))


def test_many_sequences():
    r = np.random.default_rng(7)
    n = 300
    check(PagedBatch(r.integers(0, 200, n), r.integers(0, 2, n), r.integers(1, 9, n), 4, 2, 128, 16, seed=8,
                     idle=(0, 5, 299), pad=9))


@pytest.mark.parametrize("spread", [0, 9, 20])
def test_page_scales_far_apart(spread):
    check(PagedBatch([500, 130], [0, 3], [8, 4], 4, 1, 128, 16, seed=9 + spread, spread=spread))


def test_query_magnitudes_and_scale():
    """Sharp and flat softmax, rows of very different size, an explicit scale."""
    check(PagedBatch([700, 20], [1, 0], [8, 5], 4, 1, 128, 64, seed=30, qstd=6.0))
    check(PagedBatch([700, 20], [1, 0], [8, 5], 4, 1, 128, 64, seed=31, qstd=2.0 ** -20))
    x = PagedBatch([700, 20], [1, 0], [8, 5], 4, 1, 128, 64, seed=32)
    f = 2.0 ** np.random.default_rng(1).integers(-30, 3, (x.rows, 4, 1))
    x.q = W.f32_to_bf16_bits((W.bf16_bits_to_f32(x.q) * f).astype(np.float32))
    x.q[3, 1] = 0
    check(x)
    check(x, scale=0.03)


def test_running_maximum_grows_late():
    """The largest scores sit in the last keys, by far."""
    x = PagedBatch([900], [0], [4], 2, 1, 128, 64, seed=33)
    q = W.bf16_bits_to_f32(x.q)
    for j in range(12, 15):     # pages 12..14 hold keys along the mean query, ever longer
        p = x.table[0, j]
        d = q.mean((0, 1)) + 0.0
        k = np.tile(d / np.abs(d).max() * 2.0 ** (j - 11), (64, 1))
        x.scale[0][p, 0] = 2.0 ** -4
        import oracle.paged as opaged
        x.codes[0][p, 0] = opaged.e4m3_codes(np.clip(k / 2.0 ** -4, -448, 448))
    x.codes[0][x.table[0, 14], 0, 900 - 14 * 64:] = 0x7F
    check(x)


def test_pages_beyond_32_bit_offsets():
    """A pool of more than 2^31 codes, its pages in use at the far end."""
    x = PagedBatch([200, 90], [0, 1], [4, 8], 4, 8 // 2, 128, 128, seed=34)
    n = (1 << 31) // (4 * 128 * 128) + 64
    t = x.device()
    shift = n - x.n_pages
    for c in "kv":
        pool = torch.empty((n, 4, 128, 128), dtype=torch.uint8, device="cuda")
        pool[:64].fill_(0x7F)
        pool[shift:] = t[c + "_cache"]
        sc = torch.full((n, 4), float("nan"), device="cuda")
        sc[shift:] = t[c + "_scale"]
        t[c + "_cache"], t[c + "_scale"] = pool, sc
    t["pages"] += shift
    check(x, t=t)


def test_workspace_reuse_and_determinism():
    """The same workspace over calls of other sizes; equal inputs give equal bits."""
    a = PagedBatch([3000, 1], [0, 0], [8, 2], 4, 2, 128, 64, seed=35)
    b = PagedBatch([100, 700, 60], [1, 0, 40], [8, 2, 30], 4, 2, 128, 64, seed=36)
    ta, tb = a.device(), b.device()
    need = [ssv.verify_attn_fp8_workspace(t["q"], t["k_cache"], t["v_cache"], t["k_scale"], t["v_scale"], t["pages"],
                                          t["k_new"], t["v_new"], t["batch"], t["tau"]).numel() for t in (ta, tb)]
    ws = torch.zeros(max(need), dtype=torch.uint8, device="cuda")
    first = [call(t, workspace=ws).clone() for t in (ta, tb)]
    for _ in range(5):
        for t, want in ((tb, first[1]), (ta, first[0])):
            assert torch.equal(call(t, workspace=ws), want)


def test_graphs_that_share_a_workspace():
    a = PagedBatch([3000, 1], [0, 0], [8, 2], 4, 2, 128, 64, seed=37)
    b = PagedBatch([100, 700], [1, 0], [8, 2], 4, 2, 128, 64, seed=38)
    ts = [a.device(), b.device()]
    want = [call(t).clone() for t in ts]
    size = max(ssv.verify_attn_fp8_workspace(t["q"], t["k_cache"], t["v_cache"], t["k_scale"], t["v_scale"],
                                             t["pages"], t["k_new"], t["v_new"], t["batch"], t["tau"]).numel()
               for t in ts)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    outs, graphs = [torch.zeros_like(w) for w in want], []
    for t, o in zip(ts, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(t, o, workspace=ws)
        graphs.append(g)
    for _ in range(4):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))


def test_two_streams_with_workspaces_of_their_own():
    xs = [PagedBatch([2000, 300], [0, 1], [8, 16], 4, 2, 128, 64, seed=39 + i) for i in range(2)]
    ts = [x.device() for x in xs]
    want = [call(t).clone() for t in ts]
    wss = [ssv.verify_attn_fp8_workspace(t["q"], t["k_cache"], t["v_cache"], t["k_scale"], t["v_scale"], t["pages"],
                                         t["k_new"], t["v_new"], t["batch"], t["tau"]) for t in ts]
    outs = [torch.zeros_like(w) for w in want]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ts]
    for _ in range(10):
        for t, ws, o, s in zip(ts, wss, outs, streams):
            call(t, o, workspace=ws, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))


def test_refused_sequences():
    """A sequence outside its buffers, or with a bad page, is reported; the others are computed."""
    x = PagedBatch([200, 90, 40], [0, 2, 1], [4, 8, 3], 4, 2, 128, 16, seed=50)
    o, tol = reference(x)
    lo, hi = int(x.seqs[1, 3]), int(x.seqs[2, 3])
    others = np.r_[0:lo, hi:x.rows]

    def broken(code, seqs=None, table=None, tau=None):
        t = x.device()
        if seqs is not None:
            t["batch"].dev.copy_(sio.int_tensor(seqs, "cuda"))
        if table is not None:
            t["pages"].copy_(sio.int_tensor(table, "cuda"))
        if tau is not None:
            t["tau"].copy_(sio.int_tensor(tau, "cuda"))
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = call(t, dev_status=status).double().cpu().numpy()
        assert ssv.get_status(status) == code
        assert (np.abs(got[others] - o[others]) <= tol[others]).all()

    for bad in (-1, x.n_pages, 0x7FFFFFFF, -2147483648):
        table = x.table.copy()
        table[1, 3] = bad
        broken(ssv.SSV_ERR_INVALID, table=table)
    for field, value in ((0, -1), (0, 201), (1, -1), (1, 3), (2, 0), (2, 9), (2, 65), (4, -1), (4, 10 ** 6), (5, -1),
                         (5, 14)):
        s = x.seqs.copy()
        s[1, field] = value
        broken(ssv.SSV_ERR_INVALID, seqs=s)
    tau = x.tau.copy()
    tau[4:12] = 2
    broken(ssv.SSV_ERR_BAD_TAU, tau=tau)


@pytest.mark.parametrize("C,hkv", [([1500], 1), ([20011], 1), ([30001], 2), ([9000, 300, 2500], 1), ([5000, 700, 0, 6400], 8)])
def test_units_cut_into_many_parts(C, hkv):
    """Few units and many CTAs: a unit's keys are dealt to several of them, as many as its length is worth."""
    n = len(C)
    check(PagedBatch(C, [1] + [0] * (n - 1), [8, 3, 16, 5][:n], 4 * hkv, hkv, 128, 64, seed=sum(C)))


@pytest.mark.parametrize("skip", [0, 5])
def test_wait_runs_out(skip):
    """One key block's copy is left out: the wait for it ends after its budget, with an error code; other CTAs wait for
    that part in vain, too.  The workspace once cleared serves a normal call."""
    x = PagedBatch([6000, 5000], [0, 40], [8, 4], 2, 1, 128, 64, seed=17)
    t = x.device()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
    out = torch.empty(x.q.shape, dtype=torch.bfloat16, device="cuda")
    try:
        ssv.set_fault_injection(ssv.FAULT_ATTN, skip, 200_000)
        call(t, out, dev_status=status, workspace=ws)
        assert ssv.get_status(status) == ssv.SSV_ERR_TIMEOUT
    finally:
        ssv.set_fault_injection(None)
    ws.zero_()
    call(t, out, dev_status=status, workspace=ws)
    assert ssv.get_status(status) == ssv.SSV_OK
    o, tol = reference(x)
    assert (np.abs(out.double().cpu().numpy() - o) <= tol).all()
