"""ssv_commit_fp8 against the float64 oracle: a power-of-two scale makes
every quotient exact in fp32, so codes, scales and lengths are compared for
equality, over the whole cache."""
import numpy as np
import pytest
import torch

from diffusion_speculative_verification_gb300 import ssv, io as sio, workloads as W
import oracle.paged as opaged
from gpu_common import ensure_built
from paged_common import PagedBatch

pytestmark = pytest.mark.gpu


def setup_module():
    ensure_built()


def run(x, strided=False, seqs=None, n_acc=None, tau=None, table=None):
    t = x.device(strided)
    if seqs is not None:
        t["batch"].dev.copy_(sio.int_tensor(seqs, "cuda"))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    nl = ssv.commit_fp8(t["k_new"], t["v_new"], t["k_cache"], t["v_cache"], t["k_scale"], t["v_scale"],
                        t["pages"] if table is None else sio.int_tensor(table, "cuda"), t["batch"],
                        t["tau"] if tau is None else sio.int_tensor(tau, "cuda"),
                        t["n_acc"] if n_acc is None else sio.int_tensor(n_acc, "cuda"), dev_status=status)
    st = ssv.get_status(status)
    return {k: t[k].cpu().numpy() for k in ("k_cache", "v_cache", "k_scale", "v_scale")}, nl.cpu().numpy(), st


def expect(x, seqs=None, n_acc=None, keep=None):
    seqs = x.seqs if seqs is None else seqs
    n_acc = x.n_acc if n_acc is None else np.asarray(n_acc)
    keep = list(range(len(seqs))) if keep is None else keep
    out = {}
    for i, (c, rows) in enumerate((("k", x.k_new), ("v", x.v_new))):
        out[c + "_cache"], out[c + "_scale"], n = opaged.commit_pages(
            seqs[keep], x.table.reshape(-1), x.tau, n_acc[keep], x.values(rows), x.codes[i], x.scale[i])
    new_len = np.full(len(seqs), -1)
    new_len[keep] = n
    return out, new_len


def same(got, want):
    for k in want:
        assert np.array_equal(got[k], want[k], equal_nan=got[k].dtype.kind == "f"), k


def check(x, **kw):
    got, nl, st = run(x, **kw)
    assert st == ssv.SSV_OK
    want, n = expect(x, n_acc=kw.get("n_acc"))
    same(got, want)
    assert np.array_equal(nl, n)


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("dtype,d", [(W.BF16, 128), (W.BF16, 64), (W.F32, 128), (W.F32, 64)])
def test_parity(page, dtype, d):
    check(PagedBatch([0, 5, page - 1, page, 3 * page + 7, 300], [0, 3, 1, 0, 2 * page + 5, 1], [1, 4, 64, 7, 32, 16],
                     2, 2, d, page, seed=page + d, dtype=dtype, pad=5), strided=page == 32)


@pytest.mark.parametrize("page", [16, 128])
def test_prompts(page):
    check(PagedBatch([0, 77], [700, 1], [3, 2], 4, 4, 128, page, seed=3), strided=True)


@pytest.mark.parametrize("which", ["none", "all"])
def test_accepted_extremes(which):
    x = PagedBatch([4, 0, 31], [0, 3, 0], [5, 64, 1], 2, 1, 128, 16, seed=5)
    check(x, n_acc=[0, 0, 0] if which == "none" else [5, 64, 1])


def test_spread_of_magnitudes():
    """Pages whose old scale is far below and far above the appended rows', zeros, and fp32's extremes."""
    x = PagedBatch([20, 20, 20, 7, 9], [2, 0, 4, 3, 1], [3, 8, 8, 4, 2], 1, 1, 64, 16, seed=6, dtype=W.F32, spread=14)
    x.k_new[:4] *= np.float32(1e30)
    x.k_new[8:20] *= np.float32(1e-33)
    x.v_new[0] = 0
    x.v_new[30:40] = 0
    x.v_new[3, 0, :4] = [np.finfo(np.float32).max, -np.finfo(np.float32).tiny, 1e-45, -0.0]
    check(x, n_acc=[3, 8, 5, 4, 2])


def test_non_finite_rows_are_stored_as_nan():
    x = PagedBatch([3], [6], [2], 1, 1, 128, 16, seed=7)
    x.k_new[0, 0, 5], x.k_new[1, 0, 6], x.v_new[2, 0, 7] = 0x7FC1, 0x7F80, 0xFF80   # NaN, inf, -inf
    x.v_new[3] = 0x7F80
    check(x, n_acc=[2])


def test_many_small_sequences_and_idle_records():
    r = np.random.default_rng(8)
    n = 300
    x = PagedBatch(r.integers(0, 60, n), r.integers(0, 3, n), r.integers(1, 6, n), 1, 1, 64, 16, seed=9,
                   idle=(0, 17, 299))
    got, nl, st = run(x)
    want, m = expect(x)
    assert st == ssv.SSV_OK and np.array_equal(nl, m)
    same(got, want)


def test_refused_sequences_are_left_alone():
    x = PagedBatch([20, 33, 8], [2, 5, 0], [4, 6, 3], 2, 2, 128, 16, seed=10)
    # (what is changed, the status)
    def broken(**kw):
        got, nl, st = run(x, **kw)
        want, m = expect(x, n_acc=kw.get("n_acc"), keep=[0, 2])
        same(got, want)
        assert np.array_equal(nl, m)
        return st
    tau = x.tau.copy()
    tau[4:10] = 1
    assert broken(tau=tau) == ssv.SSV_ERR_BAD_TAU
    assert broken(n_acc=[1, 7, 2]) == ssv.SSV_ERR_INVALID
    assert broken(n_acc=[1, -1, 2]) == ssv.SSV_ERR_INVALID
    for bad in (-1, x.n_pages, 0x7FFFFFFF):
        table = x.table.copy()
        table[1, 2] = bad                                   # its first touched page
        assert broken(table=table) == ssv.SSV_ERR_INVALID
    for field, value in ((0, -1), (1, -1), (1, 10 ** 9), (2, 0), (2, 65), (4, -1), (4, 10 ** 6), (5, -1), (5, 9)):
        s = x.seqs.copy()
        s[1, field] = value
        assert broken(seqs=s) == ssv.SSV_ERR_INVALID, (field, value)


def test_bad_page_behind_the_touched_ones_is_not_looked_at():
    x = PagedBatch([20], [2], [4], 1, 1, 128, 16, seed=11, extra=9)
    x.table = np.concatenate([x.table, np.full((1, 2), -5, np.int32)], 1)
    check(x)


def test_appends_pass_after_pass():
    """Rows appended one pass at a time meet the oracle's codes after every pass."""
    x = PagedBatch([0, 30], [40, 0], [8, 8], 2, 2, 128, 32, seed=12)
    x.table = np.random.default_rng(2).permutation(40)[:20].reshape(2, 10).astype(np.int32)
    x.seqs[:, 4] = [0, 10]
    x.codes = [np.concatenate([c, np.full((40 - len(c),) + c.shape[1:], 0x7F, np.uint8)]) for c in x.codes]
    x.scale = [np.concatenate([s, np.full((40 - len(s), 2), np.nan, np.float32)]) for s in x.scale]
    for i in range(2):   # sequence 1's cached rows
        for j in range(1):
            x.codes[i][x.table[1, 0]], x.scale[i][x.table[1, 0]] = 0x30, 0.25
    x.n_pages = 40
    t = x.device()
    r = np.random.default_rng(13)
    for step in range(5):
        acc = np.array([r.integers(0, 9), r.integers(0, 9)], np.int32)
        grow = np.float32(1.7 ** step)
        rows = [W.f32_to_bf16_bits(W.bf16_bits_to_f32(y) * grow) for y in (x.k_new, x.v_new)]
        for name, y in zip(("k_new", "v_new"), rows):
            t[name].copy_(sio.tensor(y, W.BF16, "cuda"))
        t["batch"].dev.copy_(sio.int_tensor(x.seqs, "cuda"))
        nl = ssv.commit_fp8(t["k_new"], t["v_new"], t["k_cache"], t["v_cache"], t["k_scale"], t["v_scale"], t["pages"],
                            t["batch"], t["tau"], sio.int_tensor(acc, "cuda"))
        for i, c in enumerate("kv"):
            x.codes[i], x.scale[i], n = opaged.commit_pages(x.seqs, x.table.reshape(-1), x.tau, acc,
                                                            x.values(rows[i]), x.codes[i], x.scale[i])
            assert np.array_equal(t[c + "_cache"].cpu().numpy(), x.codes[i])
            assert np.array_equal(t[c + "_scale"].cpu().numpy(), x.scale[i], equal_nan=True)
        assert np.array_equal(nl.cpu().numpy(), n)
        x.seqs[:, 0] = n
        if step == 0:  # the prompt is in: later passes bring its tail rows only
            x.seqs[0, 1] = 0
            x.seqs[1, 3] = x.seqs[0, 3] + 16


def test_graph_replay():
    x = PagedBatch([20, 33], [2, 5], [4, 6], 2, 2, 128, 16, seed=14)
    want, n = expect(x)
    t = x.device()
    nl = torch.zeros(2, dtype=torch.int32, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ssv.commit_fp8(t["k_new"], t["v_new"], t["k_cache"], t["v_cache"], t["k_scale"], t["v_scale"], t["pages"],
                       t["batch"], t["tau"], t["n_acc"], new_len=nl)
    g.replay()
    g.replay()     # the same rows again: nothing changes any more
    torch.cuda.synchronize()
    same({k: t[k].cpu().numpy() for k in want}, want)
    assert np.array_equal(nl.cpu().numpy(), n)


@pytest.mark.parametrize("hkv,rows", [(16, 15000), (5, 71000)])
def test_prompts_long_enough_for_ctas_with_several_groups(hkv, rows):
    """More chunks of rows than CTAs at once: a CTA takes several groups of heads in turn, also unevenly many."""
    check(PagedBatch([0, 77], [rows, 300], [3, 2], hkv, hkv, 64, 128, seed=rows))


def test_scales_that_are_no_powers_of_two():
    """Scales that the caller has put there: kept where they suffice, and each code within a rounding of its value.  An
    e4m3 rounding is off by at most 2^-4 of the value, or 2^-10 of the scale below the normal range; x (1 / s), or
    code (s_old / s), by at most 2^-22 of it before."""
    x = PagedBatch([5, 300, 77, 129], [0, 3, 40, 1], [8, 4, 16, 64], 2, 2, 128, 64, seed=21, spread=5)
    old = [s.copy() for s in x.scale]
    for s in x.scale:
        s *= np.float32(1.37)
    got, nl, st = run(x)
    assert st == ssv.SSV_OK
    want, n = expect(x)
    assert np.array_equal(nl, n)
    grown = kept = 0
    for i, c in enumerate("kv"):
        s = got[c + "_scale"]
        assert np.array_equal(s, want[c + "_scale"], equal_nan=True)
        a = opaged.e4m3_values(got[c + "_cache"]) * s[:, :, None, None].astype(np.float64)
        b = opaged.e4m3_values(want[c + "_cache"]) * s[:, :, None, None].astype(np.float64)
        live = ~np.isnan(b)
        assert np.array_equal(np.isnan(a), ~live)
        # both are roundings of one value: apart by at most two half steps
        step = 2 * (2.0 ** -4 * np.maximum(np.abs(a), np.abs(b)) * (1 + 2.0 ** -4) + 2.0 ** -10 * s[:, :, None, None])
        assert (np.abs(a - b) <= step)[live].all()
        assert (a != b)[live].mean() < 1e-3   # and the same code but near a tie
        grown += int((s > old[i] * np.float32(1.37)).sum())
        kept += int((s == old[i] * np.float32(1.37)).sum())
    assert grown > 0 and kept > 0
