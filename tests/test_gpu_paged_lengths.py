"""Lengths that a serving loop keeps on the device: what commit returns is the
next plan's input, over passes in which a request gets no pages, has ended, or
is rejected.  Each pass's attention and pages are checked against the oracles."""
import numpy as np
import pytest
import torch

from diffusion_speculative_verification_gb300 import ssv, io as sio, workloads as W
import oracle.paged as opaged
from gpu_common import ensure_built
from paged_common import PagedBatch
from test_gpu_attn_fp8 import reference

pytestmark = pytest.mark.gpu
HQ, HKV, D, PAGE = 4, 2, 128, 16


def setup_module():
    ensure_built()


class Loop:
    """The device's state and its host mirror."""

    def __init__(self, batch, n_pages, seed):
        self.r = np.random.default_rng(seed)
        self.batch, self.n_pages = batch, n_pages
        self.C, self.held = np.zeros(batch, np.int32), np.zeros(batch, np.int32)
        self.table = np.full((batch, n_pages), -1, np.int32)
        self.free, self.n_free = self.r.permutation(n_pages).astype(np.int32), n_pages
        self.codes = [np.full((n_pages, HKV, PAGE, D), 0x7F, np.uint8) for _ in range(2)]
        self.scale = [np.full((n_pages, HKV), np.nan, np.float32) for _ in range(2)]
        self.g = dict(C=self.ints(self.C), held=self.ints(self.held), pages=self.ints(self.table),
                      free=self.ints(self.free), n_free=self.ints([n_pages]))
        self.cache = [torch.from_numpy(c.copy()).cuda() for c in self.codes]
        self.sc = [torch.from_numpy(s.copy()).cuda() for s in self.scale]
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    @staticmethod
    def ints(x):
        return sio.int_tensor(np.asarray(x, np.int32), "cuda")

    def run(self, N, B, errors=(), bad_tau=None, in_place=False):
        """One pass; `errors`: what the plan reports; bad_tau: a request whose stage map is broken in the commit."""
        r, g, batch = self.r, self.g, self.batch
        N, B = np.array(N, np.int32), np.array(B, np.int32)
        rows, slots = int(np.sum((N + 2 * B)[self.C >= 0])), int(B[self.C >= 0].sum())
        seqs, _, slot_off, g["held"], g["n_free"] = ssv.page_plan(
            g["C"], self.ints(N), self.ints(B), g["held"], g["pages"], g["free"], g["n_free"], PAGE, rows,
            dev_status=self.status)
        plan, err = opaged.page_plan(self.C, N, B, self.held, self.table, self.free, self.n_free, PAGE, rows)
        assert err == set(errors) and np.array_equal(seqs.cpu().numpy(), plan["seqs"])
        assert ssv.get_status(self.status) == (ssv.SSV_ERR_NO_PAGES if err else ssv.SSV_OK)
        self.held, self.table, self.free, self.n_free = plan["held"], plan["pages"], plan["free_list"], plan["n_free"]
        x = PagedBatch.__new__(PagedBatch)
        x.Hq, x.Hkv, x.d, x.page, x.dtype, x.n_pages = HQ, HKV, D, PAGE, W.BF16, self.n_pages
        x.seqs, x.table, x.codes, x.scale, x.rows = plan["seqs"], self.table, self.codes, self.scale, rows
        x.idle = {b for b in range(batch) if x.seqs[b, 2] == 0}
        tau = [W.random_tau(r, int(b)) for b, c in zip(B, self.C) if c >= 0]
        x.tau = np.concatenate(tau).astype(np.int32)
        x.q, x.k_new, x.v_new = (W._store(r.standard_normal((rows, h, D)).astype(np.float32), W.BF16)
                                 for h in (HQ, HKV, HKV))
        q, k, v = (sio.tensor(y, W.BF16, "cuda") for y in (x.q, x.k_new, x.v_new))
        dev = ssv.Batch.from_device(seqs, rows, slots, 16 * self.n_pages, int(N.max()), int(B.max()))
        t = self.ints(x.tau)
        o = ssv.verify_attn_fp8(q, *self.cache, *self.sc, g["pages"], k, v, dev, t, dev_status=self.status)
        assert ssv.get_status(self.status) == ssv.SSV_OK
        want, tol = reference(x)
        live = ~np.isnan(want)
        assert (np.abs(o.double().cpu().numpy() - want)[live] <= tol[live]).all()
        n_acc = np.array([r.integers(0, b + 1) for b in B], np.int32)
        seqs_host = x.seqs.copy()
        if bad_tau is not None:
            off = int(seqs_host[bad_tau, 5])
            t[off:off + int(B[bad_tau])] = 1
            seqs_host[bad_tau, 1:3] = 0         # nothing of it is written
        old = g["C"].clone()
        g["C"] = ssv.commit_fp8(k, v, *self.cache, *self.sc, g["pages"], dev, t, self.ints(n_acc),
                                new_len=g["C"] if in_place else None, dev_status=self.status, cache_len=g["C"])
        assert in_place or torch.equal(old, self.ints(self.C))
        assert ssv.get_status(self.status) == (ssv.SSV_OK if bad_tau is None else ssv.SSV_ERR_BAD_TAU)
        for i, y in enumerate((x.k_new, x.v_new)):
            self.codes[i], self.scale[i], n = opaged.commit_pages(seqs_host, self.table.reshape(-1), x.tau, n_acc,
                                                                  x.values(y), self.codes[i], self.scale[i], self.C)
            assert np.array_equal(self.cache[i].cpu().numpy(), self.codes[i])
            assert np.array_equal(self.sc[i].cpu().numpy(), self.scale[i], equal_nan=True)
        assert np.array_equal(g["C"].cpu().numpy(), n)
        self.C = n.astype(np.int32)

    def end(self, b):
        self.C[b] = -1
        self.g["C"][b] = -1


@pytest.mark.parametrize("in_place", [False, True])
def test_a_request_refused_for_one_pass_goes_on(in_place):
    s = Loop(3, 12, 1)                                                     # 192 tokens in all
    s.run([40, 70, 20], [2, 3, 2], in_place=in_place)                      # 3 + 5 + 2 pages
    held = s.C.copy()
    s.run([10, 30, 20], [3, 4, 5], {"no pages"}, in_place=in_place)        # the second and third get none
    assert s.C[0] > held[0] and (s.C[1:] == held[1:]).all()
    s.end(0)
    s.run([0, 30, 20], [1, 4, 5], in_place=in_place)                       # and go on where they were
    assert s.C[0] == -1 and s.C[1] >= held[1] + 30 and s.C[2] >= held[2] + 20
    s.run([0, 1, 1], [4, 4, 4], in_place=in_place)
    assert s.C[0] == -1 and s.held[0] == 0                                 # the ended one stays ended


def test_a_rejected_sequence_keeps_its_length_and_pages():
    s = Loop(3, 30, 2)
    s.run([40, 33, 20], [2, 3, 2])
    n = s.C.copy()
    s.run([1, 2, 1], [4, 4, 4], bad_tau=1)
    assert s.C[1] == n[1] and s.C[0] > n[0] and s.C[2] > n[2]
    s.run([1, 2, 1], [4, 4, 4])
    assert s.C[1] >= n[1] + 2


def test_lengths_without_those_of_the_plan():
    """As before: a rejected sequence -1, an idle record its own cache_len."""
    x = PagedBatch([20, 33, 5], [1, 1, 1], [4, 4, 4], HQ, HKV, D, PAGE, seed=3, idle=(2,))
    t = x.device()
    t["tau"][4:8] = 3
    n = ssv.commit_fp8(t["k_new"], t["v_new"], t["k_cache"], t["v_cache"], t["k_scale"], t["v_scale"], t["pages"],
                       t["batch"], t["tau"], t["n_acc"])
    assert n.tolist() == [20 + 1 + int(x.n_acc[0]), -1, 0]


def test_slot_map_names_the_rows_that_the_commit_fills():
    """By stage, not by slot: row N + s - 1 of a request's entries is where the data row of stage s goes."""
    s = Loop(2, 20, 4)
    s.run([37, 5], [3, 2])
    N, B = [3, 0], [6, 8]
    table, held = s.g["pages"], s.g["held"]
    seqs, slot_map, _, held, _ = ssv.page_plan(s.g["C"], s.ints(N), s.ints(B), held, table, s.g["free"], s.g["n_free"],
                                               PAGE, 31)
    rows, tau = 31, np.array([3, 1, 6, 2, 5, 4, 8, 1, 7, 2, 6, 3, 5, 4], np.int32)
    k = torch.zeros(rows, HKV, D, dtype=torch.bfloat16, device="cuda")
    k[:, 0, :rows] = 448 * torch.eye(rows, device="cuda").to(k)            # each row is one of its own
    batch = ssv.Batch.from_device(seqs, rows, 14, 320, 3, 8)
    cache, sc = [torch.zeros_like(c) for c in s.cache], [torch.ones_like(y) for y in s.sc]
    ssv.commit_fp8(k, k, *cache, *sc, table, batch, s.ints(tau), s.ints(B), cache_len=s.g["C"])
    at = slot_map.cpu().numpy()
    codes, scale = cache[0].cpu().numpy(), sc[0].cpu().numpy()
    row0 = 0
    for b in range(2):
        t = tau[6 * b: 6 * b + B[b]]
        for j in range(N[b] + B[b]):
            row = row0 + (j if j < N[b] else N[b] + int(np.flatnonzero(t == j - N[b] + 1)[0]))
            page, o = divmod(int(at[row0 + j]), PAGE)
            got = opaged.e4m3_values(codes[page, 0, o]) * scale[page, 0]
            assert got[row] == 448 and got.sum() == 448
        row0 += N[b] + 2 * B[b]
