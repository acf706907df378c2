"""The paged-cache operators together, as a serving loop runs them: tables
from the lengths, head norm and rotation, attention over the pages,
acceptance, commit -- several passes, lengths never read by the host between
them, one request ending and another taking its pages.  Each pass's outputs are
checked against the oracles on the same bytes."""
import numpy as np
import pytest
import torch

from diffusion_speculative_verification_gb300 import ssv, io as sio, workloads as W
import oracle.accept as oacc
import oracle.paged as opaged
from gpu_common import ensure_built
from paged_common import PagedBatch
from test_gpu_attn_fp8 import reference

pytestmark = pytest.mark.gpu


def setup_module():
    ensure_built()


@pytest.mark.parametrize("page", [16, 64])
def test_passes_of_a_serving_loop(page):
    r = np.random.default_rng(page)
    batch, Hq, Hkv, d, V, mp, n_pages, passes = 3, 4, 2, 128, 97, 256 // page, 3 * 256 // page, 5
    zeros = lambda *s: np.zeros(s, np.int32)  # noqa: E731
    # host mirrors of what the device holds
    C, held, table, free, n_free = zeros(batch), zeros(batch), np.full((batch, mp), -1, np.int32), \
        r.permutation(n_pages).astype(np.int32), n_pages
    codes = [np.full((n_pages, Hkv, page, d), 0x7F, np.uint8) for _ in range(2)]
    scale = [np.full((n_pages, Hkv), np.nan, np.float32) for _ in range(2)]
    g = dict(C=sio.int_tensor(C, "cuda"), held=sio.int_tensor(held, "cuda"), pages=sio.int_tensor(table, "cuda"),
             free=sio.int_tensor(free, "cuda"), n_free=sio.int_tensor([n_free], "cuda"))
    cache = [torch.from_numpy(c.copy()).cuda() for c in codes]
    sc = [torch.from_numpy(s.copy()).cuda() for s in scale]
    w = [W._store((1 + 0.2 * r.standard_normal(d)).astype(np.float32), W.BF16) for _ in range(2)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for step in range(passes):
        N = np.array([40, 3, 17], np.int32) if step == 0 else r.integers(0, 2, batch).astype(np.int32)
        B = r.integers(1, 9, batch).astype(np.int32)
        if step == 3:           # request 1 ends; in the pass after, a new one comes in its place
            C[1] = -1
            g["C"][1] = -1
        if step == 4:
            C[1], N[1] = 0, 60
            g["C"][1] = 0
        live = C >= 0
        rows = int(np.sum((N + 2 * B)[live]))
        seqs, slot_map, slot_off, g["held"], g["n_free"] = ssv.page_plan(
            g["C"], sio.int_tensor(N, "cuda"), sio.int_tensor(B, "cuda"), g["held"], g["pages"], g["free"],
            g["n_free"], page, rows, dev_status=status)
        plan, err = opaged.page_plan(C, N, B, held, table, free, n_free, page, rows)
        assert not err and np.array_equal(seqs.cpu().numpy(), plan["seqs"])
        assert np.array_equal(slot_map.cpu().numpy(), plan["slot_map"])
        held, table, free, n_free = plan["held"], plan["pages"], plan["free_list"], plan["n_free"]
        assert np.array_equal(g["pages"].cpu().numpy(), table) and int(g["n_free"]) == n_free

        def rnd(h):
            return W._store(r.standard_normal((rows, h, d)).astype(np.float32), W.BF16)

        slots = int(B[live].sum())
        x = PagedBatch.__new__(PagedBatch)
        x.Hq, x.Hkv, x.d, x.page, x.dtype, x.n_pages = Hq, Hkv, d, page, W.BF16, n_pages
        x.seqs, x.table, x.codes, x.scale, x.rows = plan["seqs"], table, codes, scale, rows
        x.idle = {b for b in range(batch) if not live[b]}
        x.tau = np.concatenate([W.random_tau(r, int(b)) for b in B[live]]).astype(np.int32)
        q_raw, k_raw, x.v_new = rnd(Hq), rnd(Hkv), rnd(Hkv)
        dev = ssv.Batch.from_device(seqs, rows, slots, 256, 60, 8)
        tau = sio.int_tensor(x.tau, "cuda")
        q, k = ssv.norm_rope_copy(sio.tensor(q_raw, W.BF16, "cuda"), sio.tensor(k_raw, W.BF16, "cuda"),
                                  *(sio.tensor(y, W.BF16, "cuda") for y in w), dev, dev_status=status)
        qr, kr = opaged.norm_rope_batch(x.seqs, x.values(q_raw), x.values(k_raw), *(x.values(y) for y in w))
        for got, want in ((q, qr), (k, kr)):
            assert (np.abs(got.double().cpu().numpy() - want) <= 2.0 ** -8 * np.abs(want) + 1e-4).all()
        x.q, x.k_new = sio.to_numpy_storage(q), sio.to_numpy_storage(k)
        v = sio.tensor(x.v_new, W.BF16, "cuda")
        o = ssv.verify_attn_fp8(q, *cache, *sc, g["pages"], k, v, dev, tau, dev_status=status)
        want, tol = reference(x)
        assert (np.abs(o.double().cpu().numpy() - want) <= tol).all()

        acc = W.make_accept_inputs("loop", W.MODE_ARGMAX, 0.0, V, B[live], B[live], seed=100 + step, tau=x.tau)
        t = sio.accept_to_device(acc, "cuda")
        n_acc_live, _, _ = ssv.accept(t["mode"], t["T"], t["logits"], t["draft_tokens"], tau, t["block"], t["gamma"],
                                      t["slot_off"], max_block=8, dev_status=status)
        assert np.array_equal(n_acc_live.cpu().numpy(), oacc.accept_batch(acc)["n_acc"])
        n_acc = torch.zeros(batch, dtype=torch.int32, device="cuda")
        n_acc[torch.from_numpy(live).cuda()] = n_acc_live
        g["C"] = ssv.commit_fp8(k, v, *cache, *sc, g["pages"], dev, tau, n_acc, dev_status=status)
        for i, y in enumerate((x.k_new, x.v_new)):
            codes[i], scale[i], n = opaged.commit_pages(x.seqs, table.reshape(-1), x.tau, n_acc.cpu().numpy(),
                                                        x.values(y), codes[i], scale[i])
            assert np.array_equal(cache[i].cpu().numpy(), codes[i])
            assert np.array_equal(sc[i].cpu().numpy(), scale[i], equal_nan=True)
        assert np.array_equal(g["C"].cpu().numpy(), n)
        C = n.astype(np.int32)
        assert ssv.get_status(status) == ssv.SSV_OK


def test_passes_without_rows_or_pages():
    """Empty calls of the other three, and attention where nothing is cached and no page exists: as over a flat cache."""
    def z(*s, dt=torch.int32):
        return torch.zeros(s, dtype=dt, device="cuda")

    bf, status = torch.bfloat16, z(1)
    none = ssv.Batch.from_device(z(0, 6), 0, 0, 0, 0, 1)
    codes, scale, w = z(4, 2, 16, 128, dt=torch.uint8), z(4, 2, dt=torch.float32), torch.ones(128, dtype=bf, device="cuda")
    q0, k0 = z(0, 4, 128, dt=bf), z(0, 2, 128, dt=bf)
    assert ssv.verify_attn_fp8(q0, codes, codes, scale, scale, z(0), k0, k0, none, z(0), dev_status=status).shape == q0.shape
    assert ssv.commit_fp8(k0, k0, codes, codes, scale, scale, z(0), none, z(0), z(0), dev_status=status).numel() == 0
    ssv.norm_rope_copy(q0, k0, w, w, none, dev_status=status)
    seqs = np.array([[0, 3, 4, 0, 0, 0]], np.int32)
    batch = ssv.Batch.from_device(torch.from_numpy(seqs).cuda(), 11, 4, 0, 3, 4)
    g = torch.Generator(device="cuda").manual_seed(5)
    q, k, v = (torch.randn(11, h, 128, device="cuda", generator=g).to(bf) for h in (4, 2, 2))
    tau = torch.tensor([2, 1, 4, 3], dtype=torch.int32, device="cuda")
    o = ssv.verify_attn_fp8(q, codes[:0], codes[:0], scale[:0], scale[:0], z(0), k, v, batch, tau, dev_status=status)
    flat = ssv.verify_attn(q, k0, k0, k, v, ssv.Batch(seqs), tau)
    assert ssv.get_status(status) == ssv.SSV_OK
    # bf16 weights and a bf16 result on either side: 2 (2^-8 + 2^-7) of at most max |v|
    assert float((o.float() - flat.float()).abs().max()) <= 2 * (2 ** -8 + 2 ** -7) * float(v.abs().max())
