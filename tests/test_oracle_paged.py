"""Pins of the paged-cache oracle on cases worked by hand, and agreement of
its pieces with independent statements (CPU)."""
import numpy as np
import torch

import oracle.paged as op
import oracle.commit as ocommit
from paged_common import PagedBatch


def test_e4m3_table_and_rounding_agree_with_torch():
    codes = torch.arange(256, dtype=torch.int64).to(torch.uint8)
    v = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.isnan(v), np.isnan(op.E4M3)) and np.array_equal(v[~np.isnan(v)], op.E4M3[~np.isnan(v)])
    x = np.random.default_rng(1).standard_normal(20000) * np.exp2(np.random.default_rng(2).integers(-14, 7, 20000))
    x = np.concatenate([np.clip(x, -448, 448).astype(np.float32), op.E4M3[~np.isnan(op.E4M3)].astype(np.float32)])
    x = np.concatenate([x, (op.E4M3[:0x7E] + op.E4M3[1:0x7F]).astype(np.float32) / 2])        # every tie
    want = torch.from_numpy(x.astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(op.e4m3_codes(x.astype(np.float32)), want)
    assert op.e4m3_codes(np.array([np.nan, np.inf, -np.inf])).tolist() == [0x7F] * 3


def test_scale_is_the_smallest_power_of_two():
    assert op.scale_for(448.0) == 1.0 and op.scale_for(448.0 * (1 + 2 ** -20)) == 2.0
    assert op.scale_for(224.0) == 0.5 and op.scale_for(0.0) == 2.0 ** -100 and op.scale_for(1e-40) == 2.0 ** -100
    assert op.scale_for(float(np.finfo(np.float32).max)) == 2.0 ** 120


def test_page_plan_by_hand():
    # request 0 runs (5 tokens, page of 16 held), 1 has ended with pages 7 and 3, 2 is new
    pages = np.array([[9, -1, -1], [7, 3, -1], [-1, -1, -1]], np.int32)
    out, err = op.page_plan([5, -1, 0], [0, 4, 17], [12, 4, 2], [1, 2, 0], pages, np.array([1, 2, 8, 0], np.int32), 1,
                            16, 60)
    assert not err
    # the stack is [1, 7, 3]: request 0 takes 3 (17 tokens), request 2 takes 7, 1 (19 tokens)
    assert out["pages"].tolist() == [[9, 3, -1], [7, 3, -1], [7, 1, -1]]
    assert out["held"].tolist() == [2, 0, 2] and out["n_free"] == 0
    assert out["seqs"].tolist() == [[5, 0, 12, 0, 0, 0], [0, 0, 0, 24, 3, 12], [0, 17, 2, 24, 6, 12]]
    m = out["slot_map"]
    assert m[:12].tolist() == [9 * 16 + t for t in range(5, 16)] + [3 * 16] and (m[12:24] == -1).all()
    assert m[24:43].tolist() == [7 * 16 + t for t in range(16)] + [16, 17, 18] and (m[43:] == -1).all()


def test_page_plan_refuses_in_order():
    pages = np.full((3, 4), -1, np.int32)
    out, err = op.page_plan([0, 0, 0], [0, 40, 0], [3, 3, 3], [0, 0, 0], pages, np.array([0, 1, 2], np.int32), 3, 16, 60)
    assert err == {"no pages"} and out["held"].tolist() == [1, 0, 0] and out["n_free"] == 2
    assert out["seqs"][:, 2].tolist() == [3, 0, 0] and out["seqs"][:, 3].tolist() == [0, 6, 52]


def test_commit_pages_by_hand_on_a_growing_scale():
    codes = np.zeros((2, 1, 16, 64), np.uint8)
    scale = np.array([[0.25], [1.0]], np.float32)
    codes[1, 0, 0] = op.e4m3_codes(np.full(64, 448.0))
    codes[0, 0, :2] = op.e4m3_codes(np.array([[400.0], [2.0 ** -9]]) * np.ones((2, 64)))
    fresh = np.zeros((4, 1, 64))
    fresh[0] = 300.0                                    # scale 1: 100 stays 100, 2^-11 falls to 0
    c, s, n = op.commit_pages([[2, 0, 2, 0, 0, 0]], [0], [2, 1], [0], fresh, codes, scale)
    assert n.tolist() == [2] and np.array_equal(c, codes) and np.array_equal(s, scale)
    c, s, n = op.commit_pages([[2, 0, 2, 0, 0, 0]], [0], [1, 2], [1], fresh, codes, scale)
    assert n.tolist() == [3] and s.tolist() == [[1.0], [1.0]]
    v = op.e4m3_values(c[0, 0, :3])
    # 400 was stored as 384 (a tie, even mantissa) and stood for 96; 300 rounds to 288
    assert (v[0] == 96.0).all() and (v[1] == 0).all() and (v[2] == 288.0).all()
    assert np.array_equal(c[1], codes[1])


def test_commit_pages_appends_the_rows_of_the_commit_oracle():
    x = PagedBatch([5, 0, 37], [3, 20, 0], [4, 1, 9], 2, 2, 64, 16, seed=4)
    k = x.values(x.k_new)
    codes, scale, n = op.commit_pages(x.seqs, x.table.reshape(-1), x.tau, x.n_acc, k, x.codes[0], x.scale[0])
    C = x.seqs[:, 0].astype(np.int64)
    room = C + x.seqs[:, 1] + x.seqs[:, 2]
    off = np.concatenate([[0], np.cumsum(room)[:-1]])
    dst = np.zeros((int(room.sum()), 2, 64))
    want, _, n2 = ocommit.commit_batch(x.seqs, x.tau, x.n_acc, k, k, dst, dst, off)
    assert np.array_equal(n, n2)
    for b in range(3):
        s = x.seqs[b].copy()
        s[0] = n[b]
        got = op.gather_cache(s, x.table.reshape(-1), codes, scale)[C[b]:]
        ref = want[off[b] + C[b]:off[b] + n[b]]
        assert got.shape == ref.shape
        # half a step of e4m3: 2^-4 of the value, or half the smallest code of the page's scale
        assert (np.abs(got - ref) <= 2.0 ** -4 * np.abs(ref) + 2.0 ** -10 * np.nanmax(scale)).all()


def test_norm_by_hand():
    y = op.rms_norm(np.array([3.0, 4.0, 0.0, 0.0]), np.array([1.0, 2.0, 1.0, 1.0]), 0.0)
    assert np.allclose(y, [1.2, 3.2, 0, 0], atol=1e-15)
