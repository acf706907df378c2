"""ssv_norm_rope_copy against the float64 oracle.

Tolerance per output element with y the normed pair (y1, y2), before any run:
the sum of squares, mean, square root, division and two products round at most
12 times in a row (each 2^-24), the two products and the sum of the rotation 3
times, and the angle's fraction rounds by 2^-25 of half a turn (pi 2^-25 =
1.6 2^-24 rad) with sincospi good to 2 ulp: in all below 24 * 2^-24 < 2^-19 of
|y1| + |y2|.  Storing in bf16 adds half a step, 2^-8 of the value."""
import numpy as np
import pytest
import torch

from diffusion_speculative_verification_gb300 import ssv, io as sio, workloads as W
import oracle.paged as opaged
from gpu_common import ensure_built

pytestmark = pytest.mark.gpu


def setup_module():
    ensure_built()


def make(C, N, B, Hq, Hkv, d, dtype, seed, pad=0):
    r = np.random.default_rng(seed)
    seqs = W.seq_table(C, N, B)
    rows = int(np.sum(np.asarray(N) + 2 * np.asarray(B))) + pad
    q, k = (W._store((r.standard_normal((rows, h, d)) * 2.0 ** r.integers(-6, 7, (rows, h, 1))).astype(np.float32),
                     dtype) for h in (Hq, Hkv))
    w = [W._store((1 + 0.5 * r.standard_normal(d)).astype(np.float32), dtype) for _ in range(2)]
    return dict(seqs=seqs, rows=rows, q=q, k=k, w=w, dtype=dtype, d=d, pad=pad)


def bound(x, seqs, what, w, ref, eps):
    y = np.abs(opaged.rms_norm(W.values_f64(x[what], x["dtype"]), W.values_f64(w, x["dtype"]), eps))
    h = x["d"] // 2
    pair = np.concatenate([y[..., :h] + y[..., h:]] * 2, -1)
    return pair * 2.0 ** -19 + (np.abs(ref) * 2.0 ** -8 * (1 + 2.0 ** -10) if x["dtype"] == W.BF16 else 0) + 1e-30


def dev(x):
    t = {n: sio.tensor(x[n], x["dtype"], "cuda") for n in ("q", "k")}
    t["w"] = [sio.tensor(w, x["dtype"], "cuda") for w in x["w"]]
    t["batch"] = ssv.Batch.from_device(sio.int_tensor(x["seqs"], "cuda"), x["rows"], 0, 0, 0, 64)
    return t


def check(x, eps=1e-6, base=10000.0, positions=None, strided=False, in_place=False):
    t = dev(x)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pos = None if positions is None else sio.int_tensor(positions, "cuda")
    q, k = t["q"], t["k"]
    if strided:
        buf = torch.full((x["rows"], q.shape[1] + 2 * k.shape[1], x["d"]), 7.0, dtype=q.dtype, device="cuda")
        buf[:, :q.shape[1]], buf[:, q.shape[1]:q.shape[1] + k.shape[1]] = q, k
        q, k = buf[:, :q.shape[1]], buf[:, q.shape[1]:q.shape[1] + k.shape[1]]
    out = {} if in_place else dict(q_out=torch.full(q.shape, 3.0, dtype=q.dtype, device="cuda"),
                                   k_out=torch.full(k.shape, 3.0, dtype=k.dtype, device="cuda"))
    before = [q.clone(), k.clone()]
    qo, ko = ssv.norm_rope_copy(q, k, *t["w"], t["batch"], base, eps, positions=pos, dev_status=status, **out)
    assert ssv.get_status(status) == ssv.SSV_OK
    seqs = x["seqs"]
    ref = opaged.norm_rope_batch(seqs, W.values_f64(x["q"], x["dtype"]), W.values_f64(x["k"], x["dtype"]),
                                 *(W.values_f64(w, x["dtype"]) for w in x["w"]), base, eps, positions)
    n = x["rows"] - x["pad"]
    for got, want, what, w, was in ((qo, ref[0], "q", x["w"][0], before[0]), (ko, ref[1], "k", x["w"][1], before[1])):
        g = got.double().cpu().numpy()
        assert (np.abs(g[:n] - want[:n]) <= bound(x, seqs, what, w, want, eps)[:n]).all(), what
        if x["pad"]:   # rows behind the last sequence are left as they were
            assert torch.equal(got[n:], was[n:] if in_place else torch.full_like(got[n:], 3.0))
    if strided and in_place:
        assert (buf[:, q.shape[1] + k.shape[1]:] == 7.0).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [W.F32, W.BF16])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (16, 8), (14, 2), (40, 8), (65, 13)])
def test_parity(hq, hkv, dtype, d):
    check(make([0, 1000, 5, 8191], [1, 0, 70, 3], [1, 8, 64, 33], hq, hkv, d, dtype, hq + d, pad=3))


@pytest.mark.parametrize("dtype", [W.F32, W.BF16])
def test_more_rows_than_fit_one_wave(dtype):
    check(make([0, 50], [1500, 7], [16, 3], 8, 2, 128, dtype, 9), strided=True)


@pytest.mark.parametrize("in_place", [False, True])
def test_strided_rows(in_place):
    check(make([7, 90], [5, 0], [4, 9], 6, 2, 128, W.BF16, 10, pad=2), strided=True, in_place=in_place)
    check(make([7, 90], [5, 0], [4, 9], 6, 3, 64, W.F32, 11, pad=2), strided=True, in_place=in_place)


def test_in_place_packed():
    check(make([7, 90], [5, 0], [4, 9], 6, 2, 128, W.F32, 12), in_place=True)


def test_far_positions_and_other_bases():
    check(make([16777000, 1 << 20], [100, 0], [16, 64], 2, 1, 128, W.F32, 13))
    check(make([131000], [20], [16], 2, 1, 64, W.F32, 14), base=1e6)
    check(make([300], [20], [16], 2, 1, 64, W.F32, 15), base=500.0, eps=0.1)


def test_position_table():
    x = make([10, 3], [2, 0], [5, 8], 4, 2, 128, W.F32, 16)
    check(x, positions=np.random.default_rng(1).integers(0, 100000, x["rows"]).astype(np.int32))


def test_many_sequences():
    r = np.random.default_rng(3)
    n = 700
    check(make(r.integers(0, 5000, n), r.integers(0, 2, n), r.integers(1, 5, n), 2, 1, 128, W.BF16, 17))


def test_zero_rows_and_large_values():
    """A zero head divides by sqrt(eps); a head of 1e17 sums its squares within fp32."""
    x = make([3], [4], [2], 4, 2, 128, W.BF16, 18)
    x["q"][0], x["k"][1] = 0, 0
    check(x)
    x["q"][1] = W.f32_to_bf16_bits(np.full((4, 128), 1e17, np.float32))
    check(x)


def test_idle_and_refused_records():
    x = make([3, 50, 9], [4, 0, 2], [2, 6, 3], 2, 1, 128, W.F32, 19)
    for rec, code in (((0, 0, 0), ssv.SSV_OK), ((5, 0, 65), ssv.SSV_ERR_INVALID), ((-1, 0, 6), ssv.SSV_ERR_INVALID),
                      ((0x7FFFFFFF, 0, 6), ssv.SSV_ERR_INVALID), ((5, 100, 6), ssv.SSV_ERR_INVALID)):
        t = dev(x)
        s = x["seqs"].copy()
        s[1, :3] = rec
        t["batch"].dev.copy_(sio.int_tensor(s, "cuda"))
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.full_like(t["q"], 3.0)
        ssv.norm_rope_copy(t["q"], t["k"], *t["w"], t["batch"], q_out=out, dev_status=status)
        assert ssv.get_status(status) == code, rec
        lo, hi = int(x["seqs"][1, 3]), int(x["seqs"][2, 3])
        assert (out[lo:hi] == 3.0).all() and (out[:lo] != 3.0).any() and (out[hi:] != 3.0).any()


def test_negative_table_entry_leaves_its_rows():
    x = make([3], [1], [2], 2, 1, 64, W.F32, 20)
    t = dev(x)
    pos = torch.tensor([4, -5, 9, 0, 0], dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full_like(t["q"], 3.0)
    ssv.norm_rope_copy(t["q"], t["k"], *t["w"], t["batch"], q_out=out, positions=pos, dev_status=status)
    assert ssv.get_status(status) == ssv.SSV_ERR_INVALID
    assert (out[[1, 3]] == 3.0).all() and (out[[0, 2, 4]] != 3.0).any()


def test_graph_on_a_side_stream():
    x = make([100, 7], [0, 3], [8, 8], 16, 8, 128, W.BF16, 21)
    t = dev(x)
    want, _ = ssv.norm_rope_copy(t["q"], t["k"], *t["w"], t["batch"], q_out=torch.empty_like(t["q"]),
                                 k_out=torch.empty_like(t["k"]))
    qo, ko = torch.zeros_like(t["q"]), torch.zeros_like(t["k"])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=torch.cuda.Stream()):
        ssv.norm_rope_copy(t["q"], t["k"], *t["w"], t["batch"], q_out=qo, k_out=ko)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(qo, want)
