"""ssv_page_plan against the one-request-at-a-time oracle: whole numbers, so
every output is compared for equality."""
import numpy as np
import pytest
import torch

from diffusion_speculative_verification_gb300 import ssv, io as sio
import oracle.paged as opaged
from gpu_common import ensure_built

pytestmark = pytest.mark.gpu


def setup_module():
    ensure_built()


def make(batch, page, seed, ended=0.2, n_hi=40, c_hi=300, slack=4, short=0, cap_rows=None):
    r = np.random.default_rng(seed)
    C, N, B = r.integers(0, c_hi + 1, batch), r.integers(0, n_hi + 1, batch), r.integers(1, 65, batch)
    gone = r.random(batch) < ended
    held = np.where(r.random(batch) < 0.5, -(-C // page), -(-(C + 20) // page))
    need = np.maximum(held, -(-(C + N + B) // page))
    mp = int(need.max(initial=1)) + 1
    n_pages = int(np.where(gone, held, need).sum()) + slack
    perm = r.permutation(n_pages).astype(np.int32)
    pages = np.full((batch, mp), -7, np.int32)
    at = 0
    for b in range(batch):
        pages[b, :held[b]] = perm[at:at + held[b]]
        at += held[b]
    n_free = max(0, n_pages - at - short)
    free = np.full(n_pages, -3, np.int32)
    free[:n_free] = perm[at:at + n_free]
    rows = int(np.sum((N + 2 * B)[~gone])) if cap_rows is None else cap_rows
    return [np.where(gone, -1 - r.integers(0, 3, batch), C).astype(np.int32), N.astype(np.int32), B.astype(np.int32),
            held.astype(np.int32), pages, free, n_free, page, rows]


def run(x, out=None):
    t = [sio.int_tensor(a, "cuda") for a in x[:6]] + [sio.int_tensor([x[6]], "cuda")]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    seqs, slot_map, slot_off, held, n_free = ssv.page_plan(*t, x[7], x[8], out=out, dev_status=status)
    got = dict(seqs=seqs, slot_map=slot_map, slot_off=slot_off, held=held, n_free=n_free, pages=t[4], free_list=t[5])
    st = ssv.get_status(status)
    assert np.array_equal(t[3].cpu().numpy(), x[3]) and int(t[6]) == x[6]     # counters are not written
    return {k: v.cpu().numpy() for k, v in got.items()}, st


def check(x):
    got, st = run(x)
    want, err = opaged.page_plan(*x)
    for k in want:
        assert np.array_equal(got[k], np.asarray(want[k]).reshape(got[k].shape)), k
    codes = {"invalid": ssv.SSV_ERR_INVALID, "no pages": ssv.SSV_ERR_NO_PAGES}
    assert (st in {codes[e] for e in err}) if err else st == ssv.SSV_OK
    return got, err


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("batch", [1, 2, 31, 64, 513, 1000])
def test_plan_parity(batch, page):
    _, err = check(make(batch, page, 100 * batch + page))
    assert not err


def test_largest_batch_and_long_prompts():
    check(make(4096, 16, 5, n_hi=2))
    check(make(3, 64, 6, n_hi=30000, c_hi=100000))
    check(make(1, 16, 7, ended=0.0, n_hi=0, c_hi=0))
    check(make(40, 16, 8, ended=1.0))                       # every request has ended: no rows


@pytest.mark.parametrize("short", [1, 3, 20, 10 ** 6])
def test_refusals_in_batch_order(short):
    """The stack runs dry: later requests that want pages are refused, those that want none are served."""
    _, err = check(make(60, 16, 11 + short, ended=0.0, slack=0, short=short))
    assert "no pages" in err


def test_invalid_requests_take_nothing():
    x = make(12, 16, 21, ended=0.2)
    x[0][3], x[1][3] = 5, -1                                # N < 0
    x[0][4], x[2][4] = 9, 65                                # B > 64
    x[0][5], x[2][5] = 9, 0                                 # B < 1
    x[0][6], x[3][6] = 9, -2                                # held out of range
    x[0][7], x[1][7] = 10, 1 << 30                          # more pages than the table has columns
    x[0][8], x[3][8] = -1, 10 ** 6                          # ended, held out of range
    x[0][9], x[1][9] = 0x7FFFFFF0, 0x7FFFFFF0               # sums beyond 32 bits
    _, err = check(x)
    assert "invalid" in err


def test_rows_that_do_not_fit():
    x = make(12, 16, 22, ended=0.0)
    x[8] //= 2
    _, err = check(x)
    assert "invalid" in err
    x[8] = 0
    check(x)


def test_slot_map_behind_the_last_row_is_minus_one():
    x = make(9, 32, 23)
    x[8] += 5000
    got, _ = check(x)
    assert (got["slot_map"][-5000:] == -1).all()


@pytest.mark.parametrize("n_free", [-1, 10 ** 9])
def test_bad_stack_height(n_free):
    x = make(5, 16, 24)
    x[6] = n_free
    _, err = check(x)
    assert "invalid" in err


def test_planned_again_from_the_same_counters():
    """held and n_free are left as they were, so a second call repeats the first."""
    x = make(50, 16, 25)
    t = [sio.int_tensor(a, "cuda") for a in x[:6]] + [sio.int_tensor([x[6]], "cuda")]
    first = [y.clone() for y in ssv.page_plan(*t, x[7], x[8])] + [t[4].clone(), t[5].clone()]
    again = list(ssv.page_plan(*t, x[7], x[8])) + [t[4], t[5]]
    assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_side_stream_and_graph():
    x = make(64, 64, 26)
    want, _ = run(x)
    t = [sio.int_tensor(a, "cuda") for a in x[:6]] + [sio.int_tensor([x[6]], "cuda")]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out = ssv.page_plan(*t, x[7], x[8])
    side.synchronize()
    assert np.array_equal(out[1].cpu().numpy(), want["slot_map"])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ssv.page_plan(*t, x[7], x[8], out=out)
    for y in out:
        y.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert np.array_equal(out[1].cpu().numpy(), want["slot_map"]) and np.array_equal(out[0].cpu().numpy(), want["seqs"])


def test_empty_batch():
    """No request: no row is anyone's, and the stack is as high as it was."""
    e = torch.zeros(0, dtype=torch.int32, device="cuda")
    free, n_free = torch.arange(5, dtype=torch.int32, device="cuda"), torch.tensor([3], dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (None, side):
        seqs, slot_map, slot_off, held, left = ssv.page_plan(e, e, e, e, e.view(0, 4), free, n_free, 16, 7, stream=stream)
        torch.cuda.synchronize()
        assert seqs.shape == (0, 6) and slot_off.numel() == held.numel() == 0
        assert slot_map.tolist() == [-1] * 7 and left.tolist() == [3] and free.tolist() == [0, 1, 2, 3, 4]
