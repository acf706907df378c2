"""ssv_page_plan at the most rows that its 32-bit arguments name: a slot map of
2^31 - 1 entries (8.6 GB), filled by one long request, and left empty."""
import pytest
import torch

from diffusion_speculative_verification_gb300 import ssv
from gpu_common import ensure_built

pytestmark = pytest.mark.gpu
ROWS, PAGE = (1 << 31) - 1, 16


def setup_module():
    ensure_built()


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def pieces(n, step=1 << 27):
    return ((a, min(a + step, n)) for a in range(0, n, step))


def test_one_request_of_nearly_all_rows():
    pages = (1 << 27) - 1
    new = pages * PAGE - 8                      # every token of every page, eight rows of a block among them
    rows = new + 16
    assert rows < ROWS
    table = torch.full((1, pages), -1, dtype=torch.int32, device="cuda")
    free = torch.arange(pages, dtype=torch.int32, device="cuda")
    status = i32(0)
    seqs, slot_map, _, held, n_free = ssv.page_plan(i32(0), i32(new), i32(8), i32(0), table, free, i32(pages), PAGE, ROWS,
                                                    dev_status=status)
    assert ssv.get_status(status) == ssv.SSV_OK
    assert seqs.tolist() == [[0, new, 8, 0, 0, 0]] and held.tolist() == [pages] and n_free.tolist() == [0]
    for a, b in pieces(pages):                  # from the top of the stack down
        assert torch.equal(table[0, a:b], torch.arange(pages - 1 - a, pages - 1 - b, -1, dtype=torch.int32, device="cuda"))
    for a, b in pieces(new + 8):
        t = torch.arange(a, b, dtype=torch.int64, device="cuda")
        assert torch.equal(slot_map[a:b].long(), (pages - 1 - t // PAGE) * PAGE + t % PAGE)
    assert (slot_map[new + 8:] == -1).all()


def test_few_rows_of_a_long_slot_map():
    table, status = torch.full((2, 4), -1, dtype=torch.int32, device="cuda"), i32(0)
    seqs, slot_map, _, _, _ = ssv.page_plan(i32(0, 0), i32(3, 4), i32(2, 5), i32(0, 0), table, i32(0, 1, 2, 3), i32(4),
                                            PAGE, ROWS, dev_status=status)
    assert ssv.get_status(status) == ssv.SSV_OK
    assert seqs.tolist() == [[0, 3, 2, 0, 0, 0], [0, 4, 5, 7, 4, 2]]
    assert slot_map[:21].tolist() == list(range(48, 53)) + [-1] * 2 + list(range(32, 41)) + [-1] * 5
    for a, b in pieces(ROWS - 21):
        assert (slot_map[21 + a:21 + b] == -1).all()
