"""assign_step_pages: what a request that is refused does to those behind it,
with every value written out by hand."""
import pytest
import torch

from paged_kv_cache_189_gb300 import pkv

pytestmark = pytest.mark.gpu


def step(new, kv, free, stack, table, tokens):
    """kv_lens_out, num_free_out, q_indptr, slots, the error bits, the table."""
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    t, ko, fo, qi, err = i32(table), i32([77] * len(kv)), i32([77]), i32([77] * (len(kv) + 1)), i32([0])
    slots, positions = (torch.full((tokens,), 77, dtype=torch.int64, device="cuda") for _ in range(2))
    pkv.assign_step_pages(i32(new), i32(kv), i32([free]), i32(stack), t, kv_lens_out=ko, num_free_out=fo, q_indptr=qi,
                          slots=slots, positions=positions, err=err)
    return ko.tolist(), int(fo), qi.tolist(), slots.tolist(), int(err), t.tolist()


def test_more_tokens_than_a_step_has():
    """20 tokens never fit a step of 16, and hold back the one behind them; withdrawn, it goes on."""
    table = [[-1, -1], [6, -1]]
    for _ in range(2):
        assert step([20, 1], [0, 5], 3, [7, 8, 9], table, 16) == ([0, 5], 3, [0, 0, 0], [-1] * 16, pkv.PKV_ERRBIT_LEN, table)
    assert step([0, 1], [0, 5], 3, [7, 8, 9], table, 16) == ([0, 6], 3, [0, 0, 1], [6 * 32 + 5] + [-1] * 15, 0, table)
    # asked for in pieces, both go on
    assert step([15, 1], [0, 5], 3, [7, 8, 9], table, 16) == (
        [15, 6], 2, [0, 15, 16], [9 * 32 + i for i in range(15)] + [6 * 32 + 5], 0, [[9, -1], [6, -1]])


def test_more_pages_than_the_table_is_wide():
    """Four pages never fit two columns; the page that the second needs is counted behind them."""
    table = [[-1, -1], [6, -1], [5, -1]]
    got = step([100, 1, 1], [0, 32, 5], 4, [1, 2, 3, 4], table, 200)
    assert got == ([0, 32, 6], 4, [0, 0, 0, 1], [5 * 32 + 5] + [-1] * 199, pkv.PKV_ERRBIT_LEN, table)
    got = step([0, 1, 1], [0, 32, 5], 4, [1, 2, 3, 4], table, 200)
    assert got == ([0, 33, 6], 3, [0, 0, 1, 2], [4 * 32, 5 * 32 + 5] + [-1] * 198, 0, [[-1, -1], [6, 4], [5, -1]])


def test_room_in_the_last_page_does_not_wait_for_pages():
    """Two pages where one is free: refused, as is the page behind them; the sequence that needs none goes on."""
    table = [[-1, -1], [6, -1], [5, -1]]
    got = step([64, 1, 1], [0, 5, 32], 1, [9], table, 70)
    assert got == ([0, 6, 32], 1, [0, 0, 1, 1], [6 * 32 + 5] + [-1] * 69, 0, table)
