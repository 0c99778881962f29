"""What the page pool reports when more than one thing went wrong, and pages that the
tables name though nobody counts them: against values written out by hand."""
import pytest
import torch

import gqa_kv_head_gb300 as fr

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def make_pool(n_pages, n_seq, max_pages, ps=16):
    return fr.PagePool(ints([0] * n_pages), ints([0] * n_seq), torch.full((n_seq, max_pages), -1, dtype=torch.int32, device="cuda"), ps)


def status(pool):
    try:
        fr.pages_check(pool)
    except fr.FrError as e:
        return e.status
    return 0


def test_both_reports_of_one_reserve():
    """Slot 0 has fewer keys than tokens, slot 1 needs three pages of two: both are told, one a check."""
    pool = make_pool(2, 2, 4)
    pool.kv_len.copy_(ints([3, 40]))
    fr.pages_reserve(pool, ints([0, 5, 45]))
    assert pool.page_table.tolist() == [[-1] * 4, [0, 1, -1, -1]] and pool.refs.tolist() == [1, 1]
    assert [status(pool) for _ in range(3)] == [7, 6, 0]


def test_reports_of_several_calls():
    """A report that was not asked for yet is not lost to one of the other kind."""
    pool = make_pool(1, 3, 2)
    fr.pages_free(pool, ints([7]))                       # no such slot
    pool.kv_len[1] = 20
    fr.pages_reserve(pool, ints([0, 0, 20, 20]))         # one page of two
    assert status(pool) == 7
    fr.pages_fork(pool, ints([2]), ints([2]))            # itself
    assert [status(pool) for _ in range(2)] == [6, 0]
    # each alone
    fr.pages_free(pool, ints([-2]))
    assert [status(pool) for _ in range(2)] == [6, 0]
    pool.kv_len[2] = 1
    fr.pages_reserve(pool, ints([0, 0, 0, 1]))
    assert [status(pool) for _ in range(2)] == [7, 0]


@pytest.mark.parametrize("n_seq,n_child", [(6, 1), (6, 4), (400, 300)])
@pytest.mark.parametrize("max_pages", [4, 700])
def test_fork_skips_a_page_without_holders(n_seq, n_child, max_pages):
    """A page that counts no holder is free, whatever an entry says: the children do not
    hold it (their entry is -1), it stays free, and the next reserve hands it out once."""
    pool = make_pool(40, n_seq, max_pages)
    pool.kv_len[0] = 50
    fr.pages_reserve(pool, ints([0] + [50] * n_seq))     # pages 0 .. 3
    assert status(pool) == 0
    pool.refs[1], pool.refs[3] = 0, -2
    children = list(range(1, 1 + n_child))
    fr.pages_fork(pool, ints([0] * n_child), ints(children))
    assert status(pool) == 6
    rows = pool.page_table.tolist()
    assert rows[0] == [0, 1, 2, 3] + [-1] * (max_pages - 4)
    for c in children:
        assert rows[c] == [0, -1, 2] + [-1] * (max_pages - 3)
    assert pool.kv_len.tolist() == [50] * (1 + n_child) + [0] * (n_seq - 1 - n_child)
    assert pool.refs.tolist() == [1 + n_child, 0, 1 + n_child, -2] + [0] * 36
    last = n_seq - 1
    pool.kv_len[last] = 16
    fr.pages_reserve(pool, ints([0] * n_seq + [16]))
    assert pool.page_table[last, 0].item() == 1 and pool.refs[1].item() == 1
    assert status(pool) == 0
