"""Calls on a paged cache whose counts, lengths or owners are not what the call needs: rows that cannot be
served stay as they are, nothing of another row is written, and the status says so."""
import numpy as np
import pytest
import torch

from test_gpu_paged import PAGE, Case, ints, same_state, sgd  # noqa: F401

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------------------------
# compaction
# ---------------------------------------------------------------------------------------------
@pytest.mark.parametrize("cu,wrong", [([0, 2, 1, 5], 1), ([0, 2, 4, 90], 2), ([-1, 2, 4, 5], 0), ([0, 2, 4, 35], 2), ([0, 2, 4, 5], None)])
def test_keep_leaves_rows_with_wrong_counts(sgd, cu, wrong):
    """cu_kept that descends, leaves the list or asks for more tokens than the row has: the row keeps all of its tokens,
    and the release that follows a keep takes no page from it.  (None: a length that no row can have.)"""
    case = Case((100, 70, 30), seed=4)
    if wrong is None:
        case.lens[1], wrong = 10 ** 6, 1
    cache, st = case.gpu(sgd), case.host()
    idx = np.tile(np.arange(40), (2, 1))
    idx[:, :5] = (3, 9, 5, 29, 29)
    if cu[2] == 1:
        idx[:, :5] = (0, 2, 9, 11, 29)
    new, ws = sgd.pages_keep(cache, ints(idx), ints(cu))
    assert sgd.workspace_status(ws) == 0x4
    want = np.diff(cu)
    want[wrong] = case.lens[wrong]
    assert new.tolist() == want.tolist()
    for b in range(3):
        for h in range(2):
            if b != wrong:
                st._compact(b, h, 0, idx[h, cu[b]:cu[b + 1]])
    same_state(cache, st)
    sgd.pages_release(cache, new)
    held = [-(-int(n) // PAGE) for n in want]
    held[wrong] = int(case.held[wrong])
    assert cache.held.tolist() == held and int(cache.ref_count.sum()) == sum(held)


@pytest.mark.parametrize("call", ["keep", "accept"])
@pytest.mark.parametrize("taken", [True, False])
def test_compaction_of_an_ended_row_writes_nothing(sgd, call, taken):
    """A row that was released but still has its old length: its table lists pages that are free, or another row's."""
    case = Case((200, 64, 130), seed=11, max_pages=8)
    cache = case.gpu(sgd)
    for t in (cache.k, cache.v):
        t.nan_to_num_(0.0)
    sgd.pages_release(cache, ints([0, 64, 130]))
    if taken:  # row 1 takes the pages
        new, ws = sgd.pages_reserve(cache.with_lens(ints([0, 64, 130])), ints([0, 200, 0]))
        assert sgd.workspace_status(ws) == 0 and new.tolist() == [0, 264, 130]
        cache.lens[1] = 264
        assert set(cache.page_table[1, 1:5].tolist()) & set(cache.page_table[0, :4].tolist())
    k, v, L = cache.k.clone(), cache.v.clone(), cache.lens.tolist()

    def go(held):
        c = sgd.PagedKv(cache.k, cache.v, cache.page_table, cache.lens, cache.held if held else None, cache.ref_count)
        if call == "keep":  # rows 1 and 2 keep everything
            parts = [np.arange(1, 150), np.arange(L[1]), np.arange(L[2])]
            cu = np.concatenate([[0], np.cumsum([len(p) for p in parts])])
            return sgd.pages_keep(c, ints(np.tile(np.concatenate(parts), (2, 1))), ints(cu))
        return sgd.pages_accept(c, ints([[3, 5, 6, -1, -1, -1, -1], [0, 1, 2, 3, 4, 5, 6], [0, 1, 2, 3, 4, 5, 6]]), ints([3, 7, 7]),
                                ints([7, 7, 7]))

    new, ws = go(True)
    assert sgd.workspace_status(ws) == 0x4 and new.tolist() == L
    assert torch.equal(cache.k, k) and torch.equal(cache.v, v)
    if not taken:  # without held the free pages themselves tell
        new, ws = go(False)
        assert sgd.workspace_status(ws) == 0x8 and new.tolist() == L
        assert torch.equal(cache.k, k) and torch.equal(cache.v, v)
