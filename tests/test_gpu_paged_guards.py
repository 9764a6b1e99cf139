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
