"""The page calls on damaged counts and lists: what the header promises of them, and nothing written outside
the arrays."""
import numpy as np
import pytest

import page_helpers as H
import pagedattention_paged_kv_gb300 as pkv
from test_gpu_pages import call_free, same

pytestmark = pytest.mark.gpu

FAR_BELOW = [-2 ** 29 - 1, -2 ** 30, -2 ** 30 - 1, -2 ** 31]   # counts as nobody would set them


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("count", FAR_BELOW)
@pytest.mark.parametrize("begin", [-1, 10 ** 6, 2 ** 31 - 1, -2 ** 31])
def test_a_refused_free_gathers_nothing(begin, count, in_place):
    """free_begin outside the list and counts far below zero, as memory that was never set up has both."""
    p = H.Pages([40, 20], 16, spare=300)
    p.begin = begin
    p.refs[::2] = count
    got = call_free(p, [0, 1], in_place)
    assert pkv.get_device_error() == pkv.DEVERR_FREE_BLOCKS
    same(got, (p.lens, p.refs, p.free, np.array([begin])))


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("lens", [[40, 20], [16 * 300, 16 * 2000 + 5, 16 * 700] * 4])   # one CTA, a cluster
@pytest.mark.parametrize("count", [-1, *FAR_BELOW])
def test_negative_counts_are_no_freed_pages(count, lens, in_place):
    """Of pages that no freed row has, and of one that a freed row has: flagged and 0 behind the call, not on
    the list; the pages that are freed are."""
    p = H.Pages(lens, 16, spare=40, share=False)
    rows = list(range(1, len(lens)))
    p.refs[p.free[p.begin:]] = count
    p.refs[p.tables[0, 1]] = count
    p.refs[p.tables[1, 0]] = count
    want = H.Pages(lens, 16, spare=40, share=False)
    w_lens, w_refs, lst, end = H.free(want, rows)
    w_refs[p.tables[0, 1]] = 0
    gone = np.setdiff1d(lst[end[0]:p.begin], p.tables[1, :1])
    w_free = p.free.copy()
    w_free[p.begin - len(gone):p.begin] = gone
    got = call_free(p, rows, in_place)
    assert pkv.get_device_error() == pkv.DEVERR_BLOCK_ID
    same(got, (w_lens, w_refs, w_free, np.array([p.begin - len(gone)])))
