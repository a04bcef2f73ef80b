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
