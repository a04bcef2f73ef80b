"""The page calls with as many rows, forks and listed rows as there may be: a cluster of 16 CTAs whose
shared memory is nearly full."""
import numpy as np
import pytest

import page_helpers as H
import pagedattention_paged_kv_gb300 as pkv
from test_gpu_pages import call_compact, call_fork, call_free, same

pytestmark = pytest.mark.gpu

ROWS = 16384


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("bs", [8, 64])
def test_as_many_rows_as_there_may_be(bs, in_place):
    lens = [1, bs, 3 * bs, 2 * bs + 5, 4 * bs - 1, 0, 7, 3 * bs + 1]
    p = H.Pages(lens, bs, seed=bs, extra_rows=ROWS - len(lens), spare=ROWS + 10)
    r = np.random.Generator(np.random.PCG64(bs))
    src = r.integers(0, len(lens), ROWS)
    dst = np.concatenate([r.permutation(np.arange(len(lens), ROWS)), np.full(len(lens), 9)])
    src[100:110] = -1                 # padding
    dst[-len(lens):] = dst[:len(lens)]   # rows that earlier forks take
    want = H.fork(p, src, dst)
    same(call_fork(p, src, dst, in_place), want)
    assert pkv.get_device_error() == pkv.DEVERR_SEQ
    p.tables, p.lens, p.refs, _, end = want
    p.begin = int(end[0])
    rows = r.permutation(ROWS)
    rows[:50] = -1
    want = H.free(p, rows)
    same(call_free(p, rows, in_place), want)
    p.lens, p.refs, p.free, end = want
    p.begin = int(end[0])
    tables, refs, pairs, count, lst, end = call_compact(p, 300, in_place)
    w_tables, w_refs, w_pairs, w_count, ids, w_end = H.compact(p, 300, p.NB)
    if in_place:   # entries of empty rows stay
        held = np.arange(p.tables.shape[1]) < -(-p.lens[:, None] // bs)
        w_tables = np.where(held, w_tables, p.tables)
    same((tables, refs, pairs, count, end), (w_tables, w_refs, w_pairs, w_count, w_end))
    assert np.array_equal(lst.cpu().numpy()[w_end[0]:], ids) and pkv.get_device_error() == 0
