"""The page calls on damaged counts and lists: what the header promises of them, and nothing written outside
the arrays."""
import numpy as np
import pytest
import torch

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


class Guarded:
    """int32 tensors on the GPU with untouched words before and behind each."""

    def __init__(self):
        self.whole = []

    def __call__(self, a):
        a = np.asarray(a, np.int64).astype(np.int32)
        x = torch.full((a.size + 128,), 77, dtype=torch.int32, device="cuda")
        self.whole.append(x)
        x[64:64 + a.size] = torch.from_numpy(a.reshape(-1)).cuda()
        return x[64:64 + a.size].view(a.shape)

    def intact(self):
        return all((x[:64] == 77).all() and (x[-64:] == 77).all() for x in self.whole)


@pytest.mark.parametrize("rows,pages", [(5, 40), (300, 9000), (40, 40000)])   # one CTA, a cluster of 4, of 16
@pytest.mark.parametrize("seed", range(12))
def test_any_contents_stay_inside_the_arrays(seed, rows, pages):
    """Every array holds whatever memory may hold: small and huge numbers of both signs."""
    r = np.random.Generator(np.random.PCG64([seed, rows]))
    width, forks, bs = 30, 50, int(r.choice([8, 16, 64]))

    def any_of(top, *shape):
        x = r.integers(-3, top + 4, shape)
        huge = r.integers(-2 ** 31, 2 ** 31, shape)
        return np.where(r.random(shape) < (0.3 if seed % 2 else 0.02), huge, x)
    g = Guarded()
    t, lens, refs = g(any_of(pages, rows, width)), g(any_of(width * bs, rows)), g(any_of(3, pages))
    lst, begin = g(any_of(pages, pages + 20)), g(any_of(pages, 1))
    src, dst, some = g(any_of(rows, forks)), g(any_of(rows, forks)), g(any_of(rows, forks))
    lens[::3] = 0
    pairs, moves, count, end = g(np.zeros((forks, 2))), g(np.zeros((37, 2))), g([0]), g([0])
    new_t, new_lens, new_refs = g(np.zeros((rows, width))), g(np.zeros(rows)), g(np.zeros(pages))
    known = pkv.DEVERR_SEQ | pkv.DEVERR_CONTEXT_LEN | pkv.DEVERR_BLOCK_ID | pkv.DEVERR_FREE_BLOCKS
    for _ in range(2):
        pkv.fork_pages(t, new_lens, new_refs, pairs, end, lens, refs, lst, begin, src, dst, bs)
        pkv.fork_pages(t, lens, refs, pairs, begin, lens, refs, lst, begin, src, dst, bs)
        pkv.compact_pages(new_t, new_refs, moves, count, lst, end, t, lens, refs, bs)
        pkv.free_pages(new_lens, new_refs, lst, end, t, lens, refs, begin, some, bs)
        pkv.free_pages(lens, refs, lst, begin, t, lens, refs, begin, some, bs)
        pkv.compact_pages(t, refs, moves, count, lst, end, t, lens, refs, bs)
        assert pkv.get_device_error() & ~known == 0 and g.intact()
