"""CPU tests of nested families of shared prefixes: documents behind one system prompt, a short or diverging
request beside a long family, and the groups of any run against all its splits."""
import itertools

import numpy as np
import pytest

from pagedattention_paged_kv_gb300 import BlockManager, _build
from pagedattention_paged_kv_gb300.scheduler import Scheduler, Sequence, shared_prefixes

BS = 16


def tables_of(rows):
    t = np.full((len(rows), max(map(len, rows))), -1, np.int32)
    for i, r in enumerate(rows):
        t[i, :len(r)] = r
    return t


def saved(start, lens):
    return sum((b - a - 1) * n for a, b, n in zip(start[:-1], start[1:], lens))


def test_documents_behind_one_system_prompt():
    """Four documents of 500 blocks behind a prompt of four, eight requests each."""
    system, fresh = list(range(4)), itertools.count(10 ** 4)
    docs = [list(range(100 + 500 * i, 600 + 500 * i)) for i in range(4)]
    rows = [system + doc + [next(fresh)] for doc in docs for _ in range(8)]
    start, lens = shared_prefixes(tables_of(rows), np.full(32, 504 * BS + 5, np.int32))
    assert start.tolist() == [0, 8, 16, 24, 32] and lens.tolist() == [504 * BS] * 4
    assert start.dtype == lens.dtype == np.int32


@pytest.mark.parametrize("place", [0, 32])
def test_a_short_request_beside_a_long_family(place):
    """32 requests on one document and one of a few tokens with the same first block."""
    doc = list(range(1, 501))
    rows = [doc + [10 ** 4 + i] for i in range(32)]
    rows.insert(place, [doc[0], 7])
    ctx = np.full(33, 500 * BS + 3, np.int32)
    ctx[place] = 20
    start, lens = shared_prefixes(tables_of(rows), ctx)
    family = [0, 1, 33] if place == 0 else [0, 32, 33]
    assert start.tolist() == family and sorted(lens.tolist()) == [0, 500 * BS]
    assert lens[1 if place == 0 else 0] == 500 * BS


def test_a_family_stays_whole_where_splitting_saves_less():
    rows = [[1, 2, 3, 4], [1, 2, 3, 4], [1, 2, 3, 9], [1, 2, 3, 9]]
    start, lens = shared_prefixes(tables_of(rows), np.full(4, 4 * BS, np.int32))
    assert start.tolist() == [0, 4] and lens.tolist() == [3 * BS]


@pytest.mark.parametrize("seed", range(40))
def test_no_split_of_a_run_saves_more(seed):
    r = np.random.Generator(np.random.PCG64(seed))
    n, depth = int(r.integers(2, 10)), int(r.integers(1, 7))
    rows = [[0] + r.integers(0, 2, depth).tolist() for _ in range(n)]
    if seed % 2:
        rows.sort()
    ctx = r.integers(1, (depth + 1) * BS + 1, n).astype(np.int32)
    t = tables_of(rows)
    start, lens = shared_prefixes(t, ctx)
    assert start[0] == 0 and start[-1] == n and (np.diff(start) > 0).all() and len(lens) == len(start) - 1

    def prefix(a, b):
        m = int(ctx[a:b].min()) // BS
        same = [j for j in range(m) if not (t[a:b, j] == t[a, j]).all()]
        return min(same, default=m) * BS if b - a > 1 else 0
    assert lens.tolist() == [prefix(a, b) for a, b in zip(start[:-1], start[1:])]
    most = max(saved(cuts, [prefix(a, b) for a, b in zip(cuts[:-1], cuts[1:])])
               for k in range(n) for inner in itertools.combinations(range(1, n), k)
               for cuts in [(0, *inner, n)])
    assert saved(start, lens) == most


def test_the_scheduler_puts_families_next_to_each_other():
    """Two documents behind one system prompt, requests on both arriving in turn, one short request."""
    _build.build_library()
    sched = Scheduler(BlockManager(400), max_num_seqs=16, chunk_size=512, prefix_cache=True, group_shared=True)
    system, docs = list(range(2 * BS)), [list(range(1000 * d, 1000 * d + 20 * BS)) for d in (1, 2)]
    fresh = itertools.count(10 ** 5)

    def add(i, tokens):
        tokens = tokens + [next(fresh) for _ in range(3)]
        sched.add(Sequence(i, len(tokens), 30, 0, prompt_tokens=tokens))
    for d in (0, 1):   # the documents enter the cache
        add(d, system + docs[d])
        sched.complete(sched.schedule())
    for i in range(2, 10):
        add(i, system + docs[i % 2])
    add(10, system)
    for _ in range(4):
        batch = sched.schedule()
        sched.complete(batch)
    assert batch.max_q_len == 1 and batch.num_seqs == 11
    start, lens = shared_prefixes(batch.block_tables, batch.context_lens)
    assert sorted(zip(np.diff(start).tolist(), lens.tolist())) == [(1, 0), (5, 22 * BS), (5, 22 * BS)]
    assert all(len({it.seq.seq_id % 2 for it in batch.items[a:b]}) == 1 for a, b in zip(start[:-1], start[1:]))
