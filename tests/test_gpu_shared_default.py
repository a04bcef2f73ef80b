"""Decode attention over shared prefixes with the groups that share by default, as a user has it: against the
64-bit reference, from the call and from the engine; and the prefix CTAs' waits."""
import numpy as np
import pytest
import torch

import pagedattention_paged_kv_gb300 as pkv
from pagedattention_paged_kv_gb300.scheduler import Sequence, shared_prefixes
from shared_helpers import Shared, check
from test_gpu_shared import run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads,kv_heads,d,bs,fp8", [
    (64, 8, 128, 16, False), (64, 8, 128, 16, True), (32, 8, 128, 8, False), (8, 8, 64, 32, False), (24, 1, 128, 16, True)])
@pytest.mark.parametrize("groups", [
    [(4096, [1, 300])], [(2000, [9, 40, 700])], [(1024, [3 * s for s in range(40)])],
    [(64 * 2 ** i, [1, None, 50] * (1 + i)) for i in range(6)], [(600, [17, 1]) for _ in range(30)]])
def test_groups_that_share_by_default(groups, heads, kv_heads, d, bs, fp8):
    b = Shared(groups, heads, kv_heads, d, bs, fp8, seed=heads + len(groups), alone=[5, 0, 900])
    got = run(b)
    assert pkv.get_device_error() == 0
    check(got, b.reference())


def test_the_engine_over_documents_behind_one_prompt():
    """Two documents behind one system prompt, requests on both and short ones, against 64 bits."""
    from pagedattention_paged_kv_gb300.engine import PagedKVEngine
    HQ, HKV, D, BS = 32, 4, 128, pkv.BLOCK_SIZE
    e = PagedKVEngine(2000, HQ, HKV, D, max_num_seqs=40, prefix_cache=True, shared_decode=True)
    g = torch.Generator(device="cuda").manual_seed(3)
    system, docs = list(range(3 * BS)), [list(range(10 ** 4 * d, 10 ** 4 * d + 70 * BS)) for d in (1, 2)]
    arrivals = {0: [(0, 0)], 4: [(1, 1)], 8: [(i, i % 2) for i in range(2, 16)] + [(16, None)], 20: [(17, None)]}
    deep = 0
    for it in range(40):
        for i, doc in arrivals.get(it, []):
            tokens = system + (docs[doc] if doc is not None else []) + [10 ** 6 + i] * 5
            e.add(Sequence(i, len(tokens), 20 + i, it, prompt_tokens=tokens))
        batch = e.schedule()
        if batch.num_seqs:
            q, k, v = (torch.randn(batch.num_tokens, h, D, generator=g, device="cuda").bfloat16() for h in (HQ, HKV, HKV))
            got = e.run(batch, q, k, v)
            start, lens = shared_prefixes(batch.block_tables, batch.context_lens)
            if batch.max_q_len == 1 and lens.any():
                deep += int((lens >= 70 * BS).sum() == 2)
                b = Shared.__new__(Shared)
                b.heads, b.kv_heads, b.d, b.bs, b.fp8, b.scale = HQ, HKV, D, BS, False, e.scale
                b.q, b.k, b.v, b.ctx = q, e.k_cache, e.v_cache, batch.context_lens.tolist()
                b.tables = torch.from_numpy(np.ascontiguousarray(batch.block_tables)).cuda()
                check(got, b.reference())
        e.complete(batch)
    assert pkv.get_device_error() == 0 and deep > 5


@pytest.mark.parametrize("n,bs", [(12, 8), (40, 16)])   # a narrow tile, whose halves share the chunks out; wide ones
def test_waits_of_the_prefix_ctas_run_out(n, bs):
    """Sequences without own tokens: nothing but the prefix CTAs has anything to wait for.  With a limit of 1 ns
    waits do run out behind a long prefix, and the launch behind is right."""
    b = Shared([(20000, [0, 0])], 64, 8, 128, bs, seed=n)
    b.tables, b.ctx = b.tables[:1].repeat(n, 1), [20000] * n
    b.lens, b.start = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (b.ctx, [0, n]))
    b.q = torch.randn(n, 64, 128, generator=torch.Generator().manual_seed(n)).bfloat16().cuda()
    ref = b.reference()
    check(run(b), ref)
    assert pkv.get_device_error() == 0
    ran_out = 0
    for _ in range(10):
        pkv.set_wait_limit_ns(1)
        try:
            short = run(b)
        finally:
            pkv.set_wait_limit_ns(0)
        healthy = run(b)  # queued directly behind
        flags = pkv.get_device_error()
        assert flags & ~pkv.DEVERR_TIMEOUT == 0
        check(healthy, ref)
        if flags:
            ran_out += 1
        else:
            check(short, ref)
    assert ran_out > 0
