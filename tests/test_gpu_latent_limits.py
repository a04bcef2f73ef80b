"""The latent-attention calls and the step metadata at the ends of their ranges: offsets past 32 bits in
the cache and in the output, the most sequences of a step, wide cache rows."""
import numpy as np
import pytest
import torch

import pagedattention_paged_kv_gb300 as pkv
from latent_helpers import ROPE, SCALE, Batch, absorbed_reference, check, expanded_reference

pytestmark = pytest.mark.gpu


def test_a_cache_past_32_bits_of_offset():
    """4.2 million slots of 576 columns, 4.8 GB and 2.4e9 elements: rows are written to its first and last
    blocks and attended to in both forms."""
    R, bs, NB, H = 512, 16, 262_144 + 3, 4
    ctx, ql = [100, 70], [3, 70]
    b = Batch(ctx, ql, H, R, R + ROPE, bs, seed=1)
    e = Batch(ctx, ql, H, R, 128 + ROPE, bs, seed=1)
    cache = torch.zeros(NB, bs, R + ROPE, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator()
    g.manual_seed(2)
    ids = torch.cat([torch.arange(NB - 9, NB), torch.arange(9)])[torch.randperm(18, generator=g)]
    tables = torch.full((2, 7), -1, dtype=torch.int32)
    tables[0], tables[1, :5] = ids[:7], ids[7:12]
    rows, slots = torch.cat(b.rows), []
    for s, c in enumerate(ctx):
        p = torch.arange(c)
        slots.append(tables[s][p // bs].long() * bs + p % bs)
    slots = torch.cat(slots).cuda()
    assert int(slots.max()) * (R + ROPE) > 2 ** 31
    pkv.latent_cache_write(cache, rows[:, :R].contiguous().cuda(), rows[:, R:].contiguous().cuda(), slots)
    assert pkv.get_device_error() == 0
    assert torch.equal(cache.view(-1, R + ROPE)[slots].cpu(), rows)
    assert cache.count_nonzero() == rows.count_nonzero()
    b.tables, b.cache, e.tables, e.rows = tables.cuda(), cache, tables.cuda(), b.rows
    out = torch.full((73, H, R), float("nan"), dtype=torch.bfloat16, device="cuda")
    pkv.latent_attention_absorbed(out, b.q, cache, b.tables, b.context_lens, SCALE, query_start_loc=b.qsl)
    check(out, *absorbed_reference(b))
    w = [(torch.randn(H, 128, R, generator=g) * R ** -0.5).bfloat16().cuda() for _ in range(2)]
    out = torch.full((73, H, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    pkv.latent_attention_expanded(out, e.q, e.qsl, cache, b.tables, e.context_lens, *w, SCALE, 170)
    check(out, *expanded_reference(e, *w))
    assert pkv.get_device_error() == 0


def test_outputs_past_32_bits_of_offset():
    """66,000 sequences of one token, 64 heads, R = 512: 2.2e9 output elements, each row its token's
    latent; every 1000th sequence is idle and gives zeros."""
    S, H, R, bs = 66_000, 64, 512, 8
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    cache = torch.randn(S, bs, R + ROPE, device="cuda", generator=g, dtype=torch.bfloat16)
    q = torch.randn(S, H, R + ROPE, device="cuda", generator=g, dtype=torch.bfloat16)
    tables = torch.randperm(S, device="cuda", generator=g).int()[:, None]
    ctx = torch.ones(S, dtype=torch.int32, device="cuda")
    ctx[::1000] = 0
    out = torch.full((S, H, R), 3.0, dtype=torch.bfloat16, device="cuda")
    pkv.latent_attention_absorbed(out, q, cache, tables, ctx, SCALE)
    assert pkv.get_device_error() == 0
    want = cache[tables[:, 0].long(), 0, :R] * ctx[:, None]
    for lo in range(0, S, 6000):
        assert torch.equal(out[lo:lo + 6000], want[lo:lo + 6000, None].expand(-1, H, -1))


@pytest.mark.parametrize("bs", [8, 64])
def test_a_step_of_the_most_sequences(bs):
    S = 16384
    r = np.random.Generator(np.random.PCG64(4))
    cached, new = r.integers(0, 200, S), r.integers(0, 4, S)
    held, after = -(-cached // bs), -(-(cached + new) // bs)
    perm = r.permutation(int(after.sum()) + 5).astype(np.int32)
    tables = np.full((S, int(after.max())), -1, np.int32)
    at = 0
    for s in range(S):
        tables[s, :held[s]] = perm[at:at + held[s]]
        at += held[s]
    free = perm[at:]
    want, slots, taken = tables.copy(), [], 0
    for s in range(S):
        for p in range(cached[s], cached[s] + new[s]):
            if p % bs == 0:
                want[s, p // bs] = free[taken]
                taken += 1
            slots.append(int(want[s, p // bs]) * bs + p % bs)
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda().int()
    t, ctx, end = dev(tables), torch.zeros(S, dtype=torch.int32, device="cuda"), dev(np.array([0]))
    qsl, sl = torch.zeros(S + 1, dtype=torch.int32, device="cuda"), torch.zeros(len(slots) + 3, dtype=torch.int64,
                                                                                 device="cuda")
    pkv.step_metadata(t, ctx, qsl, sl, end, dev(cached), dev(new), dev(free), dev(np.array([0])), len(perm), bs)
    assert pkv.get_device_error() == 0
    assert np.array_equal(t.cpu().numpy(), want) and int(end) == taken
    assert np.array_equal(ctx.cpu().numpy(), cached + new)
    assert np.array_equal(qsl.cpu().numpy(), np.concatenate([[0], np.cumsum(new)]))
    assert sl.tolist() == slots + [-1] * 3


@pytest.mark.parametrize("tokens,latent,rope", [(1500, 8, 8), (700, 4096, 512), (40, 65536, 65536), (1200, 24, 2048)])
def test_cache_rows_of_any_width(tokens, latent, rope):
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    c, r = (torch.randn(tokens, n, device="cuda", generator=g, dtype=torch.bfloat16) for n in (latent, rope))
    slots = torch.randperm(tokens + 24, device="cuda", generator=g)[:tokens]
    slots[::9] = -1
    cache = torch.zeros(-(-(tokens + 24) // 8), 8, latent + rope, dtype=torch.bfloat16, device="cuda")
    want = cache.clone().view(-1, latent + rope)
    keep = slots >= 0
    want[slots[keep]] = torch.cat([c, r], 1)[keep]
    pkv.latent_cache_write(cache, c, r, slots)
    assert pkv.get_device_error() == 0
    assert torch.equal(cache.view(-1, latent + rope), want)
