"""The step metadata built on the GPU, against a token-by-token restatement; and whole steps
(metadata, cache write, attention) captured as a graph and replayed."""
import numpy as np
import pytest
import torch

import pagedattention_paged_kv_gb300 as pkv

pytestmark = pytest.mark.gpu


def plain(tables, cached, new, free, begin, room, bs):
    tables = tables.copy()
    slots, qsl, taken = [], [0], begin
    for s, (c, n) in enumerate(zip(cached, new)):
        for p in range(c, c + n):
            if p % bs == 0:
                tables[s, p // bs] = free[taken]
                taken += 1
            slots.append(int(tables[s, p // bs]) * bs + p % bs)
        qsl.append(qsl[-1] + n)
    slots += [-1] * (room - len(slots))
    return tables, np.add(cached, new), np.array(qsl), np.array(slots, np.int64), taken


def dev(a, dt=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda").to(dt)


def setup(cached, new, bs, seed, room=None, begin=0, short=0):
    r = np.random.Generator(np.random.PCG64(seed))
    cached, new = np.asarray(cached), np.asarray(new)
    held, after = -(-cached // bs), -(-(cached + new) // bs)
    need = int((after - held).sum())
    perm = r.permutation(int(held.sum()) + need + 9).astype(np.int32)
    tables = np.full((len(cached), max(1, int(after.max(initial=1))) + 2), -1, np.int32)
    at = 0
    for s, h in enumerate(held):
        tables[s, :h] = perm[at:at + h]
        at += h
    free = np.concatenate([np.full(begin, -5, np.int32), perm[at:at + need - short]]) if short else \
        np.concatenate([np.full(begin, -5, np.int32), perm[at:]])
    room = int(new.sum()) if room is None else room
    return tables, cached, new, free, len(perm), room


def call(tables, cached, new, free, begin, NB, room, bs, in_place=False):
    S = len(cached)
    t = dev(tables)
    c, n = dev(cached), dev(new)
    b = dev([begin])
    ctx = c if in_place else torch.full((S,), 77, dtype=torch.int32, device="cuda")
    end = b if in_place else torch.full((1,), 77, dtype=torch.int32, device="cuda")
    qsl = torch.full((S + 1,), 77, dtype=torch.int32, device="cuda")
    slots = torch.full((room,), 77, dtype=torch.int64, device="cuda")
    pkv.step_metadata(t, ctx, qsl, slots, end, c, n, dev(free), b, NB, bs)
    return [x.cpu().numpy() for x in (t, ctx, qsl, slots, end)]


@pytest.mark.parametrize("bs", [8, 16, 32, 64])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("name", ["one", "decode", "chunks", "idle", "many", "long"])
def test_against_the_restatement(name, bs, in_place):
    r = np.random.Generator(np.random.PCG64(len(name)))
    cached, new = {
        "one": ([0], [1]),
        "decode": (r.integers(0, 300, 128), np.ones(128, int)),
        "chunks": (r.integers(0, 2000, 50), r.integers(0, 600, 50)),
        "idle": ([0, 5, 0, 16, 31], [0, 0, 0, 0, 0]),
        "many": (r.integers(0, 40, 5000), r.integers(0, 3, 5000)),
        "long": ([17, 3], [40000, 1]),
    }[name]
    tables, cached, new, free, NB, room = setup(cached, new, bs, 3, begin=4)
    room += 5
    want = plain(tables, cached, new, free, 4, room, bs)
    got = call(tables, cached, new, free, 4, NB, room, bs, in_place)
    assert pkv.get_device_error() == 0
    for g, w in zip(got, want):
        assert np.array_equal(g.reshape(-1), np.asarray(w).reshape(-1))


def test_agrees_with_the_host_slot_mapping():
    tables, cached, new, free, NB, room = setup([3, 16, 40], [20, 1, 9], 16, 5)
    got = call(tables, cached, new, free, 0, NB, room, 16)
    seq = np.repeat(np.arange(3), new).astype(np.int32)
    pos = np.concatenate([np.arange(c, c + n) for c, n in zip(cached, new)]).astype(np.int32)
    assert np.array_equal(got[3], pkv.slot_mapping(got[0], seq, pos, 16))


@pytest.mark.parametrize("case", ["tokens", "blocks", "begin"])
def test_a_step_that_does_not_fit_is_refused_whole(case):
    cached, new = [3, 16, 40], [20, 1, 9]
    tables, cached, new, free, NB, room = setup(cached, new, 16, 5, short=1 if case == "blocks" else 0)
    begin = 0
    if case == "tokens":
        room -= 1
    if case == "begin":
        begin = len(free) + 1
    t, ctx, qsl, slots, end = call(tables, cached, new, free, begin, NB, room, 16)
    assert pkv.get_device_error() == (pkv.DEVERR_QUERY_LEN if case == "tokens" else pkv.DEVERR_FREE_BLOCKS)
    assert np.array_equal(t, tables) and np.array_equal(ctx, cached)
    assert not qsl.any() and (slots == -1).all() and end[0] == begin


def test_bad_sequences_take_no_part():
    tables, cached, new, free, NB, room = setup([3, 16, 40, 8], [20, 1, 9, 1], 16, 5)
    new2 = new.copy()
    new2[1] = -4
    got = call(tables, cached, new2, free, 0, NB, room, 16)
    assert pkv.get_device_error() == pkv.DEVERR_QUERY_LEN
    new2[1] = 0
    want = plain(tables, cached, new2, free, 0, room, 16)
    for g, w in zip(got, want):
        assert np.array_equal(g.reshape(-1), np.asarray(w).reshape(-1))
    new2[1] = 10 ** 6  # past its table row
    got = call(tables, cached, new2, free, 0, NB, room, 16)
    assert pkv.get_device_error() == pkv.DEVERR_CONTEXT_LEN
    for g, w in zip(got, want):
        assert np.array_equal(g.reshape(-1), np.asarray(w).reshape(-1))


def test_block_ids_outside_the_pool_are_flagged():
    tables, cached, new, free, NB, room = setup([3, 16], [1, 1], 16, 5)
    free[0] = NB            # opened by the second sequence
    t, ctx, qsl, slots, end = call(tables, cached, new, free, 0, NB, room, 16)
    assert pkv.get_device_error() == pkv.DEVERR_BLOCK_ID
    assert t[1, 1] == -1 and slots[1] == -1 and slots[0] == tables[0, 0] * 16 + 3
    tables[0, 0] = -3       # held by the first
    free[0] = 1
    t, ctx, qsl, slots, end = call(tables, cached, new, free, 0, NB, room, 16)
    assert pkv.get_device_error() == pkv.DEVERR_BLOCK_ID
    assert slots[0] == -1 and slots[1] == 16


def test_a_replayed_decode_loop_advances_itself():
    """Metadata, cache write and absorbed attention captured once; each replay adds a token to
    every live sequence.  Compared with the same steps from host-built metadata."""
    from pagedattention_paged_kv_gb300.graph import CapturedStep
    S, H, R, P, bs, steps = 5, 16, 256, 64, 16, 40
    start = [0, 15, 16, 100, 0]
    live = [1, 1, 1, 1, 0]   # the last slot is empty
    NB = 64
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    cache = torch.randn(NB, bs, R + P, device="cuda", generator=g).bfloat16()
    ref_cache = cache.clone()
    ids = np.random.Generator(np.random.PCG64(2)).permutation(NB).astype(np.int32)
    tables = np.full((S, 12), -1, np.int32)
    at = 0
    for s, c in enumerate(start):
        n = -(-c // bs)
        tables[s, :n] = ids[at:at + n]
        at += n
    free = ids[at:]
    t, lens, new, fr = dev(tables), dev(start), dev(live), dev(free)
    taken = dev([0])
    qsl = torch.zeros(S + 1, dtype=torch.int32, device="cuda")
    slots = torch.zeros(S, dtype=torch.int64, device="cuda")
    lat, rope, q = (torch.zeros(S, n, dtype=torch.bfloat16, device="cuda") for n in (R, P, H * (R + P)))
    q = q.view(S, H, R + P)
    out = torch.zeros(S, H, R, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(pkv.latent_workspace_size(pkv.OP_LATENT_ABSORBED, S, S, H, R, P), dtype=torch.uint8, device="cuda")

    def step():
        pkv.step_metadata(t, lens, qsl, slots, taken, lens, new, fr, taken, NB, bs)
        pkv.latent_cache_write(cache, lat, rope, slots)
        pkv.latent_attention_absorbed(out, q, cache, t, lens, 0.07, query_start_loc=qsl, workspace=ws)

    saved = [x.clone() for x in (t, lens, taken, cache)]
    cap = CapturedStep(step, warmup=1)  # the warm-up advanced the state: put it back
    torch.cuda.synchronize()
    for x, y in zip((t, lens, taken, cache), saved):
        x.copy_(y)
    host_tables, host_len, host_at = tables.copy(), list(start), 0
    for i in range(steps):
        vals = [torch.randn(*x.shape, device="cuda", generator=g).bfloat16() for x in (lat, rope, q)]
        for x, y in zip((lat, rope, q), vals):
            x.copy_(y)
        torch.cuda.synchronize()
        cap.replay()
        cap.synchronize()
        # the same step with host metadata
        for s in range(S):
            if live[s]:
                if host_len[s] % bs == 0:
                    host_tables[s, host_len[s] // bs] = free[host_at]
                    host_at += 1
                host_len[s] += 1
        n = sum(live)
        pos = np.array([host_len[s] - 1 for s in range(S) if live[s]], np.int32)
        sl = pkv.slot_mapping(host_tables, np.arange(n, dtype=np.int32), pos, bs)
        pkv.latent_cache_write(ref_cache, vals[0][:n].contiguous(), vals[1][:n].contiguous(), dev(sl, torch.int64))
        want = torch.empty(n, H, R, dtype=torch.bfloat16, device="cuda")
        pkv.latent_attention_absorbed(want, vals[2][:n].contiguous(), ref_cache, dev(host_tables[:n]),
                                      dev(host_len[:n]), 0.07)
        assert torch.equal(out[:n], want)
        assert np.array_equal(t.cpu().numpy(), host_tables) and lens.tolist() == host_len
    assert int(taken) == host_at
    assert pkv.get_device_error() == 0
    assert torch.equal(cache.view(torch.int16), ref_cache.view(torch.int16))
