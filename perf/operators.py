"""Cases of the latent-attention operators and of the GPU-built step metadata.

Four operators, as a serving loop strings them together on one stream:

  step_metadata              context lengths, query offsets, block tables and slot map of a
                             step, built on the GPU from the lengths of the requests
  latent_cache_write         a token's latent row and rotary key row into its slot of the
                             block-paged latent cache
  latent_attention_absorbed  attention over that cache with the key and value projections
                             folded into the query and the output (single tokens, and the few
                             tokens of a verification step)
  latent_attention_expanded  attention with per-head keys and values expanded from the cached
                             latents (prompts and prompt chunks)

With ``own`` false, run() is the plain form: elementary torch operations in 32 bits.  With
``own`` true it makes this package's calls.  Sequence lengths follow a case's own
``lens_seed``; block placement and every value follow prepare()'s seed.
"""
from __future__ import annotations

import math
import random

import numpy as np
import torch

own = False

ROPE = 64       # rotary columns of a cached row and of a query
NOPE = 128      # columns of an expanded key that carry no rotary part
VDIM = 128      # columns of an expanded value


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # the four short requests of the tiny decode workload: one step's metadata, pure latency
        dict(name="step_tiny", op="step", seqs=4, ctx_lo=1, ctx_hi=100, chunks=0, chunk=0, block_size=16,
             table=16, lens_seed=11),
        # 128 running requests, one token each
        dict(name="step_decode_128", op="step", seqs=128, ctx_lo=500, ctx_hi=2500, chunks=0, chunk=0,
             block_size=16, table=512, lens_seed=12),
        # a large batch in which 64 requests bring a 512-token chunk
        dict(name="step_chunks_1024", op="step", seqs=1024, ctx_lo=1, ctx_hi=4000, chunks=64, chunk=512,
             block_size=16, table=512, lens_seed=13),
        # the new rows of 128 decoding requests
        dict(name="write_decode_128", op="write", tokens=128, blocks=13000, block_size=16, latent=512,
             padding=0.0, lens_seed=21),
        # a padded batch of prompt chunks
        dict(name="write_chunks_32k", op="write", tokens=32771, blocks=4096, block_size=16, latent=512,
             padding=0.05, lens_seed=22),
        # four short requests, heads of one small model: latency
        dict(name="absorbed_tiny", op="absorbed", seqs=4, ctx_lo=1, ctx_hi=100, long=0, long_ctx=0, q_lo=1,
             q_hi=1, heads=16, latent=256, block_size=16, lens_seed=31),
        # one layer's decode step of 128 requests with 64 heads
        dict(name="absorbed_decode_128", op="absorbed", seqs=128, ctx_lo=500, ctx_hi=2500, long=0, long_ctx=0,
             q_lo=1, q_hi=1, heads=64, latent=512, block_size=16, lens_seed=32),
        # four 32k contexts among short ones, 16 heads (a head-sharded layer)
        dict(name="absorbed_skewed_64", op="absorbed", seqs=64, ctx_lo=256, ctx_hi=2048, long=4, long_ctx=32768,
             q_lo=1, q_hi=1, heads=16, latent=512, block_size=16, lens_seed=33),
        # verification of a few drafted tokens a request, 128 heads
        dict(name="absorbed_verify_32", op="absorbed", seqs=32, ctx_lo=257, ctx_hi=8191, long=0, long_ctx=0,
             q_lo=1, q_hi=4, heads=128, latent=512, block_size=16, lens_seed=34),
        # short ragged prompts without a prefix, 16 heads
        dict(name="expanded_short_16", op="expanded", seqs=16, pre_lo=0, pre_hi=0, q_lo=1, q_hi=300, heads=16,
             latent=256, block_size=16, lens_seed=41),
        # one 512-token chunk of a long prompt behind a 16k prefix, 64 heads
        dict(name="expanded_chunk_16k", op="expanded", seqs=1, pre_lo=16384, pre_hi=16384, q_lo=512, q_hi=512,
             heads=64, latent=512, block_size=16, lens_seed=42),
        # eight whole prompts at once, 64 heads
        dict(name="expanded_prompts_8", op="expanded", seqs=8, pre_lo=0, pre_hi=0, q_lo=500, q_hi=2500, heads=64,
             latent=512, block_size=16, lens_seed=43),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the listed ranges (`rng`: random.Random)."""
    most = {op: max(_cost(c) for c in listed() if c["op"] == op) for op in ("step", "write", "absorbed", "expanded")}
    op = rng.choice(["step", "write", "absorbed", "absorbed", "expanded", "expanded"])
    while True:
        c = dict(op=op, block_size=rng.choice([8, 16, 32, 64]), lens_seed=rng.randrange(1 << 30))
        if op == "step":
            seqs = _log_int(rng, 1, 1024)
            hi = _log_int(rng, 1, 6000)
            c.update(seqs=seqs, ctx_lo=rng.randint(0, hi), ctx_hi=hi, chunks=rng.randint(0, min(seqs, 64)),
                     chunk=_log_int(rng, 2, 512), table=-(-(hi + 512) // c["block_size"]) + rng.randint(0, 33))
        elif op == "write":
            tokens = _log_int(rng, 1, 32771)
            c.update(tokens=tokens, blocks=-(-tokens // c["block_size"]) + _log_int(rng, 1, 3000),
                     latent=rng.choice([256, 512]), padding=rng.choice([0.0, 0.05, 0.5]))
        elif op == "absorbed":
            hi = _log_int(rng, 1, 16384)
            q_lo = rng.choice([1, 1, 1, rng.randint(0, 4)])
            c.update(seqs=_log_int(rng, 1, 256), ctx_lo=rng.randint(1, hi), ctx_hi=hi, long=rng.choice([0, 0, 1, 3]),
                     long_ctx=rng.randint(4096, 32768), q_lo=q_lo, q_hi=q_lo + rng.choice([0, 0, 0, rng.randint(1, 7)]),
                     heads=rng.choice([1, 5, 8, 16, 24, 32, 40, 64, 96, 128]), latent=rng.choice([256, 512]))
        else:
            hi = _log_int(rng, 1, 4096)
            pre = rng.choice([0, 0, _log_int(rng, 1, 16384)])
            c.update(seqs=_log_int(rng, 1, 24), pre_lo=rng.randint(0, pre), pre_hi=pre, q_lo=rng.randint(0, hi),
                     q_hi=hi, heads=rng.choice([1, 3, 8, 16, 32, 64, 128]), latent=rng.choice([256, 512]))
        if _cost(c) <= most[op]:
            return c


def _lens(case):
    """(tokens already cached, tokens of this step) of every sequence of a case."""
    r = np.random.Generator(np.random.PCG64(case["lens_seed"]))
    S = case.get("seqs", 0)
    if case["op"] == "step":
        cached = r.integers(case["ctx_lo"], case["ctx_hi"] + 1, size=S)
        new = np.ones(S, dtype=np.int64)
        if case["chunks"]:
            new[r.permutation(S)[:case["chunks"]]] = case["chunk"]
        return cached, new
    if case["op"] == "absorbed":
        ctx = r.integers(case["ctx_lo"], case["ctx_hi"] + 1, size=S)
        q = r.integers(case["q_lo"], case["q_hi"] + 1, size=S)
        if case["long"]:
            ctx[r.permutation(S)[:case["long"]]] = case["long_ctx"]
        q = np.minimum(q, ctx)
        q[0] = max(q[0], 1)  # a step has at least one token
        return ctx - q, q
    pre, q = (r.integers(case[k + "_lo"], case[k + "_hi"] + 1, size=S) for k in ("pre", "q"))
    q[0] = max(q[0], 1)
    return pre, q


def _visible(pre, q):
    """(query, key) pairs under the causal mask."""
    return int((pre * q + q * (q + 1) // 2).sum())


def work(case):
    op = case["op"]
    if op == "step":
        cached, new = _lens(case)
        bs = case["block_size"]
        need = int((-(-(cached + new) // bs) + (-cached // bs)).sum())
        S, T = len(new), int(new.sum())
        # lengths in; offsets, contexts, new table entries (read from the free list, written) and slots out;
        # a sequence whose first new token falls into a block it holds reads that block's id
        held = int(((new > 0) & (cached % bs != 0)).sum())
        return {"bytes": 4 * (2 * S + (S + 1) + S + 2 + 2 * need + held) + 8 * T, "flops": 0}
    if op == "write":
        row = 2 * (case["latent"] + ROPE)
        kept = case["tokens"] - int(round(case["padding"] * case["tokens"]))
        return {"bytes": 2 * row * kept + 8 * case["tokens"], "flops": 0}
    pre, q = _lens(case)
    ctx, H, R = pre + q, case["heads"], case["latent"]
    live = ctx[q > 0]
    T, pairs = int(q.sum()), _visible(pre, q)
    kv = int(live.sum()) * (R + ROPE) * 2 + int((-(-live // case["block_size"])).sum()) * 4 + 8 * len(q)
    if op == "absorbed":
        return {"bytes": kv + T * H * (R + ROPE) * 2 + T * H * R * 2, "flops": 2 * pairs * H * (2 * R + ROPE)}
    # expanded: the per-head keys and values of every visible token, then the attention over them
    return {"bytes": kv + H * (NOPE + VDIM) * R * 2 + T * H * (NOPE + ROPE) * 2 + T * H * VDIM * 2,
            "flops": 2 * int(live.sum()) * H * (NOPE + VDIM) * R + 2 * pairs * H * (NOPE + ROPE + VDIM)}


def _cost(case):
    w = work(case)
    return w["bytes"] / 6e12 + w["flops"] / 1.5e15


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def _inputs(case, seed):
    """What a serving program has in hand before the call, from the seed alone."""
    dev = _device()
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    r = np.random.Generator(np.random.PCG64([seed, case["lens_seed"]]))
    op, bs = case["op"], case["block_size"]

    def normal(*shape, std=1.0):
        return (torch.randn(shape, generator=g, device=dev, dtype=torch.float32) * std).to(torch.bfloat16)

    def ints(a, dt=torch.int32):
        return torch.from_numpy(np.ascontiguousarray(a)).to(dev).to(dt)

    if op == "write":
        R, NB, T = case["latent"], case["blocks"], case["tokens"]
        slots = r.permutation(NB * bs)[:T].astype(np.int64)
        slots[r.permutation(T)[:int(round(case["padding"] * T))]] = -1
        return dict(cache=normal(NB, bs, R + ROPE), latent=normal(T, R), rope=normal(T, ROPE),
                    slots=ints(slots, torch.int64))
    pre, q = _lens(case)
    S = len(q)
    ctx = pre + q
    if op == "step":
        held = -(-pre // bs)
        need = -(-ctx // bs) - held
        NB = int(held.sum() + need.sum()) + 64
        perm = r.permutation(NB).astype(np.int32)
        tables = np.full((S, case["table"]), -1, np.int32)
        at = 0
        for s in range(S):
            tables[s, :held[s]] = perm[at:at + held[s]]
            at += held[s]
        begin = int(r.integers(0, 7))
        free = np.concatenate([np.zeros(begin, np.int32), perm[at:]])
        return dict(tables=ints(tables), cached=ints(pre), new=ints(q), free=ints(free), begin=ints([begin]),
                    num_blocks=NB, tokens=int(q.sum()) + case["lens_seed"] % 9)  # a little room in the slot map
    R, H = case["latent"], case["heads"]
    blocks = -(-ctx // bs)
    NB = int(blocks.sum() * 1.1) + 1
    perm = r.permutation(NB).astype(np.int32)
    tables = np.full((S, max(1, int(blocks.max()))), -1, np.int32)
    at = 0
    for s in range(S):
        tables[s, :blocks[s]] = perm[at:at + blocks[s]]
        at += blocks[s]
    T = int(q.sum())
    d = dict(cache=normal(NB, bs, R + ROPE), tables=ints(tables), ctx=ints(ctx),
             qsl=ints(np.concatenate([[0], np.cumsum(q)])), host_ctx=ctx.tolist(), host_q=q.tolist(),
             # the softmax scale of the unabsorbed head: its key has NOPE + ROPE columns
             scale=1.0 / math.sqrt(NOPE + ROPE), single=bool((q == 1).all()))
    if op == "absorbed":
        d["q"] = normal(T, H, R + ROPE)
    else:
        d["q"] = normal(T, H, NOPE + ROPE)
        # projections that keep unit variance: keys and values of N(0, 1) from latents of N(0, 1)
        d["w_k"], d["w_v"] = normal(H, NOPE, R, std=R ** -0.5), normal(H, VDIM, R, std=R ** -0.5)
    return d


def prepare(case, seed):
    d = _inputs(case, seed)
    dev, op = _device(), case["op"]
    d["op"] = op
    if op == "step":
        S = d["new"].shape[0]
        d.update(context_lens=torch.empty(S, dtype=torch.int32, device=dev),
                 query_start_loc=torch.empty(S + 1, dtype=torch.int32, device=dev),
                 slots=torch.empty(d["tokens"], dtype=torch.int64, device=dev),
                 free_end=torch.empty(1, dtype=torch.int32, device=dev), bs=case["block_size"])
    elif op in ("absorbed", "expanded"):
        T, H = d["q"].shape[0], d["q"].shape[1]
        d["out"] = torch.empty(T, H, case["latent"] if op == "absorbed" else VDIM, dtype=torch.bfloat16, device=dev)
        if own:
            import pagedattention_paged_kv_gb300 as pkv
            S = len(d["host_q"])
            if op == "absorbed":
                n = pkv.latent_workspace_size(pkv.OP_LATENT_ABSORBED, S, T, H, case["latent"], ROPE)
            else:
                d["total_context"] = sum(d["host_ctx"])
                n = pkv.latent_workspace_size(pkv.OP_LATENT_EXPANDED, S, T, H, case["latent"], ROPE,
                                              total_context=d["total_context"])
            d["ws"] = torch.empty(n, dtype=torch.uint8, device=dev)
    return d


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(st):
    import pagedattention_paged_kv_gb300 as pkv
    op = st["op"]
    if op == "step":
        pkv.step_metadata(st["tables"], st["context_lens"], st["query_start_loc"], st["slots"], st["free_end"],
                          st["cached"], st["new"], st["free"], st["begin"], st["num_blocks"], st["bs"])
        return [st[k] for k in ("tables", "context_lens", "query_start_loc", "slots", "free_end")]
    if op == "write":
        pkv.latent_cache_write(st["cache"], st["latent"], st["rope"], st["slots"])
        return st["cache"]
    if op == "absorbed":
        pkv.latent_attention_absorbed(st["out"], st["q"], st["cache"], st["tables"], st["ctx"], st["scale"],
                                      query_start_loc=None if st["single"] else st["qsl"], workspace=st["ws"])
        return st["out"]
    pkv.latent_attention_expanded(st["out"], st["q"], st["qsl"], st["cache"], st["tables"], st["ctx"], st["w_k"],
                                  st["w_v"], st["scale"], total_context=st["total_context"], workspace=st["ws"])
    return st["out"]


def _run_plain(st):
    return {"step": _plain_step, "write": _plain_write, "absorbed": _plain_absorbed,
            "expanded": _plain_expanded}[st["op"]](st)


def _plain_step(st):
    bs, tables, T = st["bs"], st["tables"], st["tokens"]
    dev = tables.device
    cached, new = st["cached"].long(), st["new"].long()
    S, MB = tables.shape
    ctx = cached + new
    held, blocks = (cached + bs - 1) // bs, (ctx + bs - 1) // bs
    need = blocks - held
    first = st["begin"].long() + torch.cumsum(need, 0) - need
    cols = torch.arange(MB, device=dev)
    fresh = (cols >= held[:, None]) & (cols < blocks[:, None])
    at = (first[:, None] + cols - held[:, None]).clamp(0, max(0, st["free"].shape[0] - 1))
    ids = st["free"][at] if st["free"].shape[0] else torch.zeros_like(tables)
    tables.copy_(torch.where(fresh, ids, tables))
    qsl = torch.cat([torch.zeros(1, dtype=torch.long, device=dev), torch.cumsum(new, 0)])
    t = torch.arange(T, device=dev)
    s = (torch.searchsorted(qsl, t, right=True) - 1).clamp(0, S - 1)
    pos = cached[s] + t - qsl[s]
    live = t < qsl[-1]
    block = tables[s, torch.where(live, pos // bs, torch.zeros_like(pos))].long()
    slots = torch.where(live, block * bs + pos % bs, torch.full_like(pos, -1))
    return [tables, ctx.to(torch.int32), qsl.to(torch.int32), slots,
            (st["begin"] + need.sum()).to(torch.int32)]


def _plain_write(st):
    cache, slots = st["cache"], st["slots"]
    flat = cache.view(-1, cache.shape[-1])
    rows = torch.cat([st["latent"], st["rope"]], dim=1)
    kept = slots >= 0
    flat[slots[kept]] = rows[kept]
    return cache


def _gather(st, seqs, width):
    """Cached rows 0 .. width - 1 of the sequences, in 32 bits: [n, width, row]."""
    bs = st["cache"].shape[1]
    pos = torch.arange(width, device=st["cache"].device)
    ids = st["tables"][seqs][:, pos // bs].clamp(min=0).long()
    return st["cache"][ids, pos % bs].float()


def _groups(st, per_token):
    """Runs of neighbouring sequences whose padded intermediates stay near 2 GB."""
    at, S = 0, len(st["host_q"])
    while at < S:
        end, width, rows = at, 0, 0
        while end < S:
            w, r = max(width, st["host_ctx"][end]), max(rows, st["host_q"][end])
            if end > at and (end + 1 - at) * w * max(1, per_token(r)) > 5e8:
                break
            end, width, rows = end + 1, w, r
        yield range(at, end), width, rows
        at = end


def _padded_queries(st, seqs, rows):
    """Queries of the sequences padded to `rows` rows each, and the flat rows they came from."""
    dev = st["q"].device
    qsl = st["qsl"].long()
    start, n = qsl[seqs.start:seqs.stop], qsl[seqs.start + 1:seqs.stop + 1] - qsl[seqs.start:seqs.stop]
    j = torch.arange(rows, device=dev)
    live = j < n[:, None]
    at = torch.where(live, start[:, None] + j, torch.zeros_like(start[:, None] + j))
    return st["q"][at].float(), live, at, n


def _mask(st, seqs, width, rows, n):
    """[n, rows, width]: keys that each padded query row may see."""
    dev = st["q"].device
    ctx = st["ctx"][seqs.start:seqs.stop].long()
    last = ctx[:, None] - n[:, None] + torch.arange(rows, device=dev)
    return torch.arange(width, device=dev) <= last[:, :, None]


def _softmax(scores, seen):
    scores = scores.masked_fill_(~seen, float("-inf"))
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    return p / torch.where(total == 0, torch.ones_like(total), total)


def _plain_absorbed(st):
    out, R, H = torch.zeros_like(st["out"]), st["out"].shape[-1], st["q"].shape[1]
    for seqs, width, rows in _groups(st, lambda r: st["cache"].shape[-1] + 2 * r * H):
        if rows == 0:
            continue
        kv = _gather(st, seqs, width)
        q, live, at, n = _padded_queries(st, seqs, rows)
        m = q.shape[0]
        s = torch.bmm(q.reshape(m, rows * H, -1), kv.transpose(1, 2)).view(m, rows, H, width) * st["scale"]
        p = _softmax(s, _mask(st, seqs, width, rows, n)[:, :, None, :])
        o = torch.bmm(p.view(m, rows * H, width), kv[..., :R]).view(m, rows, H, R)
        out[at[live]] = o[live].to(out.dtype)
    return out


def _plain_expanded(st):
    out, H = torch.zeros_like(st["out"]), st["q"].shape[1]
    R = st["w_k"].shape[-1]
    w_k, w_v = st["w_k"].float().reshape(-1, R), st["w_v"].float().reshape(-1, R)
    for s, (c, n) in enumerate(zip(st["host_ctx"], st["host_q"])):
        if n == 0:
            continue
        kv = _gather(st, range(s, s + 1), c)[0]
        k = torch.cat([(kv[:, :R] @ w_k.t()).view(c, H, NOPE), kv[:, None, R:].expand(c, H, ROPE)], dim=-1)
        v = (kv[:, :R] @ w_v.t()).view(c, H, VDIM).transpose(0, 1)
        lo = sum(st["host_q"][:s])
        q = st["q"][lo:lo + n].float().transpose(0, 1)
        seen = torch.arange(c, device=q.device) <= (c - n + torch.arange(n, device=q.device))[:, None]
        step = max(1, int(5e8 // (n * c)))  # heads at once: scores near 2 GB
        for h in range(0, H, step):
            p = torch.bmm(q[h:h + step], k.transpose(0, 1)[h:h + step].transpose(1, 2)) * st["scale"]
            p = _softmax(p, seen)
            out[lo:lo + n, h:h + step] = torch.bmm(p, v[h:h + step]).transpose(0, 1).to(out.dtype)
    return out


# ---------------------------------------------------------------------------
# the definition, in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    """What run() returns for these inputs, from the operators' definitions: one sequence, one
    token and one head after the other where that is affordable, in 64 bits."""
    d = _inputs(case, seed)
    op = case["op"]
    if op == "step":
        bs = case["block_size"]
        tables, free = d["tables"].cpu().numpy().copy(), d["free"].cpu().numpy()
        taken = int(d["begin"][0])
        ctx, qsl, slots = [], [0], []
        for s, (c, n) in enumerate(zip(d["cached"].tolist(), d["new"].tolist())):
            for p in range(c, c + n):
                if p % bs == 0:  # the first token of a block takes the next free one
                    tables[s, p // bs] = free[taken]
                    taken += 1
                slots.append(int(tables[s, p // bs]) * bs + p % bs)
            ctx.append(c + n)
            qsl.append(qsl[-1] + n)
        slots += [-1] * (d["tokens"] - len(slots))
        return [tables, np.array(ctx, np.int32), np.array(qsl, np.int32), np.array(slots, np.int64),
                np.array([taken], np.int32)]
    if op == "write":
        bs = case["block_size"]
        cache = d["cache"].double()
        R = case["latent"]
        keep = [(t, s) for t, s in enumerate(d["slots"].tolist()) if s >= 0]
        if keep:
            t = torch.tensor([k[0] for k in keep], device=cache.device)
            b = torch.tensor([k[1] // bs for k in keep], device=cache.device)
            o = torch.tensor([k[1] % bs for k in keep], device=cache.device)
            cache[b, o, :R] = d["latent"][t].double()
            cache[b, o, R:] = d["rope"][t].double()
        return cache
    pre, q = _lens(case)
    if (work(case)["flops"] if torch.cuda.is_available() else 60 * work(case)["flops"]) > 8e12:
        return None
    R, H, bs = case["latent"], case["heads"], case["block_size"]
    out = torch.zeros(d["q"].shape[0], H, R if op == "absorbed" else VDIM, dtype=torch.float64, device=d["q"].device)
    row = 0
    for s in range(len(q)):
        n, c = int(q[s]), int(pre[s] + q[s])
        if n == 0:
            continue
        blocks = d["tables"][s, :-(-c // bs)].long()
        rows = d["cache"][blocks].reshape(-1, R + ROPE)[:c].double()
        # later queries see more keys: tokens in runs, each cut at its own last position
        for a in range(0, n, 64):
            e = min(n, a + 64)
            see = c - n + e
            hidden = torch.ones(e - a, see, dtype=torch.bool, device=rows.device).triu(see - (e - a) + 1)
            for h in range(0, H, 16):
                qq = d["q"][row + a:row + e, h:h + 16].double()
                if op == "absorbed":
                    sc = torch.einsum("thd,kd->htk", qq, rows[:see])
                    val = rows[:see, :R].expand(qq.shape[1], see, R)
                else:
                    if a == 0:  # this sequence's keys and values of these heads
                        kk = torch.einsum("kr,hdr->hkd", rows[:, :R], d["w_k"][h:h + 16].double())
                        vv = torch.einsum("kr,hdr->hkd", rows[:, :R], d["w_v"][h:h + 16].double())
                        _exact_kv[h] = (kk, vv)
                    kk, vv = _exact_kv[h]
                    sc = torch.einsum("thd,hkd->htk", qq[..., :NOPE], kk[:, :see])
                    sc += torch.einsum("thd,kd->htk", qq[..., NOPE:], rows[:see, R:])
                    val = vv[:, :see]
                w = torch.softmax((sc * d["scale"]).masked_fill(hidden, -math.inf), -1)
                out[row + a:row + e, h:h + 16] = torch.einsum("htk,hkd->thd", w, val)
        row += n
    _exact_kv.clear()
    return out


_exact_kv: dict = {}
