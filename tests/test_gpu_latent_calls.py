"""The latent-attention calls as a program uses them: what the binding refuses, workspaces, two
streams at once, graphs that share a workspace, waits that run out, and a prompt followed by a
decode loop."""
import pytest
import torch

import pagedattention_paged_kv_gb300 as pkv
from latent_helpers import ROPE, SCALE, Batch, absorbed_reference, attend, check, expanded_reference
from pagedattention_paged_kv_gb300.graph import CapturedStep

pytestmark = pytest.mark.gpu


def weights(heads, latent, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return [(torch.randn(heads, 128, latent, device="cuda", generator=g) * latent ** -0.5).bfloat16() for _ in range(2)]


def absorbed(b, out=None, **kw):
    out = torch.full((b.q.shape[0], b.heads, b.latent), float("nan"), dtype=torch.bfloat16, device="cuda") \
        if out is None else out
    pkv.latent_attention_absorbed(out, b.q, b.cache, b.tables, b.context_lens, SCALE, query_start_loc=b.qsl, **kw)
    return out


def expanded(b, w, out=None, **kw):
    out = torch.full((b.q.shape[0], b.heads, 128), float("nan"), dtype=torch.bfloat16, device="cuda") \
        if out is None else out
    pkv.latent_attention_expanded(out, b.q, b.qsl, b.cache, b.tables, b.context_lens, *w, SCALE, sum(b.ctx), **kw)
    return out


def workspace(op, b):
    n = pkv.latent_workspace_size(op, len(b.ctx), b.q.shape[0], b.heads, b.latent, ROPE,
                                  total_context=sum(b.ctx))
    return torch.empty(n, dtype=torch.uint8, device="cuda")


def test_the_binding_refuses_what_does_not_fit():
    b = Batch([40, 9], [2, 1], 8, 256, 256 + ROPE)
    out = torch.zeros(3, 8, 256, dtype=torch.bfloat16, device="cuda")
    args = [out, b.q, b.cache, b.tables, b.context_lens]

    def refused(error, at, value, **kw):
        a = list(args)
        a[at] = value
        with pytest.raises(error):
            pkv.latent_attention_absorbed(*a, SCALE, query_start_loc=b.qsl, **kw)

    refused(ValueError, 0, out.float())                              # type
    refused(ValueError, 0, out.cpu())                                # device
    refused(ValueError, 0, None)
    refused(ValueError, 0, out[:2])                                  # rows
    refused(ValueError, 1, b.q.transpose(0, 1))                      # strides
    refused(ValueError, 1, b.q[..., :256].contiguous())              # no rotary columns
    refused(ValueError, 3, b.tables[:1])                             # sequences
    refused(ValueError, 3, b.tables.long())
    refused(ValueError, 4, b.context_lens[:1])
    refused(pkv.PagedKVError, 0, out[..., :128].contiguous())        # a latent width that is not built
    ws = workspace(pkv.OP_LATENT_ABSORBED, b)
    refused(pkv.PagedKVError, 0, out, workspace=ws[:-1])             # too small
    refused(ValueError, 0, out, workspace=ws.cpu())
    big = torch.empty(ws.numel() + 256, dtype=torch.uint8, device="cuda")
    refused(pkv.PagedKVError, 0, out, workspace=big[16:])            # not 256-byte aligned
    with pytest.raises(ValueError):
        pkv.latent_attention_absorbed(*args, SCALE)                  # one row a sequence without offsets
    e = Batch([40, 9], [2, 1], 8, 256, 128 + ROPE)
    w = weights(8, 256, 1)
    eo = torch.zeros(3, 8, 128, dtype=torch.bfloat16, device="cuda")
    for bad in ((w[0][:4].contiguous(), w[1]), (w[0], w[1][..., :128].contiguous()), (w[0].float(), w[1]),
                (w[0][:, :64].contiguous(), w[1])):
        with pytest.raises(ValueError):
            expanded(e, bad, eo)
    with pytest.raises(pkv.PagedKVError):
        expanded(e, w, eo, workspace=workspace(pkv.OP_LATENT_EXPANDED, e)[:-1])
    with pytest.raises(ValueError):
        pkv.latent_cache_write(b.cache, torch.zeros(2, 256, dtype=torch.bfloat16, device="cuda"),
                               torch.zeros(2, 32, dtype=torch.bfloat16, device="cuda"),
                               torch.zeros(2, dtype=torch.int64, device="cuda"))
    assert pkv.get_device_error() == 0
    assert not out.any() and not eo.any()


def test_two_calls_at_once_on_two_streams():
    a = Batch([900, 77, 2000], [1, 1, 1], 32, 512, 512 + ROPE, seed=1)
    e = Batch([700, 300], [300, 300], 16, 512, 128 + ROPE, seed=2)
    w = weights(16, 512, 3)
    wa, we = workspace(pkv.OP_LATENT_ABSORBED, a), workspace(pkv.OP_LATENT_EXPANDED, e)
    alone = absorbed(a, workspace=wa), expanded(e, w, workspace=we)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    oa, oe = torch.zeros_like(alone[0]), torch.zeros_like(alone[1])
    torch.cuda.synchronize()
    for _ in range(8):
        absorbed(a, oa, workspace=wa, stream=s1)
        expanded(e, w, oe, workspace=we, stream=s2)
    torch.cuda.synchronize()
    assert pkv.get_device_error() == 0
    assert torch.equal(oa, alone[0]) and torch.equal(oe, alone[1])
    check(oa, *absorbed_reference(a))
    check(oe, *expanded_reference(e, *w))


def test_graphs_that_share_a_workspace():
    a = Batch([500, 33], [3, 1], 16, 256, 256 + ROPE, seed=4)
    e = Batch([500, 33], [300, 33], 16, 256, 128 + ROPE, seed=5)
    w = weights(16, 256, 6)
    want = absorbed(a), expanded(e, w)
    sizes = [workspace(pkv.OP_LATENT_ABSORBED, a), workspace(pkv.OP_LATENT_EXPANDED, e)]
    ws = max(sizes, key=lambda x: x.numel())
    oa, oe = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    stream = torch.cuda.Stream()
    ga = CapturedStep(lambda: absorbed(a, oa, workspace=ws), stream=stream)
    ge = CapturedStep(lambda: expanded(e, w, oe, workspace=ws), stream=stream)
    torch.cuda.synchronize()
    for _ in range(3):
        oa.zero_()
        oe.zero_()
        torch.cuda.synchronize()
        for g in (ga, ge, ga, ge, ge, ga):
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(oa, want[0]) and torch.equal(oe, want[1])
    assert pkv.get_device_error() == 0


@pytest.mark.parametrize("heads,latent", [(3, 256), (16, 512)])
def test_what_the_workspace_held_has_no_effect(heads, latent):
    """NaN everywhere in it, contexts around the sizes of tiles and chunks, room to spare."""
    ctx = [1, 95, 96, 97, 127, 128, 129, 191, 192, 193, 255, 256, 257, 288, 289, 384, 385, 500, 128]
    ql = [1, 95, 1, 97, 64, 128, 129, 2, 192, 193, 255, 256, 1, 288, 33, 384, 300, 257, 128]
    e = Batch(ctx, ql, heads, latent, 128 + ROPE, seed=11)
    w = weights(heads, latent, 12)
    n = pkv.latent_workspace_size(pkv.OP_LATENT_EXPANDED, len(ctx), e.q.shape[0], heads, latent, ROPE,
                                  total_context=sum(ctx) + 1000)
    for causal in (True, False):
        ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
        out = torch.full((e.q.shape[0], heads, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
        pkv.latent_attention_expanded(out, e.q, e.qsl, e.cache, e.tables, e.context_lens, *w, SCALE, sum(ctx) + 1000,
                                      causal=causal, workspace=ws)
        assert pkv.get_device_error() == 0
        check(out, *expanded_reference(e, *w, causal=causal), f"causal {causal}")
    a = Batch(ctx, ql, heads, latent, latent + ROPE, seed=13)
    ws = workspace(pkv.OP_LATENT_ABSORBED, a).fill_(0xFF)
    out = absorbed(a, workspace=ws)
    assert pkv.get_device_error() == 0
    check(out, *absorbed_reference(a))


@pytest.mark.parametrize("form", ["absorbed", "expanded"])
def test_a_wait_that_runs_out_flags_timeout_and_returns(form):
    cols = 512 if form == "absorbed" else 128
    b = Batch([2000, 1500, 3000, 10], [130, 1, 40, 10], 16, 512, cols + ROPE, seed=7, fill=0.0)
    w = weights(16, 512, 8)
    go = (lambda: absorbed(b)) if form == "absorbed" else (lambda: expanded(b, w))
    assert pkv.get_device_error() == 0
    flags = []
    try:
        pkv.set_wait_limit_ns(1)
        for _ in range(5):
            go()
            flags.append(pkv.get_device_error())
            if flags[-1] & pkv.DEVERR_TIMEOUT:
                break
    finally:
        pkv.set_wait_limit_ns(0)
    assert flags[-1] & pkv.DEVERR_TIMEOUT, f"no wait ran out: flags {flags}"
    # (a value computed from tiles that never came may also have been out of range)
    assert all(f & ~(pkv.DEVERR_TIMEOUT | pkv.DEVERR_VALUE) == 0 for f in flags), flags
    ref = absorbed_reference(b) if form == "absorbed" else expanded_reference(b, *w)
    out = go()
    assert pkv.get_device_error() == 0
    check(out, *ref)


def test_a_prompt_and_the_decode_steps_behind_it():
    """A small serving loop on device-built metadata: each step's latent rows are written through
    the step's own slot map, the prompts attend in the expanded form, the decode steps absorbed
    (a captured graph); every step against the attention of the definition in 64 bits."""
    H, R, bs, S, NB, steps = 8, 256, 16, 3, 40, 20
    prompt = [37, 150, 16]
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=g).bfloat16()
    w_k, w_v = weights(H, R, 10)
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    cache = torch.full((NB, bs, R + ROPE), float("nan"), dtype=torch.bfloat16, device="cuda")
    tables = torch.full((S, 16), -1, dtype=torch.int32, device="cuda")
    lens, taken, free = dev([0] * S), dev([0]), dev(torch.randperm(NB, generator=torch.Generator().manual_seed(1)).tolist())
    qsl = torch.zeros(S + 1, dtype=torch.int32, device="cuda")
    history = [torch.zeros(0, R + ROPE, dtype=torch.bfloat16, device="cuda") for _ in range(S)]

    def definition(q_parts):
        """out [sum n, H, 128] of the new positions, with the tolerance of keys and values kept exact."""
        outs, mags, scs = [], [], []
        for s, q in enumerate(q_parts):
            rows = history[s].double()
            k = torch.einsum("cr,hdr->hcd", rows[:, :R], w_k.double())
            v = torch.einsum("cr,hdr->hcd", rows[:, :R], w_v.double())
            k = torch.cat([k, rows[None, :, R:].expand(H, len(rows), ROPE)], -1)
            o, m, c = attend(q, k, v, len(q), SCALE, True)
            outs.append(o)
            mags.append(m)
            scs.append(c)
        return torch.cat(outs), torch.cat(mags), torch.cat(scs)

    # prompts
    T = sum(prompt)
    slots = torch.zeros(T, dtype=torch.int64, device="cuda")
    lat, rope, q = rnd(T, R), rnd(T, ROPE), rnd(T, H, 128 + ROPE)
    pkv.step_metadata(tables, lens, qsl, slots, taken, lens, dev(prompt), free, taken, NB, bs)
    pkv.latent_cache_write(cache, lat, rope, slots)
    out = torch.full((T, H, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    pkv.latent_attention_expanded(out, q, qsl, cache, tables, lens, w_k, w_v, SCALE, T)
    off = [0, prompt[0], prompt[0] + prompt[1], T]
    assert qsl.tolist() == off
    for s in range(S):
        history[s] = torch.cat([lat[off[s]:off[s + 1]], rope[off[s]:off[s + 1]]], 1)
    o, mag, sc = definition([q[off[s]:off[s + 1]] for s in range(S)])
    # keys rounded to bf16, weights and values to fp16, the result to bf16 (see expanded_reference)
    tol = 2.0 ** -8 * o.abs() + (2 * 2.0 ** -11 + 2 * (2.0 ** -8 + 192 * 2.0 ** -24) * sc[..., None] + 2.0 ** -18) * mag \
        + 2.0 ** -25 * (1 + 150 * 8)
    check(out, o, tol, "prompts")

    # decode: the queries' latents and the outputs are rounded to bf16 by the projections outside
    slots1 = torch.zeros(S, dtype=torch.int64, device="cuda")
    lat1 = torch.zeros(S, R, dtype=torch.bfloat16, device="cuda")
    rope1 = torch.zeros(S, ROPE, dtype=torch.bfloat16, device="cuda")
    qa = torch.zeros(S, H, R + ROPE, dtype=torch.bfloat16, device="cuda")
    oa = torch.zeros(S, H, R, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(pkv.latent_workspace_size(pkv.OP_LATENT_ABSORBED, S, S, H, R, ROPE), dtype=torch.uint8,
                     device="cuda")
    ones = dev([1] * S)

    def step():
        pkv.step_metadata(tables, lens, qsl, slots1, taken, lens, ones, free, taken, NB, bs)
        pkv.latent_cache_write(cache, lat1, rope1, slots1)
        pkv.latent_attention_absorbed(oa, qa, cache, tables, lens, SCALE, query_start_loc=qsl, workspace=ws)

    saved = [x.clone() for x in (tables, lens, taken, cache)]
    cap = CapturedStep(step, warmup=1)
    torch.cuda.synchronize()
    for x, y in zip((tables, lens, taken, cache), saved):  # the warm-up advanced the state: put it back
        x.copy_(y)
    for i in range(steps):
        q1 = rnd(S, H, 128 + ROPE)
        lat1.copy_(rnd(S, R))
        rope1.copy_(rnd(S, ROPE))
        q_lat = torch.einsum("thd,hdr->thr", q1[..., :128].double(), w_k.double())
        qa.copy_(torch.cat([q_lat.bfloat16(), q1[..., 128:]], -1))
        torch.cuda.synchronize()
        cap.replay()
        cap.synchronize()
        for s in range(S):
            history[s] = torch.cat([history[s], torch.cat([lat1[s], rope1[s]])[None]])
        # the absorbed attention itself, tight, then the definition through it
        outs, tols = [], []
        for s in range(S):
            rows = history[s]
            o1, m1, c1 = attend(qa[s:s + 1], rows, rows[:, :R], 1, SCALE, True)
            outs.append(o1)
            tols.append(2.0 ** -8 * o1.abs() + (2.0 ** -8 + 2 * (R + ROPE) * 2.0 ** -24 * c1[..., None] + 2.0 ** -18) * m1)
        check(oa, torch.cat(outs), torch.cat(tols), f"step {i}")
        o, mag, sc = definition([q1[s:s + 1] for s in range(S)])
        got = torch.einsum("thr,hdr->thd", oa.double(), w_v.double())
        rms = float((got - o).square().mean().sqrt() / o.square().mean().sqrt())
        # query latents, weights and output latents each rounded once to bf16: 2^-8 / sqrt(3) each in
        # the mean square, the first through scores of size about 1
        assert rms <= 2 * 2.0 ** -8, f"step {i}: {rms}"
    assert pkv.get_device_error() == 0
    assert lens.tolist() == [p + steps for p in prompt]


def test_the_complaint_names_the_tensor_and_what_is_wrong():
    b = Batch([40, 9], [2, 1], 8, 256, 256 + ROPE)
    out = torch.zeros(3, 8, 256, dtype=torch.bfloat16, device="cuda")
    for at, value, said in ((0, out.view(24, 256), "out must have 3 dims"), (1, b.q[:, ::2], "q must be contiguous"),
                            (2, b.cache.float(), "latent_cache must be torch.bfloat16"),
                            (3, b.tables.view(-1), "block_tables must have 2 dims"),
                            (3, b.tables.cpu(), "block_tables must be a CUDA tensor"),
                            (4, b.context_lens[:1], "shape mismatch")):
        args = [out, b.q, b.cache, b.tables, b.context_lens]
        args[at] = value
        with pytest.raises(ValueError, match=said):
            pkv.latent_attention_absorbed(*args, SCALE, query_start_loc=b.qsl)
    assert pkv.get_device_error() == 0 and not out.any()
