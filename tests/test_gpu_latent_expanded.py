"""The expanded latent attention on the GPU, against 64-bit references; the slots outside every
context hold NaN.  The two forms of latent attention against each other."""
import pytest
import torch

import pagedattention_paged_kv_gb300 as pkv
from latent_helpers import ROPE, SCALE, Batch, check, expanded_reference

pytestmark = pytest.mark.gpu


def weights(heads, latent, seed=1):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return [(torch.randn(heads, 128, latent, device="cuda", generator=g) * latent ** -0.5).bfloat16() for _ in range(2)]


def make(ctx, ql, heads, latent, bs=16, seed=0, **kw):
    return Batch(ctx, ql, heads, latent, 128 + ROPE, bs, seed=seed, **kw), *weights(heads, latent, seed + 1)


def run(b, w_k, w_v, causal=True, fill=float("nan"), total=None, scale=SCALE, **kw):
    out = torch.full((b.q.shape[0], b.heads, 128), fill, dtype=torch.bfloat16, device="cuda")
    total = sum(c for c, n in zip(b.ctx, b.q_lens) if n) if total is None else total
    pkv.latent_attention_expanded(out, b.q, b.qsl, b.cache, b.tables, b.context_lens, w_k, w_v, scale, total,
                                  causal=causal, **kw)
    return out


@pytest.mark.parametrize("heads,latent,bs", [(16, 256, 16), (1, 512, 8), (3, 512, 64), (20, 256, 32)])
@pytest.mark.parametrize("causal", [True, False])
def test_ragged_prompts(heads, latent, bs, causal):
    ctx = [1, 2, 127, 128, 129, 300, 255, 256, 257, 500, 40, 9]
    ql = [1, 2, 127, 128, 129, 300, 1, 256, 257, 130, 0, 3]
    b, w_k, w_v = make(ctx, ql, heads, latent, bs, seed=heads)
    out = run(b, w_k, w_v, causal)
    assert pkv.get_device_error() == 0
    check(out, *expanded_reference(b, w_k, w_v, causal))


@pytest.mark.parametrize("ctx,ql,heads,latent", [
    ([4096 + 512], [512], 16, 512),       # a chunk behind a prefix
    ([3001], [3001], 4, 512),             # a whole prompt
    ([9000, 50], [1, 7], 8, 256),         # few queries, split along the keys
    ([700] * 9, [300] * 9, 64, 512)])
def test_chunks(ctx, ql, heads, latent):
    b, w_k, w_v = make(ctx, ql, heads, latent, seed=2)
    out = run(b, w_k, w_v)
    assert pkv.get_device_error() == 0
    check(out, *expanded_reference(b, w_k, w_v))


def test_more_sequences_than_threads():
    ctx = [(13 * i) % 90 + 1 for i in range(500)]
    ql = [min(c, i % 4) for i, c in enumerate(ctx)]
    b, w_k, w_v = make(ctx, ql, 2, 256, seed=3)
    out = run(b, w_k, w_v)
    assert pkv.get_device_error() == 0
    check(out, *expanded_reference(b, w_k, w_v))


def test_rows_behind_the_last_sequence_are_left_alone():
    b, w_k, w_v = make([40, 9], [30, 2], 4, 256, seed=4, extra_rows=5)
    b.q[32:] = float("nan")
    out = run(b, w_k, w_v, fill=7.0)
    assert pkv.get_device_error() == 0
    ref, tol = expanded_reference(b, w_k, w_v)
    check(out[:32], ref[:32], tol[:32])
    assert (out[32:] == 7.0).all()


def test_infinite_slots_past_the_context():
    b, w_k, w_v = make([33, 130], [33, 5], 4, 512, seed=5, fill=float("inf"))
    out = run(b, w_k, w_v)
    assert pkv.get_device_error() == 0
    check(out, *expanded_reference(b, w_k, w_v))


def test_growing_scores_rescale_the_running_sum():
    # w_k picks one latent column, so the keys are exact in bf16 and scores carry no rounding of
    # theirs: the tolerance keeps its other terms, each relative to the weighted |values| (which
    # reach hundreds here, so no absolute figure would do).
    b, w_k, w_v = make([1500], [400], 2, 256, seed=6, q_std=0.0)
    b.q[..., 0] = 1.0
    w_k.zero_()
    w_k[:, 0, 0] = 1.0
    b.rows[0][:, 0] = torch.linspace(0, 3000.0, 1500).bfloat16()
    for i in range(1500):
        b.cache[b.tables[0, i // 16], i % 16] = b.rows[0][i].cuda()
    out = run(b, w_k, w_v, scale=1.0)
    ref, tol = expanded_reference(b, w_k, w_v, scale=1.0, exact_keys=True)
    check(out, ref, tol)


def test_bad_sequences_are_flagged_and_zero_and_leave_the_others():
    b, w_k, w_v = make([100, 50, 64], [20, 30, 40], 4, 256, seed=7)
    ref, tol = expanded_reference(b, w_k, w_v)
    b.context_lens[1] = 29
    out = run(b, w_k, w_v, fill=5.0)
    assert pkv.get_device_error() == pkv.DEVERR_QUERY_LEN
    keep = list(range(20)) + list(range(50, 90))
    check(out[keep], ref[keep], tol[keep])
    assert not out[20:50].any()


def test_values_past_fp16_are_clamped_and_flagged():
    b, w_k, w_v = make([40], [40], 2, 256, seed=12)
    w_v.zero_()
    w_v[:, 3, 7] = 1.0
    b.cache[b.tables[0, 1], 2, 7] = 1e5   # token 18, alone past the range
    b.rows[0][18, 7] = 65504.0
    out = run(b, w_k, w_v)
    assert pkv.get_device_error() == pkv.DEVERR_VALUE
    w_k2 = w_k.clone()
    w_k2[..., 7] = 0                      # its key would move with the clamp too
    w_k[..., 7] = 0
    out = run(b, w_k, w_v)
    assert pkv.get_device_error() == pkv.DEVERR_VALUE
    check(out, *expanded_reference(b, w_k2, w_v))


def test_a_batch_past_its_total_context_is_refused():
    b, w_k, w_v = make([300, 500], [20, 30], 4, 256, seed=8)
    out = run(b, w_k, w_v, fill=5.0, total=300)
    assert pkv.get_device_error() == pkv.DEVERR_CONTEXT_LEN
    assert not out.any()


def test_a_block_id_outside_the_pool_is_flagged():
    b, w_k, w_v = make([100, 50], [10, 10], 4, 256, seed=9)
    ref, tol = expanded_reference(b, w_k, w_v)
    b.tables[0, 2] = -7
    out = run(b, w_k, w_v)
    assert pkv.get_device_error() == pkv.DEVERR_BLOCK_ID
    check(out[10:], ref[10:], tol[10:])


def test_absorbed_form_gives_the_same_attention():
    """The run as a serving step uses the two forms: the prompt chunk expanded, and the same rows
    absorbed with the projections applied outside."""
    heads, latent = 16, 512
    b, w_k, w_v = make([200, 77], [60, 5], heads, latent, seed=10)
    ref, tol = expanded_reference(b, w_k, w_v)
    check(run(b, w_k, w_v), ref, tol)
    q_lat = torch.einsum("thd,hdr->thr", b.q[..., :128].float(), w_k.float()).bfloat16()
    qa = torch.cat([q_lat, b.q[..., 128:]], -1).contiguous()
    o = torch.empty(65, heads, latent, dtype=torch.bfloat16, device="cuda")
    pkv.latent_attention_absorbed(o, qa, b.cache, b.tables, b.context_lens, SCALE, query_start_loc=b.qsl)
    assert pkv.get_device_error() == 0
    got = torch.einsum("thr,hdr->thd", o.double(), w_v.double())
    # the query latents and the output latents are rounded to bf16 on this side: the same kinds of
    # rounding as the keys' and values' on the other
    rms = float((got - ref).square().mean().sqrt() / ref.square().mean().sqrt())
    assert rms <= 2 * 2.0 ** -8


def test_captured_and_replayed():
    from pagedattention_paged_kv_gb300.graph import CapturedStep
    b, w_k, w_v = make([600, 130], [512, 1], 8, 512, seed=11)
    n = pkv.latent_workspace_size(pkv.OP_LATENT_EXPANDED, 2, 513, 8, 512, ROPE, total_context=730)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    eager = run(b, w_k, w_v, workspace=ws)
    out = torch.zeros_like(eager)
    cap = CapturedStep(lambda: pkv.latent_attention_expanded(out, b.q, b.qsl, b.cache, b.tables, b.context_lens, w_k,
                                                             w_v, SCALE, 730, workspace=ws))
    for _ in range(3):
        out.zero_()
        torch.cuda.synchronize()
        cap.replay()
        cap.synchronize()
        assert torch.equal(out, eager)
    assert pkv.get_device_error() == 0
