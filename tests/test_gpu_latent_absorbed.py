"""The absorbed latent attention and the latent cache write on the GPU, against 64-bit
references; the slots outside every context hold NaN."""
import pytest
import torch

import pagedattention_paged_kv_gb300 as pkv
from latent_helpers import ROPE, SCALE, Batch, absorbed_reference, check

pytestmark = pytest.mark.gpu


def run(b, decode, causal=True, scale=SCALE, fill=float("nan"), **kw):
    out = torch.full((b.q.shape[0], b.heads, b.latent), fill, dtype=torch.bfloat16, device="cuda")
    pkv.latent_attention_absorbed(out, b.q, b.cache, b.tables, b.context_lens, scale,
                                  query_start_loc=None if decode else b.qsl, causal=causal, **kw)
    assert pkv.get_device_error() == 0
    return out


@pytest.mark.parametrize("heads,latent,block_size", [
    (16, 256, 16), (64, 512, 16), (1, 512, 8), (5, 256, 64), (40, 512, 32), (128, 512, 16), (72, 256, 16)])
def test_decode(heads, latent, block_size):
    ctx = [1, 2, 7, 8, 9, 63, 64, 65, 127, 128, 129, 200, 1000]
    b = Batch(ctx, [1] * len(ctx), heads, latent, latent + ROPE, block_size, seed=heads)
    check(run(b, True), *absorbed_reference(b))


def test_one_sequence_of_one_token_returns_its_latent():
    b = Batch([1], [1], 64, 512, 512 + ROPE, seed=3)
    out = run(b, True)
    assert torch.equal(out, b.rows[0][:, None, :512].expand(1, 64, 512).cuda())


def test_idle_slots_are_zero_rows():
    ctx = [0, 70, 0, 0, 1, 0]
    b = Batch(ctx, [1] * 6, 16, 512, 512 + ROPE, seed=4)
    out = run(b, True)
    check(out, *absorbed_reference(b))
    assert not out[[0, 2, 3, 5]].any()


def test_only_idle_slots():
    b = Batch([0, 0, 0], [1] * 3, 16, 256, 256 + ROPE, seed=5)
    assert not run(b, True).any()


@pytest.mark.parametrize("ctx,heads,latent", [
    ([20011], 64, 512), ([32768, 300, 5, 9000], 16, 512), ([9999, 10001], 128, 256)])
def test_long_contexts_split_over_the_grid(ctx, heads, latent):
    b = Batch(ctx, [1] * len(ctx), heads, latent, latent + ROPE, seed=6)
    check(run(b, True), *absorbed_reference(b))


def test_many_short_sequences():
    ctx = [(37 * i) % 150 for i in range(900)]  # idle ones among them
    b = Batch(ctx, [1] * len(ctx), 16, 256, 256 + ROPE, seed=7)
    check(run(b, True), *absorbed_reference(b))


@pytest.mark.parametrize("heads,latent,block_size", [(16, 512, 16), (24, 256, 8), (128, 512, 16), (3, 256, 32)])
@pytest.mark.parametrize("causal", [True, False])
def test_ragged_rows(heads, latent, block_size, causal):
    ctx = [5, 64, 65, 300, 17, 640, 1, 130]
    ql = [5, 1, 4, 0, 17, 33, 1, 2]
    b = Batch(ctx, ql, heads, latent, latent + ROPE, block_size, seed=8)
    check(run(b, False, causal), *absorbed_reference(b, causal))


def test_rows_behind_the_last_sequence_are_left_alone():
    b = Batch([40, 9], [3, 2], 16, 512, 512 + ROPE, seed=9, extra_rows=6)
    b.q[5:] = float("nan")
    out = run(b, False, fill=7.0)
    ref, tol = absorbed_reference(b)
    check(out[:5], ref[:5], tol[:5])
    assert (out[5:] == 7.0).all()


def test_growing_scores_rescale_the_running_sum():
    # Later keys score far higher than earlier ones, so the running maximum jumps by more than
    # 2^8 again and again, within a share and across shares.
    b = Batch([2000, 700], [1, 1], 16, 512, 512 + ROPE, seed=10, q_std=0.0)
    b.q[..., 0] = 1.0
    for s in range(2):
        b.rows[s][:, 0] = torch.linspace(0, 3000.0, b.ctx[s]).bfloat16()
        for i in range(b.ctx[s]):
            b.cache[b.tables[s, i // 16], i % 16] = b.rows[s][i].cuda()
    check(run(b, True, scale=1.0), *absorbed_reference(b, scale=1.0))


def test_infinite_slots_past_the_context():
    b = Batch([33, 5], [1, 1], 64, 512, 512 + ROPE, seed=11, fill=float("inf"))
    check(run(b, True), *absorbed_reference(b))


def test_a_bad_sequence_is_flagged_and_zero_and_leaves_the_others():
    b = Batch([100, 50, 64], [2, 3, 4], 16, 512, 512 + ROPE, seed=12)
    ref, tol = absorbed_reference(b)
    b.context_lens[1] = 2  # fewer than its query rows
    out = torch.full((9, 16, 512), 5.0, dtype=torch.bfloat16, device="cuda")
    pkv.latent_attention_absorbed(out, b.q, b.cache, b.tables, b.context_lens, SCALE, query_start_loc=b.qsl)
    assert pkv.get_device_error() == pkv.DEVERR_QUERY_LEN
    keep = [0, 1, 5, 6, 7, 8]
    check(out[keep], ref[keep], tol[keep])
    assert not out[2:5].any()
    b.context_lens[1] = 10 ** 6  # past its block-table row
    pkv.latent_attention_absorbed(out, b.q, b.cache, b.tables, b.context_lens, SCALE, query_start_loc=b.qsl)
    assert pkv.get_device_error() == pkv.DEVERR_CONTEXT_LEN
    check(out[keep], ref[keep], tol[keep])


def test_a_block_id_outside_the_pool_is_flagged():
    b = Batch([100, 50], [1, 1], 16, 512, 512 + ROPE, seed=13)
    ref, tol = absorbed_reference(b)
    b.tables[0, 2] = b.num_blocks
    out = torch.empty(2, 16, 512, dtype=torch.bfloat16, device="cuda")
    pkv.latent_attention_absorbed(out, b.q, b.cache, b.tables, b.context_lens, SCALE)
    assert pkv.get_device_error() == pkv.DEVERR_BLOCK_ID
    check(out[1:], ref[1:], tol[1:])


def test_repeats_are_bit_identical_and_streams_agree():
    b = Batch([700, 3, 1500, 64], [1] * 4, 64, 512, 512 + ROPE, seed=14)
    first = run(b, True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = torch.zeros_like(first)
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        pkv.latent_attention_absorbed(out, b.q, b.cache, b.tables, b.context_lens, SCALE, stream=s)
        s.synchronize()
        assert torch.equal(out, first)


@pytest.mark.parametrize("tokens,latent,rope,block_size", [
    (1, 512, 64, 16), (7, 256, 64, 8), (128, 512, 64, 16), (5000, 512, 64, 64), (33, 8, 8, 16), (100, 40, 24, 32)])
def test_cache_write(tokens, latent, rope, block_size):
    g = torch.Generator(device="cuda")
    g.manual_seed(tokens)
    NB = -(-tokens // block_size) + 5
    cache = torch.randn(NB, block_size, latent + rope, device="cuda", generator=g).bfloat16()
    c, r = (torch.randn(tokens, n, device="cuda", generator=g).bfloat16() for n in (latent, rope))
    slots = torch.randperm(NB * block_size, device="cuda", generator=g)[:tokens]
    slots[::7] = -1
    want = cache.clone().view(-1, latent + rope)
    keep = slots >= 0
    want[slots[keep]] = torch.cat([c, r], 1)[keep]
    pkv.latent_cache_write(cache, c, r, slots)
    assert pkv.get_device_error() == 0
    assert torch.equal(cache.view(-1, latent + rope).view(torch.int16), want.view(torch.int16))


def test_cache_write_skips_and_flags_slots_outside_the_pool():
    cache = torch.zeros(2, 16, 320, dtype=torch.bfloat16, device="cuda")
    c, r = torch.ones(3, 256, dtype=torch.bfloat16, device="cuda"), torch.ones(3, 64, dtype=torch.bfloat16, device="cuda")
    pkv.latent_cache_write(cache, c, r, torch.tensor([32, 5, 1 << 40], device="cuda"))
    assert pkv.get_device_error() == pkv.DEVERR_SLOT
    assert cache[0, 5].float().sum() == 320 and cache.float().sum() == 320


def test_cache_write_of_nothing():
    cache = torch.zeros(2, 16, 320, dtype=torch.bfloat16, device="cuda")
    e = torch.zeros(0, 256, dtype=torch.bfloat16, device="cuda")
    pkv.latent_cache_write(cache, e, e[:, :64].contiguous(), torch.zeros(0, dtype=torch.int64, device="cuda"))
    assert pkv.get_device_error() == 0
