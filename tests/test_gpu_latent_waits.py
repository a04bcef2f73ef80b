"""Latent-attention launches whose waits run out although every copy was asked for: work so short
that the loads of a CTA never wait for a free place, with a limit of 1 ns.  The launch must return
with no flag but the timeout's (and that of values made from rows that never came), and a launch
right behind it must be right: no copy of the first lands in the shared memory of the second."""
import pytest
import torch

import pagedattention_paged_kv_gb300 as pkv
from latent_helpers import ROPE, SCALE, Batch, absorbed_reference, check, expanded_reference

pytestmark = pytest.mark.gpu


def run_out_then_healthy(short, healthy, ref):
    allowed = pkv.DEVERR_TIMEOUT | pkv.DEVERR_VALUE
    assert pkv.get_device_error() == 0
    for _ in range(10):
        try:
            pkv.set_wait_limit_ns(1)
            short()
        finally:
            pkv.set_wait_limit_ns(0)
        out = healthy()  # queued directly behind
        assert pkv.get_device_error() & ~allowed == 0
        check(out, *ref)
    healthy()
    assert pkv.get_device_error() == 0


@pytest.mark.parametrize("ctx,heads,latent", [([64, 1, 30], 16, 256), ([64], 64, 512), ([128] * 40, 64, 512)])
def test_absorbed_shares_of_one_or_two_tiles(ctx, heads, latent):
    b = Batch(ctx, [1] * len(ctx), heads, latent, latent + ROPE, seed=1, fill=0.0)
    outs = [torch.zeros(len(ctx), heads, latent, dtype=torch.bfloat16, device="cuda") for _ in range(2)]

    def go(out):
        pkv.latent_attention_absorbed(out, b.q, b.cache, b.tables, b.context_lens, SCALE)
        return out

    run_out_then_healthy(lambda: go(outs[0]), lambda: go(outs[1]), absorbed_reference(b))


@pytest.mark.parametrize("ctx,ql,heads,latent", [([128, 7], [128, 7], 2, 256), ([128], [1], 1, 512),
                                                 ([256] * 4, [256] * 4, 16, 512)])
def test_expanded_shares_of_one_or_two_chunks(ctx, ql, heads, latent):
    b = Batch(ctx, ql, heads, latent, 128 + ROPE, seed=2, fill=0.0)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    w = [(torch.randn(heads, 128, latent, device="cuda", generator=g) * latent ** -0.5).bfloat16() for _ in range(2)]
    outs = [torch.zeros(sum(ql), heads, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]

    def go(out):
        pkv.latent_attention_expanded(out, b.q, b.qsl, b.cache, b.tables, b.context_lens, *w, SCALE, sum(ctx))
        return out

    run_out_then_healthy(lambda: go(outs[0]), lambda: go(outs[1]), expanded_reference(b, *w))


def test_the_limit_does_not_count_the_expansion():
    """A limit of 200 us: the longest wait inside either kernel takes microseconds, the expansion of
    65,536 tokens for 64 heads (1.1 TFLOP of products, 2.1 GB written) far longer than the limit."""
    ctx, heads = 65536, 64
    b = Batch([ctx], [16], heads, 512, 128 + ROPE, seed=4, fill=0.0, block_size=64)
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    w = [(torch.randn(heads, 128, 512, device="cuda", generator=g) * 512 ** -0.5).bfloat16() for _ in range(2)]
    n = pkv.latent_workspace_size(pkv.OP_LATENT_EXPANDED, 1, 16, heads, 512, ROPE, total_context=ctx)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")

    def go():
        out = torch.full((16, heads, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
        pkv.latent_attention_expanded(out, b.q, b.qsl, b.cache, b.tables, b.context_lens, *w, SCALE, ctx, workspace=ws)
        return out

    want = go()
    assert pkv.get_device_error() == 0
    try:
        pkv.set_wait_limit_ns(200_000)
        for _ in range(5):
            got = go()
            assert pkv.get_device_error() == 0
            assert torch.equal(got, want)
    finally:
        pkv.set_wait_limit_ns(0)
