"""Calls on a side stream that take a fresh workspace while the current stream still works on a
buffer of that size which the program has given back."""
import pytest
import torch

import pagedattention_paged_kv_gb300 as pkv
from latent_helpers import ROPE, SCALE, Batch

pytestmark = pytest.mark.gpu


def busy(nbytes):
    """The current stream fills a buffer of nbytes for a while; the buffer is given back at once."""
    x = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    for _ in range(300):
        x.fill_(0xFF)


def check_side_stream(call, out, nbytes):
    call(out, None)
    torch.cuda.synchronize()
    want = out.clone()
    side = torch.cuda.Stream()
    for _ in range(5):
        out.zero_()
        torch.cuda.synchronize()
        busy(nbytes)
        call(out, side)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert pkv.get_device_error() == 0


def test_absorbed():
    b = Batch([900, 77, 2000], [1, 1, 1], 32, 512, 512 + ROPE, seed=1)
    out = torch.zeros(3, 32, 512, dtype=torch.bfloat16, device="cuda")
    check_side_stream(lambda o, s: pkv.latent_attention_absorbed(o, b.q, b.cache, b.tables, b.context_lens, SCALE,
                                                                 stream=s),
                      out, pkv.latent_workspace_size(pkv.OP_LATENT_ABSORBED, 3, 3, 32, 512, ROPE))


def test_expanded():
    b = Batch([700, 300], [300, 300], 16, 512, 128 + ROPE, seed=2)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    w = [(torch.randn(16, 128, 512, device="cuda", generator=g) * 512 ** -0.5).bfloat16() for _ in range(2)]
    out = torch.zeros(600, 16, 128, dtype=torch.bfloat16, device="cuda")
    check_side_stream(lambda o, s: pkv.latent_attention_expanded(o, b.q, b.qsl, b.cache, b.tables, b.context_lens, *w,
                                                                 SCALE, 1000, stream=s),
                      out, pkv.latent_workspace_size(pkv.OP_LATENT_EXPANDED, 2, 600, 16, 512, ROPE, total_context=1000))


def test_paged_decode():
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    S, blocks = 4, 60
    kc, vc = (torch.randn(S * blocks, 16, 2, 128, device="cuda", generator=g).bfloat16() for _ in range(2))
    q = torch.randn(S, 16, 128, device="cuda", generator=g).bfloat16()
    tables = torch.randperm(S * blocks, device="cuda", generator=g).int().view(S, blocks)
    lens = torch.tensor([900, 77, 960, 1], dtype=torch.int32, device="cuda")
    out = torch.zeros_like(q)
    check_side_stream(lambda o, s: pkv.paged_attention_decode(o, q, kc, vc, tables, lens, 0.09, stream=s), out,
                      pkv.workspace_size(pkv.OP_DECODE, S, S, 16, 2, 128))
