"""Paged-attention launches whose waits run out although every copy was asked for: batches so small
that no CTA's loads wait for a free stage, with a limit of 1 ns.  The launch must return with no
flag but the timeout's, and a launch right behind it must match the oracle."""
import pytest

from gpu_helpers import bf16_bits_to_f64, bf16_to_np, compare, oracle_step, torch_bf16
from pagedattention_paged_kv_gb300 import workloads as W

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", ["decode", "chunk"])
def test_a_launch_behind_one_that_ran_out_is_right(name):
    import torch
    import pagedattention_paged_kv_gb300 as pkv
    if name == "decode":
        b = W.tiny_decode(seed=81)
    else:
        b = W.make_batch("short_chunk", context_lens=[32, 20, 64], q_lens=[32, 20, 16], num_heads=16, num_kv_heads=4,
                         head_dim=128, seed=82)
    slots = pkv.slot_mapping(b.block_tables, b.new_token_seq, b.new_token_pos, b.block_size)
    kc, vc = torch_bf16(b.k_cache), torch_bf16(b.v_cache)
    pkv.reshape_and_cache(kc, vc, torch_bf16(b.k_new), torch_bf16(b.v_new), torch.from_numpy(slots).cuda())
    q = torch_bf16(b.q)
    bt, cl = torch.from_numpy(b.block_tables).cuda(), torch.from_numpy(b.context_lens).cuda()
    qsl = None if b.query_start_loc is None else torch.from_numpy(b.query_start_loc).cuda()
    outs = [torch.zeros_like(q) for _ in range(2)]

    def go(out):
        if qsl is None:
            pkv.paged_attention_decode(out, q, kc, vc, bt, cl, b.scale)
        else:
            pkv.paged_attention_varlen(out, q, qsl, kc, vc, bt, cl, b.scale, causal=b.causal,
                                       max_q_len=int(b.q_lens.max()))

    assert pkv.get_device_error() == 0
    ref, _, _ = oracle_step(b)
    for _ in range(10):
        try:
            pkv.set_wait_limit_ns(1)
            go(outs[0])
        finally:
            pkv.set_wait_limit_ns(0)
        go(outs[1])  # queued directly behind
        assert pkv.get_device_error() & ~pkv.DEVERR_TIMEOUT == 0
        compare(bf16_bits_to_f64(bf16_to_np(outs[1])), ref)
    go(outs[1])
    assert pkv.get_device_error() == 0
