"""The expanded latent attention over the range of its values and of its weights: values far from
1, different from token to token, and weights far below a row's largest."""
import math

import pytest
import torch

import pagedattention_paged_kv_gb300 as pkv
from latent_helpers import BF16_HALF, ROPE

pytestmark = pytest.mark.gpu


def many_small_weights(first_value):
    """200,000 keys of weight 2^-25.43 and value 1 behind one of weight 1 and first_value; 160 heads, so
    that most contexts are not split.  Returns (out, the small keys' share of the sum before it is
    normalised)."""
    n, R, bs, H = 200_001, 256, 64, 160
    blocks = -(-n // bs)
    cache = torch.zeros(blocks, bs, R + ROPE, dtype=torch.bfloat16, device="cuda")
    cache[..., 0] = 1.0
    cache[..., R] = -17.625            # e^-17.625 = 2^-25.43
    cache[0, 0, R] = 0.0
    cache[0, 0, 0] = first_value
    q = torch.zeros(1, H, 128 + ROPE, dtype=torch.bfloat16, device="cuda")
    q[..., 128] = 1.0
    w_k = torch.zeros(H, 128, R, dtype=torch.bfloat16, device="cuda")
    w_v = torch.zeros(H, 128, R, dtype=torch.bfloat16, device="cuda")
    w_v[..., 0] = 1.0
    tables = torch.arange(blocks, dtype=torch.int32, device="cuda")[None]
    out = torch.zeros(1, H, 128, dtype=torch.bfloat16, device="cuda")
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    pkv.latent_attention_expanded(out, q, dev([0, 1]), cache, tables, dev([n]), w_k, w_v, 1.0, n)
    assert pkv.get_device_error() == 0
    return out.double(), (n - 1) * math.exp(-17.625)


def test_many_small_weights_beside_a_value_of_zero():
    """What the small weights add up to is all there is of the output, 0.44%.  A weight may be off by
    2^-32 of the largest (half of fp16's smallest step, weights held 2^7 times larger), which is
    2^-6.57 of 2^-25.43; the result is rounded to bf16; 2^-16 for fp32."""
    out, share = many_small_weights(0.0)
    want = share / (1 + share)
    assert ((out - want).abs() <= (2.0 ** -6.57 + BF16_HALF + 2.0 ** -16) * want).all(), \
        f"{out.min().item()} .. {out.max().item()}, not {want}"


def test_many_small_weights_beside_an_equal_value():
    """Equal values come back.  The sum of weights x values is held in fp32: a product of 2^-25.43 is
    below half a step (2^-24) of the 1 that the first key brought, so in one running sum each may be
    lost whole, whatever order the hardware adds in: 0.44% of the output, to which the weights'
    roundings (200,000 x 2^-32) and the result's (2^-9 below 1) come."""
    out, share = many_small_weights(1.0)
    assert ((out - 1.0).abs() <= share + 200_000 * 2.0 ** -32 + 2.0 ** -9).all(), \
        f"{out.min().item()} .. {out.max().item()}"
