"""The expanded latent attention over the range of its values and of its weights: values far from
1, different from token to token, and weights far below a row's largest."""
import pytest
import torch

import pagedattention_paged_kv_gb300 as pkv
from latent_helpers import ROPE

pytestmark = pytest.mark.gpu


def test_many_small_weights_keep_their_sum():
    """Equal values come back whatever the weights: 200,000 keys of weight 2^-25.4 beside one of 1
    hold 0.44% of the sum.  Each weight may be off by 2^-32 of the largest (half of fp16's smallest
    step, weights held 2^7 times larger): 4.7e-5 in all, under the 2^-9 at which 1 would round to
    another bf16 number.  160 heads, so that most contexts are not split."""
    n, R, bs, H = 200_001, 256, 64, 160
    blocks = -(-n // bs)
    cache = torch.zeros(blocks, bs, R + ROPE, dtype=torch.bfloat16, device="cuda")
    cache[..., 0] = 1.0
    cache[..., R] = -17.625            # e^-17.625 = 2^-25.43
    cache[0, 0, R] = 0.0
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
    assert (out == 1.0).all(), f"{out.float().min().item()} .. {out.float().max().item()}"
