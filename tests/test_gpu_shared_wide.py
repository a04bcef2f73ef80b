"""Decode attention over shared prefixes with as many query heads as a call may have."""
import pytest
import torch

import pagedattention_paged_kv_gb300 as pkv
from shared_helpers import FP8_SCALE, Shared, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,fp8", [(64, False), (128, False), (128, True)])
def test_a_million_query_heads(d, fp8):
    """One sequence of 20 tokens, 16 query heads to each of 65,536 KV heads (8 a work item, 8192 items);
    the first, the last and some KV heads between looked at."""
    kv_heads, group, bs, ctx = 1 << 16, 16, 16, 20
    heads = kv_heads * group
    g = torch.Generator(device="cuda").manual_seed(d)
    k, v = (torch.randn(2, bs, kv_heads, d, generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    if fp8:
        k, v = ((x.float() / FP8_SCALE).to(torch.float8_e4m3fn).view(torch.uint8) for x in (k, v))
    q = torch.randn(1, heads, d, generator=g, device="cuda", dtype=torch.bfloat16)
    tables = torch.tensor([[1, 0]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([ctx], dtype=torch.int32, device="cuda")
    start, prefix = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 1], [16]))
    some = torch.tensor([0, 1, 2047, 2048, 32767, 40000, 65534, 65535], device="cuda")
    part = Shared.__new__(Shared)
    part.heads, part.kv_heads, part.d, part.bs, part.fp8 = len(some) * group, len(some), d, bs, fp8
    part.scale, part.ctx, part.tables, part.lens = d ** -0.5, [ctx], tables, lens
    part.k, part.v = k[:, :, some], v[:, :, some]
    rows = (some[:, None] * group + torch.arange(group, device="cuda")).flatten()
    part.q = q[:, rows]
    out = torch.full_like(q, float("nan"))
    pkv.paged_attention_decode_shared(out, q, k, v, tables, lens, start, prefix, part.scale, **part.scales())
    assert pkv.get_device_error() == 0 and out.isfinite().all()
    check(out[:, rows], part.reference())
