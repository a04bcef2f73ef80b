"""Scores that are not numbers or infinite, in the latent attention: what softmax makes of them by its
definition, whether a context is split over the grid or not."""
import pytest
import torch

import pagedattention_paged_kv_gb300 as pkv
from latent_helpers import ROPE, SCALE, Batch, absorbed_reference, check, expanded_reference

pytestmark = pytest.mark.gpu

R = 256
# contexts of one chunk, and of one chunk a CTA of a 152-SM grid or more
CTX = [100, 152 * 128, 40000]


def run(form, b, w):
    if form == "absorbed":
        out = torch.full((b.q.shape[0], b.heads, R), 5.0, dtype=torch.bfloat16, device="cuda")
        pkv.latent_attention_absorbed(out, b.q, b.cache, b.tables, b.context_lens, SCALE, query_start_loc=b.qsl)
    else:
        out = torch.full((b.q.shape[0], b.heads, 128), 5.0, dtype=torch.bfloat16, device="cuda")
        pkv.latent_attention_expanded(out, b.q, b.qsl, b.cache, b.tables, b.context_lens, *w, SCALE, sum(b.ctx))
    assert pkv.get_device_error() == 0
    return out


def make(form, ctx, ql, heads=1):
    b = Batch(ctx, ql, heads, R, (R if form == "absorbed" else 128) + ROPE, 64, seed=3)
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    w = [(torch.randn(heads, 128, R, device="cuda", generator=g) * R ** -0.5).bfloat16() for _ in range(2)]
    return b, w


def reference(form, b, w):
    return absorbed_reference(b) if form == "absorbed" else expanded_reference(b, *w)


@pytest.mark.parametrize("form", ["absorbed", "expanded"])
@pytest.mark.parametrize("ctx", CTX)
def test_a_query_row_of_nan_gives_nan_there_and_nowhere_else(form, ctx):
    b, w = make(form, [ctx, 30], [3, 1])
    ref, tol = reference(form, b, w)
    b.q[1] = float("nan")
    out = run(form, b, w)
    assert torch.isnan(out[1]).all()
    keep = [0, 2, 3]
    check(out[keep], ref[keep], tol[keep])


@pytest.mark.parametrize("form", ["absorbed", "expanded"])
@pytest.mark.parametrize("ctx", CTX[1:])
def test_a_chunk_of_nan_keys_gives_nan(form, ctx):
    b, w = make(form, [ctx, 30], [1, 1])
    ref, tol = reference(form, b, w)
    for blk in range(100, 102):      # tokens 6400 .. 6527, one 128-token chunk
        b.cache[b.tables[0, blk]] = float("nan")
    out = run(form, b, w)
    assert torch.isnan(out[0]).all()
    check(out[1:], ref[1:], tol[1:])


@pytest.mark.parametrize("form", ["absorbed", "expanded"])
@pytest.mark.parametrize("ctx", CTX)
def test_scores_of_minus_infinity_alone_give_nan(form, ctx):
    b, w = make(form, [ctx, 30], [1, 1])
    ref, tol = reference(form, b, w)
    b.q[0] = 0
    b.q[0, :, -1] = 1.0
    b.cache[b.tables[0, :-(-ctx // 64)].long(), :, :-1] = 0
    b.cache[b.tables[0, :-(-ctx // 64)].long(), :, -1] = float("-inf")
    out = run(form, b, w)
    # (0 x -inf = NaN in the columns that are zero in both does not arise: the others are finite)
    assert torch.isnan(out[0]).all()
    check(out[1:], ref[1:], tol[1:])


@pytest.mark.parametrize("form", ["absorbed", "expanded"])
def test_a_score_of_minus_infinity_among_others_has_no_weight(form):
    b, w = make(form, [300], [1])
    b.q[0, :, -1] = 1.0
    keep = torch.tensor([j for j in range(300) if j != 77])
    full = b.rows[0]
    b.cache[b.tables[0, 1], 77 - 64, -1] = float("-inf")
    out = run(form, b, w)
    b.rows[0], b.ctx[0] = full[keep], 299
    check(out, *reference(form, b, w))
