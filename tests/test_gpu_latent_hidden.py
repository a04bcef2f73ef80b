"""What the header says of cache rows that are not finite, inside a context, and of block ids outside
the pool: which query rows they reach in either form of the latent attention, and what those are."""
import pytest
import torch

import pagedattention_paged_kv_gb300 as pkv
from latent_helpers import ROPE, SCALE, Batch, absorbed_reference, check, expanded_reference

pytestmark = pytest.mark.gpu

R, HEADS = 256, 2
FORMS = ["absorbed", "expanded"]


def make(form, ctx, ql):
    b = Batch(ctx, ql, HEADS, R, (R if form == "absorbed" else 128) + ROPE, 16, seed=5)
    g = torch.Generator(device="cuda")
    g.manual_seed(6)
    w = [(torch.randn(HEADS, 128, R, device="cuda", generator=g) * R ** -0.5).bfloat16() for _ in range(2)]
    return b, w


def run(form, b, w):
    out = torch.full((b.q.shape[0], HEADS, R if form == "absorbed" else 128), 5.0, dtype=torch.bfloat16, device="cuda")
    if form == "absorbed":
        pkv.latent_attention_absorbed(out, b.q, b.cache, b.tables, b.context_lens, SCALE, query_start_loc=b.qsl)
    else:
        pkv.latent_attention_expanded(out, b.q, b.qsl, b.cache, b.tables, b.context_lens, *w, SCALE, sum(b.ctx))
    return out


def reference(form, b, w):
    return absorbed_reference(b) if form == "absorbed" else expanded_reference(b, *w)


def finite_rows(out):
    return torch.isfinite(out).all(-1).all(-1).cpu()


# the token lies in the 128-token chunk 384 .. 511; the first tile's rows see chunks up to 255
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("token", [384, 400, 511])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_latent_part_that_is_not_finite(form, token, value):
    b, w = make(form, [512, 40], [512, 40])
    ref, tol = reference(form, b, w)
    b.cache[b.tables[0, token // 16], token % 16, 3] = value
    out = run(form, b, w)
    assert pkv.get_device_error() == 0
    rows = finite_rows(out)
    assert not rows[token:512].any()
    check(out[512:], ref[512:], tol[512:])
    if form == "absorbed":
        assert not rows[:512].any()
    else:
        check(out[:256], ref[:256], tol[:256])


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("token", [0, 63, 64, 400, 511])
def test_a_rotary_part_of_nan_reaches_the_rows_that_see_it(form, token):
    b, w = make(form, [512, 40], [512, 40])
    ref, tol = reference(form, b, w)
    b.cache[b.tables[0, token // 16], token % 16, R + 9] = float("nan")
    out = run(form, b, w)
    assert pkv.get_device_error() == 0
    assert not finite_rows(out)[token:512].any()
    keep = [*range(token), *range(512, 552)]
    check(out[keep], ref[keep], tol[keep])


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("bad", [-1, 10 ** 6])
def test_the_tokens_of_a_block_outside_the_pool_count_as_zeros(form, bad):
    b, w = make(form, [300, 50], [40, 50])
    b.tables[0, 2] = bad
    out = run(form, b, w)
    assert pkv.get_device_error() == pkv.DEVERR_BLOCK_ID
    b.rows[0][32:48] = 0
    check(out, *reference(form, b, w))


@pytest.mark.parametrize("form", FORMS)
def test_a_sequence_with_bad_offsets_has_no_rows(form):
    b, w = make(form, [100, 50, 30], [20, 30, 10])
    ref, tol = reference(form, b, w)
    b.qsl[3] = 10 ** 6      # past the rows of q
    out = run(form, b, w)
    assert pkv.get_device_error() == pkv.DEVERR_QUERY_LEN
    check(out[:50], ref[:50], tol[:50])
    assert (out[50:] == 5.0).all()
