"""The expanded latent attention over the range of its values and of its weights: values far from
1, different from token to token, and weights far below a row's largest."""
import math

import pytest
import torch

import pagedattention_paged_kv_gb300 as pkv
from latent_helpers import BF16_HALF, F16_HALF, ROPE, SCALE, Batch, check

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
    2^-6.57 of 2^-25.43; the result is rounded to bf16; a running fp32 sum of 200,000 like terms is
    off by 200,000 x 2^-23 of itself at most (every addition truncated)."""
    out, share = many_small_weights(0.0)
    want = share / (1 + share)
    assert ((out - want).abs() <= (2.0 ** -6.57 + BF16_HALF + 200_000 * 2.0 ** -23) * want).all(), \
        f"{out.min().item()} .. {out.max().item()}, not {want}"


def test_many_small_weights_beside_an_equal_value():
    """Equal values come back.  The sum of weights x values is held in fp32: a product of 2^-25.43 is
    below half a step (2^-24) of the 1 that the first key brought, so in one running sum each may be
    lost whole, whatever order the hardware adds in: 0.44% of the output, to which the weights'
    roundings (200,000 x 2^-32) and the result's (2^-9 below 1) come."""
    out, share = many_small_weights(1.0)
    assert ((out - 1.0).abs() <= share + 200_000 * 2.0 ** -32 + 2.0 ** -9).all(), \
        f"{out.min().item()} .. {out.max().item()}"


def reference(b, w_v, causal):
    """(out, tolerance) with w_k the identity on the first 128 latent columns, so keys are exact.

    Roundings: the result bf16; a value fp16 (2^-11 of itself, 2^-39 of the largest value of its 32
    tokens, 2^-89); a weight fp16, twice where a chunk's second half moves the maximum (2^-11 of
    itself, and 2 x 2^-32 of the largest contribution of the row, where a contribution is weight x
    largest value of the 32 tokens, which a stored value is at most twice of); a score's 192 products
    in fp32; the exponent in fp32, two roundings of a number below 256: 2 x 2^-25 x 256 x ln 2 < 2^-16."""
    R, H = b.latent, b.heads
    out = torch.zeros(b.q.shape[0], H, 128, dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(out)
    for s, (c, n) in enumerate(zip(b.ctx, b.q_lens)):
        rows = b.rows[s].cuda().double()
        k = torch.cat([rows[:, :128], rows[:, R:]], -1)
        v = torch.einsum("cr,hdr->hcd", rows[:, :R], w_v.double())
        top = torch.zeros(H, -(-c // 32) * 32, dtype=torch.float64, device="cuda")
        top[:, :c] = v.abs().amax(-1)
        top = top.view(H, -1, 32).amax(-1, keepdim=True).expand(-1, -1, 32).reshape(H, -1)[:, :c]
        q = b.q[b.offsets[s]:b.offsets[s + 1]].double().transpose(0, 1)
        sc = SCALE * q @ k.t()
        size = SCALE * (q.abs() @ k.abs().t()).amax(-1)
        if causal:
            sc = sc.masked_fill(torch.ones(n, c, dtype=torch.bool, device="cuda").triu(c - n + 1), -math.inf)
        p = torch.softmax(sc, -1)
        o, mag = p @ v, p @ v.abs()
        delta = 192 * 2.0 ** -24 * size[..., None]
        low = 2.0 ** -39 * (p @ top[..., None]) + 2.0 ** -89 + 2.0 ** -30 * c * (p * top[:, None]).amax(-1, keepdim=True)
        t = BF16_HALF * o.abs() + (3 * F16_HALF + 2 * delta + 2.0 ** -16) * mag + low
        out[b.offsets[s]:b.offsets[s + 1]] = o.transpose(0, 1)
        tol[b.offsets[s]:b.offsets[s + 1]] = t.transpose(0, 1)
    return out, tol


def run_scaled(ctx, ql, heads, latent, factor, w_scale=1.0, causal=True, bs=16, seed=0):
    """factor(s, c): what each token's latent vector is multiplied by, powers of two (or 0)."""
    b = Batch(ctx, ql, heads, latent, 128 + ROPE, bs, seed=seed)
    for s, c in enumerate(ctx):
        b.rows[s][:, :latent] *= factor(s, c)[:, None].bfloat16()
        at = torch.arange(c)
        b.cache[b.tables[s].cpu()[at // bs].long().cuda(), (at % bs).cuda()] = b.rows[s].cuda()
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1)
    w_v = (torch.randn(heads, 128, latent, device="cuda", generator=g) * latent ** -0.5).bfloat16() * w_scale
    w_k = torch.zeros_like(w_v)
    w_k[:, range(128), range(128)] = 1.0
    out = torch.full((sum(ql), heads, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    pkv.latent_attention_expanded(out, b.q, b.qsl, b.cache, b.tables, b.context_lens, w_k, w_v, SCALE, sum(ctx),
                                  causal=causal)
    assert pkv.get_device_error() == 0
    ref, tol = reference(b, w_v, causal)
    return out, ref, tol


def ones(s, c):
    return torch.ones(c)


@pytest.mark.parametrize("power", [12, 0, -10, -14, -17, -20, -27, -40, -48, -60])
def test_values_of_one_size(power):
    out, ref, tol = run_scaled([300, 1, 700], [300, 1, 5], 3, 256, ones, w_scale=2.0 ** power, seed=power + 70)
    check(out, ref, tol)


def test_values_of_one_size_in_a_split_context():
    out, ref, tol = run_scaled([9000, 50], [1, 7], 2, 512, ones, w_scale=2.0 ** -24, seed=1)
    check(out, ref, tol)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("run", [1, 7, 32, 96, 128])
def test_values_of_many_sizes(run, causal):
    """Runs of tokens whose latents differ by up to 2^36, small ones before large ones among them:
    the rows of a prompt that see only small ones keep their bits."""
    g = torch.Generator()
    g.manual_seed(run)

    def factor(s, c):
        powers = torch.randint(-36, 1, (-(-c // run),), generator=g).float()
        if s == 0:
            powers = powers.sort().values
        return torch.exp2(powers).repeat_interleave(run)[:c]

    out, ref, tol = run_scaled([600, 300, 129], [600, 40, 129], 4, 256, factor, causal=causal, seed=2)
    for lo, hi in ((0, 600), (600, 640), (640, 769)):
        check(out[lo:hi], ref[lo:hi], tol[lo:hi])


@pytest.mark.parametrize("small", [0, -30])
def test_values_of_zero_beside_others_count_in_the_sum_only(small):
    """Whole chunks and groups of 32 tokens with values of zero, the others about 2^small."""
    def factor(s, c):
        f = torch.full((c,), 2.0 ** small)
        f[: c // 3] = 0.0
        f[c // 2: c // 2 + 40] = 0.0
        return f

    out, ref, tol = run_scaled([900, 5000], [900, 2], 2, 512, factor, seed=3)
    check(out[:900], ref[:900], tol[:900])
    check(out[900:], ref[900:], tol[900:])


def test_large_values_up_to_the_range_of_fp16_are_not_clamped():
    out, ref, tol = run_scaled([200, 64], [200, 64], 2, 256, lambda s, c: torch.full((c,), 2.0 ** 6), w_scale=2.0 ** 7,
                               seed=4)
    assert 20000 < ref.abs().max() < 65504
    check(out, ref, tol)
