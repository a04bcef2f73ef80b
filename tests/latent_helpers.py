"""Inputs and 64-bit references of the latent-attention tests (plain torch, no code of the
package)."""
from __future__ import annotations

import math

import torch

ROPE = 64
BF16_HALF = 2.0 ** -8      # half a bf16 step, relative
F16_HALF = 2.0 ** -11      # half an fp16 step, relative
SCALE = 1.0 / math.sqrt(128 + ROPE)


class Batch:
    """A paged latent cache whose slots outside every context hold `fill` (NaN by default), and
    the queries over it."""

    def __init__(self, ctx, q_lens, heads, latent, q_cols, block_size=16, seed=0, fill=float("nan"),
                 q_std=1.0, extra_rows=0, table_room=0):
        dev = "cuda"
        g = torch.Generator(device="cpu")
        g.manual_seed(seed)
        S = len(ctx)
        self.ctx, self.q_lens, self.heads, self.latent, self.bs = list(ctx), list(q_lens), heads, latent, block_size
        blocks = [-(-c // block_size) for c in ctx]
        self.num_blocks = max(1, sum(blocks) + 3)
        perm = torch.randperm(self.num_blocks, generator=g)
        self.tables = torch.full((S, max([1] + blocks) + table_room), -1, dtype=torch.int32)
        cache = torch.full((self.num_blocks, block_size, latent + ROPE), fill)
        self.rows = []
        at = 0
        for s in range(S):
            ids = perm[at:at + blocks[s]]
            at += blocks[s]
            self.tables[s, :blocks[s]] = ids.int()
            r = torch.randn(ctx[s], latent + ROPE, generator=g).bfloat16()
            self.rows.append(r)
            for b in range(blocks[s]):
                part = r[b * block_size:(b + 1) * block_size]
                cache[ids[b], :part.shape[0]] = part.float()
        T = sum(q_lens) + extra_rows
        self.q = (torch.randn(T, heads, q_cols, generator=g) * q_std).bfloat16().to(dev)
        self.cache = cache.bfloat16().to(dev)
        self.tables = self.tables.to(dev)
        self.context_lens = torch.tensor(self.ctx, dtype=torch.int32, device=dev)
        off = [0]
        for n in q_lens:
            off.append(off[-1] + n)
        self.offsets = off
        self.qsl = torch.tensor(off, dtype=torch.int32, device=dev)


def attend(q, keys, vals, n, scale, causal):
    """One sequence in 64 bits: q [n, H, d], keys [c, d] or [H, c, d], vals likewise; its last n
    positions.  Returns out [n, H, dv], the same sums with |values|, and the largest
    scale * sum |q||k| of a query row."""
    q, keys, vals = q.double(), keys.double(), vals.double()
    if keys.dim() == 2:
        keys, vals = keys.expand(q.shape[1], *keys.shape), vals.expand(q.shape[1], *vals.shape)
    c = keys.shape[1]
    qh = q.transpose(0, 1)
    s = scale * qh @ keys.transpose(1, 2)
    mag = scale * (qh.abs() @ keys.abs().transpose(1, 2)).amax(-1)
    if causal:
        hidden = torch.ones(n, c, dtype=torch.bool, device=q.device).triu(c - n + 1)
        s = s.masked_fill(hidden, -math.inf)
    p = torch.softmax(s, -1)
    return ((p @ vals).transpose(0, 1), (p @ vals.abs()).transpose(0, 1), mag.transpose(0, 1))


def absorbed_reference(b: Batch, causal=True, scale=SCALE):
    """(out, tolerance) of the absorbed form, zeros where a sequence has no context.

    The tolerance counts the kernel's roundings: each softmax weight to bf16 (half a step of it,
    so 2^-8 of the sum of weight x |value|), the result to bf16 (2^-8 of it), and the fp32 sums
    of a score's latent + 64 products, at most their count x 2^-24 of the sum of |q||k|, which
    moves a weight and the normalising sum by that much each; 2^-18 covers exp2 and the fp32
    sums of the weights and of the output."""
    T = b.q.shape[0]
    out = torch.zeros(T, b.heads, b.latent, dtype=torch.float64, device=b.q.device)
    tol = torch.zeros_like(out)
    for s, (c, n) in enumerate(zip(b.ctx, b.q_lens)):
        if n == 0 or c == 0:
            continue
        lo = b.offsets[s]
        rows = b.rows[s].to(b.q.device)
        o, mag, sc = attend(b.q[lo:lo + n], rows, rows[:, :b.latent], n, scale, causal)
        delta = (b.latent + ROPE) * 2.0 ** -24 * sc
        out[lo:lo + n] = o
        tol[lo:lo + n] = BF16_HALF * o.abs() + (BF16_HALF + 2 * delta[..., None] + 2.0 ** -18) * mag
    return out, tol


def expanded_reference(b: Batch, w_k, w_v, causal=True, scale=SCALE, exact_keys=False):
    """(out, tolerance) of the expanded form.  The kernel rounds keys to bf16: half a step moves a
    score by at most 2^-8 of the sum of |q||k|, hence a weight and the normalising sum by that
    much each.  Weights and values are fp16, half a step 2^-11 of each, and 2^-25 for values
    under fp16's normal range (weights there are below 2^-14 of the row's largest: 2^-25 of it
    for each key).  The rest as in the absorbed form.
    exact_keys: the keys are bf16 numbers, their rounding does nothing."""
    T, H, R = b.q.shape[0], b.heads, b.latent
    out = torch.zeros(T, H, w_v.shape[1], dtype=torch.float64, device=b.q.device)
    tol = torch.zeros_like(out)
    for s, (c, n) in enumerate(zip(b.ctx, b.q_lens)):
        if n == 0 or c == 0:
            continue
        lo = b.offsets[s]
        rows = b.rows[s].to(b.q.device).double()
        k = torch.einsum("cr,hdr->hcd", rows[:, :R], w_k.double())
        v = torch.einsum("cr,hdr->hcd", rows[:, :R], w_v.double())
        k = torch.cat([k, rows[None, :, R:].expand(H, c, ROPE)], -1)
        o, mag, sc = attend(b.q[lo:lo + n], k, v, n, scale, causal)
        delta = ((0.0 if exact_keys else BF16_HALF) + 192 * 2.0 ** -24) * sc
        out[lo:lo + n] = o
        tol[lo:lo + n] = BF16_HALF * o.abs() + (2 * F16_HALF + 2 * delta[..., None] + 2.0 ** -18) * mag \
            + 2.0 ** -25 * (1 + v.abs().sum(1))
    return out, tol


def check(got, ref, tol, what=""):
    got = got.double()
    assert torch.isfinite(got).all(), f"{what}: {int((~torch.isfinite(got)).sum())} values not finite"
    over = (got - ref).abs() - tol
    worst = int(over.argmax())
    assert (over <= 0).all(), (f"{what}: {int((over > 0).sum())} of {over.numel()} out of tolerance, worst at "
                               f"{worst}: got {got.flatten()[worst]:.6g} want {ref.flatten()[worst]:.6g} "
                               f"tol {tol.flatten()[worst]:.3g}")
    # Independent roundings: each of the result, the weights and (expanded) the values and keys is
    # off by 2^-8 / sqrt(3) of itself at most in the mean square, together under 2 x that.
    rms = float((got - ref).square().mean().sqrt() / ref.square().mean().sqrt().clamp(min=1e-300)) if ref.any() else 0.0
    assert rms <= 2 * BF16_HALF, f"{what}: rms error {rms:.3g} of the result"
