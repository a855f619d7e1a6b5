"""64-bit definitions of the rotating appends and of attention over the latent
pool, with error bounds, for the tests (torch float64 on the CPU).

Bounds.  u = finfo(type).eps / 2 is the largest relative rounding to a 16-bit
type; fp32 sums of n products are off by at most n * 2^-23 of the sum of the
products' magnitudes (2^-24 a rounding, twice that where a tensor core
truncates).
"""
from __future__ import annotations

import math

import torch

F64 = torch.float64


def half_step(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def tiny_step(dtype) -> float:
    """Half the spacing of the type's subnormals: the least absolute rounding."""
    info = torch.finfo(dtype)
    return info.tiny * info.eps / 2


def angle_table(positions: int, rot: int) -> torch.Tensor:
    half = rot // 2
    rate = 10000.0 ** (-torch.arange(half, dtype=F64) / max(half, 1))
    at = torch.arange(positions, dtype=F64)[:, None] * rate
    return torch.cat([at.cos(), at.sin()], 1).float()


def normed(x, weight, eps):
    x = x.to(F64)
    if weight is None:
        return x
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * weight.to(F64)


def rotated(x, cos_sin, positions, interleaved):
    """(rotated x, bound of its fp32 error before the last rounding) for x
    [T][H][D] in float64.  A pair's results are off by less than 2^-20 of the
    pair's magnitudes: at most 12 roundings in the sum of squares (halved by
    the square root), 2 units in rsqrtf, 2 products, 3 operations of the
    rotation, each 2^-24 and together under 16 * 2^-24."""
    rot = cos_sin.shape[1]
    half = rot // 2
    angle = cos_sin.to(F64)[positions.clamp(0, cos_sin.shape[0] - 1)][:, None, :]
    c, s = angle[..., :half], angle[..., half:]
    out, mag = x.clone(), x.abs()
    lo = slice(0, rot, 2) if interleaved else slice(0, half)
    hi = slice(1, rot, 2) if interleaved else slice(half, rot)
    a, b = x[..., lo], x[..., hi]
    out[..., lo], out[..., hi] = a * c - b * s, b * c + a * s
    mag[..., lo] = mag[..., hi] = a.abs() + b.abs()
    return out, mag * 2.0 ** -20


def assert_rounded(got, ref, slack, dtype, what):
    """got is ref (off by at most `slack`) rounded once to dtype."""
    got, u = got.to(F64), half_step(dtype)
    bound = slack + u * (ref.abs() + slack) + tiny_step(dtype)
    bad = ~((got - ref).abs() <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} elements off; worst " \
        f"{float(((got - ref).abs() - bound)[bad].max()):.3g} over the bound"


def context_rows(cache, table, ctx):
    """(rows [ctx][W] float64, which of them lie in the pool)."""
    num_blocks, block, width = cache.shape
    t = torch.arange(ctx)
    page = table[t // block].long()
    ok = (page >= 0) & (page < num_blocks)
    rows = torch.zeros(ctx, width, dtype=F64)
    rows[ok] = cache[page[ok], t[ok] % block].to(F64)
    return rows, ok


def attend(q, keys, values, seen, scale, dtype, key_slack=None, value_slack=0.0, scaled=False):
    """(out, bound) of softmax(scale q keys^T) values for q [n][D], keys
    [t][D], values [t][E], seen [n][t].  The bound: score errors of at most
    e = scale * (D 2^-23 |q| |k| + |q| key_slack) change a weight by a factor
    within exp(2 e); weights and values rounded to the type, the fp16 weights
    also to multiples of 2^-24 of the largest; sums of t terms.  `scaled`: weights
    and values in fp16 with the values' powers of two, so a weight times its
    values' power (at most twice their largest magnitude) is rounded by 2^-11, or
    by 2^-25 of the largest such product."""
    u = half_step(dtype)
    u_w = 2.0 ** -11 if scaled else u
    score = (q @ keys.T) * scale
    e = (q.abs() @ keys.abs().T) * (q.shape[1] * 2.0 ** -23)
    if key_slack is not None:
        e = e + q.abs() @ key_slack.T
    e = (e * abs(scale) + score.abs() * 2.0 ** -22).masked_fill(~seen, 0).amax(1, keepdim=True)
    score = score.masked_fill(~seen, -math.inf)
    top = score.amax(1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(score - top)
    total = p.sum(1, keepdim=True)
    p = torch.where(total > 0, p / total.clamp(min=1e-300), 0.0)
    out = p @ values
    mass = p @ values.abs()
    t = keys.shape[0]
    rel = u_w + torch.expm1(2 * e) + (t + 8) * 2.0 ** -23
    bound = rel * mass + p @ torch.broadcast_to(torch.as_tensor(value_slack, dtype=F64),
                                                values.shape)
    if scaled:
        bound = bound + t * 2.0 ** -24 * values.abs().amax()
    elif dtype == torch.float16:
        bound = bound + t * 2.0 ** -25 * values.abs().amax(0, keepdim=True)
    return out, bound * (1 + u) + u * out.abs() + tiny_step(dtype)


def assert_within(got, ref, bound, what):
    got = got.to(F64)
    assert torch.isfinite(got).all(), f"{what}: not finite"
    bad = ~((got - ref).abs() <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} elements off; worst " \
        f"{float((got - ref).abs().max()):.3g}, over its bound by " \
        f"{float(((got - ref).abs() - bound).max()):.3g}"


def latent_decode(query, cache, tables, context_lens, scale, max_context=None):
    """(out, bound) [S][H][L] of pa_latent_decode; L is the width less 64."""
    dtype, lat = query.dtype, cache.shape[2] - 64
    shape = (*query.shape[:2], lat)
    out, bound = torch.zeros(shape, dtype=F64), torch.zeros(shape, dtype=F64)
    for s, ctx in enumerate(context_lens.tolist()):
        if ctx <= 0 or (max_context is not None and ctx > max_context) \
                or ctx > tables.shape[1] * cache.shape[1]:
            continue
        rows, ok = context_rows(cache, tables[s], ctx)
        out[s], bound[s] = attend(query[s].to(F64), rows, rows[:, :lat],
                                  ok[None, :].expand(query.shape[1], -1), scale, dtype)
    return out, bound


def latent_prefill(query, cache, w_kv, tables, starts, context_lens, scale):
    """(out, bound) [T][H][128] of pa_latent_prefill."""
    dtype, lat, u = query.dtype, cache.shape[2] - 64, half_step(query.dtype)
    heads = query.shape[1]
    out = torch.zeros(*query.shape[:2], 128, dtype=F64)
    bound = torch.zeros_like(out)
    for s, ctx in enumerate(context_lens.tolist()):
        a, b = int(starts[s]), int(starts[s + 1])
        n = b - a
        if n == 0 or ctx < n:
            continue
        rows, ok = context_rows(cache, tables[s], ctx)
        seen = (torch.arange(ctx)[None, :] <= torch.arange(ctx - n, ctx)[:, None]) & ok
        for h in range(heads):
            w = w_kv[h].to(F64)
            kv = rows[:, :lat] @ w.T
            # the expanded key: a sum of `lat` products rounded to the type; the value:
            # to fp16 below the power of two over its largest of 32 tokens, or all
            sums = (lat * 2.0 ** -23) * (rows[:, :lat].abs() @ w.abs().T)
            slack = u * kv.abs() + sums + tiny_step(dtype)
            slack[:, 128:] = 2.0 ** -11 * kv[:, 128:].abs() + sums[:, 128:] \
                + 2.0 ** -24 * kv[:, 128:].abs().amax()
            key = torch.cat([kv[:, :128], rows[:, lat:]], 1)
            key_slack = torch.cat([slack[:, :128], torch.zeros_like(rows[:, lat:])], 1)
            out[a:b, h], bound[a:b, h] = attend(query[a:b, h].to(F64), key, kv[:, 128:], seen,
                                                scale, dtype, key_slack, slack[:, 128:], True)
    return out, bound
