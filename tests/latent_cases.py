"""Prompts whose errors tell more than a worst-case bound does, and how far
off they may be: shared by the tests on the CPU (where mistakes are planted in
the oracle) and on the GPU."""
from __future__ import annotations

import torch

from tests.latent_reference import F64

SCALE = 192 ** -0.5


def row_error(got, ref):
    """[T][H]: root mean square error of each output row, of the row's."""
    err = (got.to(F64) - ref).pow(2).mean(-1).sqrt()
    return err / ref.pow(2).mean(-1).sqrt()


def row_tolerance(dtype) -> float:
    """For rows over hundreds of tokens of random queries, keys and values.  A
    rounding to a type whose half step is u has an rms of 0.42 u (uniform in
    [-u, u] of the binade's lower end, mantissas uniform over the binade's
    logarithm).  The output's own: 0.42 u.  The key's 128 rounded elements move a
    score by SCALE sqrt(128) 0.42 u = 0.82 * 0.42 u, each key's for itself, which
    is what they move the output by.  Weights and values in fp16: 0.42 * 2^-11
    each.  Together 0.0021 in bf16, 0.00038 in fp16; a single row (128 elements,
    its query's length, how few keys lead it) is within 2.5 of that."""
    u = torch.finfo(dtype).eps / 2
    parts = [u, 0.82 * u, 2.0 ** -11, 2.0 ** -11]
    return 2.5 * 0.42 * sum(p * p for p in parts) ** 0.5


def edges(tokens):
    """The tokens next to the borders of 64 keys, up to `tokens`."""
    at = {t for b in range(0, tokens + 64, 64) for t in (b - 1, b, b + 1)}
    return sorted(t for t in at | {tokens - 1} if 0 <= t < tokens)


def point_queries(x, old):
    """Makes every query of the one-sequence prompt x look for one token next to
    a border of 64 keys, each of them in turn: its weight is all but 1."""
    query, cache, w, tables, starts, ctx = x
    n, block = query.shape[0], cache.shape[1]
    targets = []
    for i in range(n):
        e = edges(old + i + 1)
        targets.append(e[(7 * i) % len(e)])
    t = torch.tensor(targets)
    part = cache[tables[0][t // block].long(), t % block, -64:].float()
    query[..., 128:] = (8 * part)[:, None].to(query.dtype)
    return t
