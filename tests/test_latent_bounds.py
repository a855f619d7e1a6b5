"""The tolerances of the prompts' tests catch mistakes: the oracle with a key
left out, on the CPU, has to leave them, and its rounded output has not."""
import pytest
import torch

from tests import latent_reference as ref64
from tests.latent_cases import SCALE, edges, point_queries, row_error, row_tolerance
from tests.test_gpu_latent import _prompt

DTYPES = [torch.float16, torch.bfloat16]


def _without(x, tokens):
    """The oracle's output where these tokens of the one sequence are not seen:
    their blocks made single-token ones outside the pool."""
    query, cache, w, tables, starts, ctx = x
    t = torch.arange(int(ctx[0]))
    rows = cache[tables[0][t // cache.shape[1]].long(), t % cache.shape[1]][:, None]
    table = t.to(torch.int32)[None].clone()
    table[0, list(tokens)] = -1
    return ref64.latent_prefill(query, rows, w, table, starts, ctx, SCALE)[0]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("missing", [[317], [1400], list(range(640, 704))])
def test_a_missing_key_shows_in_the_row_error(dtype, missing):
    x = _prompt(2, 256, 16, [100], [1401], dtype, seed=3)
    want, _ = ref64.latent_prefill(*x, SCALE)
    top = row_tolerance(dtype)
    # (what a row's error counts: the output's own rounding)
    assert float(row_error(want.to(dtype), want).max()) <= top
    # a single key's share of the rms of 1400 random ones is about 1 / 37, times what
    # its row gives it (a factor e either way is common): some of 200 rows tell
    assert float(row_error(_without(x, missing), want).max()) > 4 * top


@pytest.mark.parametrize("dtype", DTYPES)
def test_a_missing_key_at_a_border_leaves_the_bound(dtype):
    new, old = 60, 450
    x = _prompt(2, 256, 16, [new], [old], dtype, seed=4)
    targets = point_queries(x, old)
    want, bound = ref64.latent_prefill(*x, SCALE)
    ref64.assert_within(want.to(dtype), want, bound, "rounded")
    assert len(set(targets.tolist())) > len(edges(old)) // 2
    for t in sorted(set(targets.tolist())):
        at = targets == t
        wrong = _without(x, [t])
        with pytest.raises(AssertionError):
            ref64.assert_within(wrong[at], want[at], bound[at], f"without {t}")
        for row in at.nonzero()[:, 0].tolist():      # every query that looks for it
            assert ((wrong[row] - want[row]).abs() > bound[row]).any()
