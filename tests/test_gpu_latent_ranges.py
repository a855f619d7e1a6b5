"""Attention over the latent pool where its references, sums and scales are
hardest: maxima that move late, values of far powers of two, long pipelines."""
import pytest
import torch

from tests.latent_reference import assert_within, latent_decode
from tests.test_gpu_latent import _decode, _pool, _prefill, _prompt

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("heads", [5, 64])
def test_decode_maximum_in_the_last_tile(dtype, heads):
    """Contexts whose last tokens score far above all before them, most of
    them a single tile: the reference moves in the tile that ends the segment.
    Right, and the same bits every time."""
    g = torch.Generator().manual_seed(heads)
    context = [2 + i % 63 for i in range(250)] + [66 + 37 * (i % 9) for i in range(30)]
    lat, block = 256, 16
    cache, tables = _pool(context, block, lat, dtype, g)
    query = torch.randn(len(context), heads, lat + 64, generator=g).to(dtype)
    query[..., -1] = 8.0
    for s, n in enumerate(context):          # scores 1.6 to 16 above (2.3 to 23 powers of two)
        t = torch.arange(max(0, n - 1 - s % 3), n)
        cache[tables[s][t // block].long(), t % block, -1] = (4.0 + 36.0 * ((s % 7) / 6))
    ctx = torch.tensor(context, dtype=torch.int32)
    ref, bound = latent_decode(query, cache, tables, ctx, 0.05)
    first = _decode(query, cache, tables, ctx, 0.05)
    assert_within(first.cpu(), ref, bound, "decode")
    for _ in range(20):
        assert torch.equal(_decode(query, cache, tables, ctx, 0.05), first)


def test_prefill_ranked_blocks_are_those_of_each_sequence_alone():
    """Blocks taken by size over all sequences (more of them than fit at once)
    give the bits that each sequence gives by itself, every time."""
    new, old = [300, 7, 129, 1, 260, 40], [0, 400, 130, 77, 0, 255]
    x = _prompt(40, 256, 16, new, old, torch.bfloat16, 41)
    query, cache, w, tables, starts, ctx = x
    first = _prefill(*x, 192 ** -0.5)
    for s, n in enumerate(new):
        a = int(starts[s])
        alone = _prefill(query[a:a + n], cache, w, tables[s:s + 1].contiguous(),
                         torch.tensor([0, n], dtype=torch.int32), ctx[s:s + 1], 192 ** -0.5)
        assert torch.equal(alone, first[a:a + n]), s
    for _ in range(20):
        assert torch.equal(_prefill(*x, 192 ** -0.5), first)
