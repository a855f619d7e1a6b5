"""Attention over the latent pool where its references, sums and scales are
hardest: maxima that move late, values of far powers of two, long pipelines."""
import pytest
import torch

from tests.latent_cases import SCALE, point_queries, row_error, row_tolerance
from tests.latent_reference import (F64, assert_within, attend, context_rows, latent_decode,
                                    latent_prefill)
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


def test_lengths_written_right_before_the_call():
    """Lengths, starts and queries that the work just before on the stream
    writes: every call follows its own, with nothing waited for between."""
    from paged_kv_cache_415_b200 import binding as B
    a = [t.cuda() for t in _prompt(6, 256, 16, [90, 200, 3], [40, 0, 300], torch.float16, 51)]
    b = [t.cuda() for t in _prompt(6, 256, 16, [150, 1, 142], [0, 330, 20], torch.float16, 52)]
    query, cache, w, tables, starts, ctx = (torch.empty_like(x) for x in a)
    width = max(a[3].shape[1], b[3].shape[1])
    blocks = max(a[1].shape[0], b[1].shape[0])
    cache = torch.zeros(blocks, *a[1].shape[1:], dtype=torch.float16, device="cuda")
    tables = torch.zeros(3, width, dtype=torch.int32, device="cuda")
    absorbed = [torch.randn(3, 6, 320, device="cuda").half() for _ in range(2)]
    n = B.pa_latent_prefill_workspace_size(3, 6, 256, 16, 340)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    n = B.pa_latent_decode_workspace_size(3, 6, 256, 16, 340)
    ws_d = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")

    def take(x, q):
        query.copy_(x[0])
        cache[:x[1].shape[0]].copy_(x[1])
        w.copy_(x[2])
        tables.zero_()
        tables[:, :x[3].shape[1]].copy_(x[3])
        starts.copy_(x[4])
        ctx.copy_(x[5])
        out = torch.empty(293, 6, 128, dtype=torch.float16, device="cuda")
        B.pa_latent_prefill(out, query, cache, w, tables, starts, ctx, 200, 340, 0.07, ws)
        dec = torch.empty(3, 6, 256, dtype=torch.float16, device="cuda")
        B.pa_latent_decode(dec, q, cache, tables, ctx, 340, 0.05, workspace=ws_d)
        return out, dec

    want = []
    for x, q in zip((a, b), absorbed):
        got = take(x, q)
        torch.cuda.synchronize()
        ref, bound = latent_prefill(*(t.cpu() for t in x), 0.07)
        assert_within(got[0].cpu(), ref, bound, "prefill")
        want.append(got)
    got = [take(x, q) for _ in range(30) for x, q in zip((a, b), absorbed)]
    for i, pair in enumerate(got):
        assert all(torch.equal(g, r) for g, r in zip(pair, want[i % 2])), i


def _far_powers(powers, dtype, seed, new=70, old=90):
    """A prompt whose tokens' latent vectors are scaled by 2^powers[g], g the
    token's group of 32 (None: zeros); keys take the rotated part alone."""
    x = _prompt(2, 256, 16, [new], [old], dtype, seed)
    query, cache, w, tables, starts, ctx = x
    w[:, :128] = 0
    t = torch.arange(new + old)
    power = torch.tensor([-1000.0 if p is None else p for p in powers])[t // 32]
    rows = cache[tables[0][t // 16].long(), t % 16]
    rows[:, :256] = (rows[:, :256].to(F64) * torch.exp2(power.to(F64))[:, None]).to(dtype)
    cache[tables[0][t // 16].long(), t % 16] = rows
    return x


@pytest.mark.parametrize("powers", [
    (None, 70, None, None, 70), (70, None, None, 70, None), (None, None, None, None, 115),
    (110, None, None, None, None), (-55, 10, 70, None, 40), (70, 40, 10, -20, -55),
    (None, -50, None, 0, 90),
])
def test_prefill_values_of_far_powers(powers):
    """Groups of 32 tokens whose values lie up to 2^170 apart, zeros among
    them: every token counts in the sum of the weights."""
    x = _far_powers(powers, torch.bfloat16, 61)
    out = _prefill(*x, 0.05)
    ref, bound = latent_prefill(*x, 0.05)
    assert_within(out.cpu(), ref, bound, f"powers {powers}")


@pytest.mark.parametrize("lean", [-1, 1])
def test_prefill_far_powers_against_the_scores(lean):
    """Values of 2^60 whose tokens score 100 powers of two lower or higher
    than those of ordinary values."""
    x = _far_powers((0, 60, 0, 60, 0), torch.bfloat16, 62)
    query, cache, w, tables, starts, ctx = x
    query[..., -1] = 8.0
    t = torch.arange(160)
    lift = torch.where((t // 32) % 2 == 1, lean * 100 * 0.6931 / (0.05 * 8.0), 0.0)
    cache[tables[0][t // 16].long(), t % 16, -1] = lift.bfloat16()
    out = _prefill(*x, 0.05)
    ref, bound = latent_prefill(*x, 0.05)
    assert_within(out.cpu(), ref, bound, f"lean {lean}")


def _leader(ctx, gap, lat, dtype, seed):
    """A context whose first token outweighs each other one by about 2^gap and
    has the value 0, so that the output is made of the faint ones alone.
    Scores come from one element of the rotated part: 8 r scale, exact but for
    the scale's rounding.  Returns (cache, tables, rows, p [ctx], total)."""
    g = torch.Generator().manual_seed(seed)
    cache, tables = _pool([ctx], 16, lat, dtype, g)
    t = torch.arange(ctx)
    rows = (torch.randn(ctx, lat + 64, generator=g) * 0.25).abs().to(dtype)
    rows[:, lat:] = 0
    rows[:, -1] = (torch.rand(ctx, generator=g) - 0.5).to(dtype)
    rows[0] = 0
    rows[0, -1] = gap
    cache[tables[0][t // 16].long(), t % 16] = rows
    p = torch.exp2(rows[:, -1].to(F64) - gap)
    return cache, tables, rows.to(F64), p, p.sum()


_EIGHTH = 0.6931471805599453 / 8                     # 8 r scale = r ln 2
# What is left to err: the scale in fp32 and the references (at most 64 * 2^-23
# together in the exponent), 2^-22 of an exponential, fp32 sums of t terms.
_SLACK = 64 * 2.0 ** -23 + 2.0 ** -22


@pytest.mark.parametrize("gap", [10, 20, 24])
@pytest.mark.parametrize("ctx", [1000, 32768])
def test_decode_faint_weights(ctx, gap):
    """fp16 weights: 2^7 of room above the reference is used, so a weight is
    off by 2^-11 of itself or by 2^-32 of the leader's."""
    lat = 256
    cache, tables, rows, p, total = _leader(ctx, gap, lat, torch.float16, gap)
    query = torch.zeros(1, 3, lat + 64, dtype=torch.float16)
    query[..., -1] = 8
    out = _decode(query, cache, tables, torch.tensor([ctx], dtype=torch.int32), _EIGHTH)
    values = rows[:, :lat]
    ref = (p @ values) / total
    off = torch.clamp(p * 2.0 ** -11, min=2.0 ** -32)
    bound = (off @ values) / total + (_SLACK + (ctx + 8) * 2.0 ** -23) * ref
    bound = bound + 2.0 ** -11 * (ref + bound) + 2.0 ** -25
    assert_within(out.cpu()[0], ref.expand(3, -1), bound.expand(3, -1), f"gap {gap}")


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("gap", [10, 20, 24])
def test_prefill_faint_weights(dtype, gap):
    """The same in the prompt's attention, whose weights are fp16 for both
    types; its values too, off by 2^-11 of themselves (the expansion here
    takes one element of the row: no sum)."""
    ctx, lat, new = 20000, 256, 3
    cache, tables, rows, p, _ = _leader(ctx, gap, lat, dtype, gap)
    u = 2.0 ** -11 if dtype == torch.float16 else 2.0 ** -8
    query = torch.zeros(new, 2, 192, dtype=dtype)
    query[..., -1] = 8
    w = torch.zeros(2, 256, lat, dtype=dtype)
    e = torch.arange(128)
    w[:, 128 + e, e] = 1
    out = _prefill(query, cache, w, tables, torch.tensor([0, new], dtype=torch.int32),
                   torch.tensor([ctx], dtype=torch.int32), _EIGHTH).cpu()
    for i in range(new):
        n = ctx - new + 1 + i
        values = rows[:n, :128]
        ref = (p[:n] @ values) / p[:n].sum()
        # a weight is taken times its 32 tokens' power of two, which is 1 or 2 here
        # (their largest value lies in [0.5, 2)), so may be half as fine as the leader's
        assert all(0.5 <= float(v.amax()) < 2 for v in values.split(32) if len(v) == 32)
        off = torch.clamp(p[:n] * 2.0 ** -11, min=2.0 ** -31)
        bound = (off @ values) / p[:n].sum() \
            + (_SLACK + 2.0 ** -11 + (n + 8) * 2.0 ** -23) * ref
        bound = bound + u * (ref + bound) + 2.0 ** -25
        assert_within(out[i], ref.expand(2, -1), bound.expand(2, -1), f"gap {gap}")


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("finite", [1, 30, 200])
def test_decode_minus_infinity_behind_bad_blocks(dtype, finite):
    """A tile of bad blocks, then a tile whose scores are all minus infinity:
    neither weighs anything, what follows is as it is alone."""
    ctx, lat = 128 + finite, 256
    g = torch.Generator().manual_seed(finite)
    cache, tables = _pool([ctx], 16, lat, dtype, g)
    query = torch.randn(1, 16, lat + 64, generator=g).to(dtype)
    query[..., lat] = query[..., lat].abs() + 0.5
    t = torch.arange(64, 128)
    cache[tables[0][t // 16].long(), t % 16, lat] = 0
    rows, _ = context_rows(cache, tables[0], ctx)
    seen = (torch.arange(ctx) >= 128).expand(16, ctx)
    ref, bound = attend(query[0].to(F64), rows, rows[:, :lat], seen, 0.05, dtype)
    cache[tables[0][t // 16].long(), t % 16, lat] = -float("inf")
    tables[0, :4] = -1
    out = _decode(query, cache, tables, torch.tensor([ctx], dtype=torch.int32), 0.05)
    assert_within(out.cpu()[0], ref, bound, "decode")


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("heads,lat,block,new,old", [
    (3, 256, 16, [256, 130], [1150, 1999]),          # 9 to 17 tiles of keys, query tiles of unequal steps
    (2, 512, 32, [300], [1000]),
    (2, 512, 64, [8, 40], [4100, 2500]),             # few new tokens behind long prefixes
    (1, 256, 8, [1500], [300]),                      # several pairs of query tiles
])
def test_prefill_long_pipeline(dtype, heads, lat, block, new, old):
    """Row by row as close to 64 bits as the roundings allow: one key of
    thousands left out or taken twice would show."""
    x = _prompt(heads, lat, block, new, old, dtype, seed=sum(old))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = _prefill(*x, SCALE, status=status).cpu()
    ref, bound = latent_prefill(*x, SCALE)
    assert_within(out, ref, bound, "prefill")
    assert float(row_error(out, ref).max()) <= row_tolerance(dtype)
    assert int(status) == 0


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("lat,block,new,old", [(256, 16, 256, 1150), (512, 32, 200, 2200)])
def test_prefill_every_key_at_a_border(dtype, lat, block, new, old):
    """Queries that give nearly all their weight to a token next to a border
    of half a tile, each such token in turn."""
    x = _prompt(2, lat, block, [new], [old], dtype, seed=new)
    point_queries(x, old)
    out = _prefill(*x, SCALE).cpu()
    ref, bound = latent_prefill(*x, SCALE)
    assert_within(out, ref, bound, "prefill")


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("heads,lat", [(128, 512), (128, 256), (65, 256)])
def test_prefill_many_heads(dtype, heads, lat):
    x = _prompt(heads, lat, 16, [5, 131], [0, 150], dtype, seed=heads + lat)
    out = _prefill(*x, SCALE).cpu()
    ref, bound = latent_prefill(*x, SCALE)
    assert_within(out, ref, bound, "prefill")


@pytest.mark.parametrize("scale", [0.0, -0.06, 2.0])
def test_prefill_scales(scale):
    """Equal scores, a negative scale, scores in the hundreds."""
    x = _prompt(2, 256, 16, [200, 3], [150, 140], torch.float16, 81)
    out = _prefill(*x, scale).cpu()
    ref, bound = latent_prefill(*x, scale)
    assert_within(out, ref, bound, f"scale {scale}")


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_query_that_is_not_finite_keeps_to_itself(dtype, value):
    """Other heads and other queries keep every bit."""
    g = torch.Generator().manual_seed(91)
    cache, tables = _pool([200, 70], 16, 256, dtype, g)
    query = torch.randn(2, 20, 320, generator=g).to(dtype)
    ctx = torch.tensor([200, 70], dtype=torch.int32)
    want = _decode(query, cache, tables, ctx, 0.05)
    query[0, 3] = value
    got = _decode(query, cache, tables, ctx, 0.05)
    assert torch.isnan(got[0, 3]).all()
    got[0, 3] = want[0, 3]
    assert torch.equal(got, want)
    x = _prompt(3, 256, 16, [150, 20], [90, 0], dtype, 92)
    want = _prefill(*x, 0.07)
    x[0][40, 1] = value
    got = _prefill(*x, 0.07)
    assert torch.isnan(got[40, 1]).all()
    got[40, 1] = want[40, 1]
    assert torch.equal(got, want)


def test_prompts_and_steps_on_two_streams():
    """Prefill and decode calls side by side, each with its own workspace: the
    bits of one after the other."""
    from paged_kv_cache_415_b200 import binding as B
    x = [t.cuda() for t in _prompt(16, 512, 16, [300, 70], [100, 900], torch.bfloat16, 95)]
    query, cache, w, tables, starts, ctx = x
    top = int(ctx.max())
    absorbed = torch.randn(2, 16, 576, device="cuda").bfloat16()
    outs = [torch.empty(370, 16, 128, dtype=torch.bfloat16, device="cuda"),
            torch.empty(2, 16, 512, dtype=torch.bfloat16, device="cuda")]
    sizes = (B.pa_latent_prefill_workspace_size(2, 16, 512, 16, top),
             B.pa_latent_decode_workspace_size(2, 16, 512, 16, top))
    spaces = [torch.empty(max(n, 16), dtype=torch.uint8, device="cuda") for n in sizes]

    def prefill(stream=None):
        B.pa_latent_prefill(outs[0], query, cache, w, tables, starts, ctx, 300, top, 0.07, spaces[0],
                            stream=stream)

    def decode(stream=None):
        B.pa_latent_decode(outs[1], absorbed, cache, tables, ctx, top, 0.05, workspace=spaces[1],
                           stream=stream)

    prefill()
    decode()
    torch.cuda.synchronize()
    want = [o.clone() for o in outs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for turn in range(10):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for _ in range(5):
            prefill(streams[turn % 2])
            for _ in range(4):
                decode(streams[1 - turn % 2])
        torch.cuda.synchronize()
        assert all(torch.equal(o, r) for o, r in zip(outs, want)), turn
