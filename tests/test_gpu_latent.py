"""pa_latent_decode and pa_latent_prefill against their 64-bit definitions,
and a prompt followed by decode steps as a model runs them."""
import pytest
import torch

from tests.latent_reference import (F64, angle_table, assert_within, attend, context_rows,
                                    half_step, latent_decode, latent_prefill, normed, rotated)

pytestmark = pytest.mark.gpu
BAD_BLOCK, BAD_CONTEXT = 1, 4


def _pool(context, block, lat, dtype, g, spare=3, fill=float("nan")):
    """A pool whose unused rows hold `fill`, and the tables of `context`."""
    need = [-(-max(c, 0) // block) for c in context]
    blocks = sum(need) + spare
    order = torch.randperm(blocks, generator=g).to(torch.int32)
    tables = torch.full((len(context), max(need + [1])), 2 ** 31 - 1, dtype=torch.int32)
    cache = torch.full((blocks, block, lat + 64), fill, dtype=dtype)
    at = 0
    for s, n in enumerate(need):
        tables[s, :n] = order[at:at + n]
        at += n
        t = torch.arange(max(context[s], 0))
        cache[tables[s][t // block].long(), t % block] = \
            torch.randn(len(t), lat + 64, generator=g).to(dtype)
    return cache, tables


def _decode(query, cache, tables, context, scale, max_context=None, status=None, stream=None,
            out=None, workspace=None):
    from paged_kv_cache_415_b200 import binding as B
    s, h, w = query.shape
    lat = w - 64
    top = max_context if max_context is not None else max(max(context.tolist()), 0)
    if workspace is None:
        n = B.pa_latent_decode_workspace_size(s, h, lat, cache.shape[1], top)
        # junk: the contents on entry must not matter
        workspace = torch.full((max(n, 16),), 0xff, dtype=torch.uint8, device="cuda")
    if out is None:
        out = torch.full((s, h, lat), 9.0, dtype=query.dtype, device="cuda")
    B.pa_latent_decode(out, query.cuda(), cache.cuda(), tables.cuda(), context.cuda(), top, scale,
                       workspace=workspace, d_status=status, stream=stream)
    return out


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("heads,lat,block,context", [
    (1, 512, 16, [1]),
    (16, 512, 16, [0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 300]),
    (16, 256, 8, [200, 0, 7, 8, 9, 1000]),
    (5, 512, 64, [64, 1, 63, 65, 640]),
    (40, 256, 32, [33, 31, 700, 1]),
    (64, 512, 32, [255, 257, 3]),
    (65, 512, 16, [100, 20]),
    (96, 256, 16, [77, 400]),
    (128, 512, 64, [1, 500, 129]),
    (128, 512, 8, [61, 62]),
    (8, 512, 16, [9000]),                           # one context over many CTAs
    (33, 256, 32, [4000, 5, 4001]),
])
def test_decode(dtype, heads, lat, block, context):
    g = torch.Generator().manual_seed(heads * 1000 + len(context))
    cache, tables = _pool(context, block, lat, dtype, g)
    query = torch.randn(len(context), heads, lat + 64, generator=g).to(dtype)
    ctx = torch.tensor(context, dtype=torch.int32)
    scale = (lat + 64) ** -0.5
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = _decode(query, cache, tables, ctx, scale, status=status)
    ref, bound = latent_decode(query, cache, tables, ctx, scale)
    assert_within(out.cpu(), ref, bound, "decode")
    assert int(status) == 0


def test_decode_many_short_sequences():
    """More sequences than CTAs, empty ones between them."""
    g = torch.Generator().manual_seed(1)
    context = [int(x) for x in torch.randint(0, 90, (411,), generator=g)]
    context[:3], context[-2:] = [0, 0, 64], [0, 0]
    cache, tables = _pool(context, 16, 256, torch.bfloat16, g)
    query = torch.randn(len(context), 12, 320, generator=g).to(torch.bfloat16)
    ctx = torch.tensor(context, dtype=torch.int32)
    out = _decode(query, cache, tables, ctx, 0.05)
    ref, bound = latent_decode(query, cache, tables, ctx, 0.05)
    assert_within(out.cpu(), ref, bound, "decode")
    assert (out[ctx == 0] == 0).all()


@pytest.mark.parametrize("scale", [0.0, -0.05, 3.0])
def test_decode_scores(scale):
    """Equal scores, a negative scale, scores in the hundreds whose maximum
    moves along the context (the running maximum is passed many times)."""
    g = torch.Generator().manual_seed(6)
    lat, heads = 512, 20
    context = [700, 64, 1, 321]
    cache, tables = _pool(context, 16, lat, torch.bfloat16, g)
    query = torch.randn(len(context), heads, lat + 64, generator=g).to(torch.bfloat16)
    for s, n in enumerate(context):                    # later tokens nearer to the first head's query
        t = torch.arange(n)
        rows = cache[tables[s][t // 16].long(), t % 16].float()
        rows += (t / n)[:, None] * query[s, 0].float()
        cache[tables[s][t // 16].long(), t % 16] = rows.to(torch.bfloat16)
    ctx = torch.tensor(context, dtype=torch.int32)
    out = _decode(query, cache, tables, ctx, scale)
    ref, bound = latent_decode(query, cache, tables, ctx, scale)
    assert_within(out.cpu(), ref, bound, f"scale {scale}")


@pytest.mark.parametrize("fill", [float("inf"), -float("inf"), float("nan")])
def test_decode_bad_blocks_and_contexts(fill):
    """Blocks outside the pool are left out, wherever they lie; a sequence of
    bad blocks alone and one of a bad length give zeros; what lies behind the
    contexts does not count, whatever it is."""
    g = torch.Generator().manual_seed(8)
    context = [130, 200, 48, 100, 80, 90]
    cache, tables = _pool(context, 16, 512, torch.float16, g, fill=fill)
    tables[0, 3], tables[1, 0], tables[1, 12] = -1, cache.shape[0], 2 ** 31 - 1
    tables[2, :3] = -5
    query = torch.randn(6, 16, 576, generator=g).to(torch.float16)
    given = torch.tensor([130, 200, 48, -3, 1 << 20, 90], dtype=torch.int32)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = _decode(query, cache, tables, given, 0.04, max_context=200, status=status)
    ref, bound = latent_decode(query, cache, tables, given, 0.04, max_context=200)
    assert_within(out.cpu(), ref, bound, "decode")
    assert (out[2:5] == 0).all()
    assert int(status) == (BAD_BLOCK | BAD_CONTEXT)


def test_decode_repeats_and_ignores_the_placement():
    """Bit for bit: again, with other physical blocks, on another stream with
    a workspace of its own while the first runs, and replayed from a graph."""
    from paged_kv_cache_415_b200 import binding as B
    g = torch.Generator().manual_seed(4)
    context = [2000, 3, 517]
    cache, tables = _pool(context, 32, 512, torch.bfloat16, g)
    query = torch.randn(3, 24, 576, generator=g).to(torch.bfloat16).cuda()
    ctx = torch.tensor(context, dtype=torch.int32)
    first = _decode(query, cache, tables, ctx, 0.05)
    order = torch.randperm(cache.shape[0], generator=g)
    moved = torch.empty_like(cache)
    moved[order] = cache
    new_tables = torch.where(tables < cache.shape[0],
                             order[tables.clamp(max=cache.shape[0] - 1).long()].int(), tables)
    n = B.pa_latent_decode_workspace_size(3, 24, 512, 32, 2000)
    spaces = [torch.empty(max(n, 16), dtype=torch.uint8, device="cuda") for _ in range(2)]
    outs = [torch.empty_like(first) for _ in range(2)]
    dev = [(t.cuda(), c.cuda()) for c, t in ((cache, tables), (moved, new_tables))]
    ctx_d = ctx.cuda()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        for (t, c), st, o, w in zip(dev, streams, outs, spaces):
            B.pa_latent_decode(o, query, c, t, ctx_d, 2000, 0.05, workspace=w, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], first) and torch.equal(outs[1], first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.pa_latent_decode(outs[0], query, dev[0][1], dev[0][0], ctx_d, 2000, 0.05,
                           workspace=spaces[0])
    for lens in ([2000, 3, 517], [1, 1999, 64]):
        ctx_d.copy_(torch.tensor(lens, dtype=torch.int32))
        if lens[1] > 3:
            dev[0][0][1] = dev[0][0][0]
        outs[0].fill_(3)
        graph.replay()
        now = torch.tensor(lens, dtype=torch.int32)
        ref, bound = latent_decode(query.cpu(), cache, dev[0][0].cpu(), now, 0.05)
        assert_within(outs[0].cpu(), ref, bound, f"replayed {lens}")


@pytest.mark.slow
def test_past_32_bit_offsets():
    """Blocks whose element offsets pass 2^31, in decode and in prefill."""
    from paged_kv_cache_415_b200 import binding as B
    g = torch.Generator().manual_seed(2)
    dtype, block = torch.bfloat16, 16
    blocks = (1 << 31) // (block * 576) + 40
    cache = torch.empty(blocks, block, 576, dtype=dtype, device="cuda")
    small, tables = _pool([300], block, 512, dtype, g, spare=0)
    far = blocks - 1 - torch.arange(small.shape[0])
    cache[far.cuda()] = small.cuda()
    far_tables = far[tables.long()].int()
    query = torch.randn(1, 16, 576, generator=g).to(dtype)
    ctx = torch.tensor([300], dtype=torch.int32)
    out = _decode(query, cache, far_tables, ctx, 0.04)
    assert torch.equal(out, _decode(query, small, tables, ctx, 0.04))
    q = torch.randn(9, 4, 192, generator=g).to(dtype).cuda()
    w = (torch.randn(4, 256, 512, generator=g) / 22).to(dtype).cuda()
    starts = torch.tensor([0, 9], dtype=torch.int32, device="cuda")
    ws = torch.empty(B.pa_latent_prefill_workspace_size(1, 4, 512, block, 300), dtype=torch.uint8,
                     device="cuda")
    outs = [torch.empty(9, 4, 128, dtype=dtype, device="cuda") for _ in range(2)]
    for o, c, t in zip(outs, (cache, small.cuda()), (far_tables, tables)):
        B.pa_latent_prefill(o, q, c, w, t.cuda(), starts, ctx.cuda(), 9, 300, 0.07, ws)
    assert torch.equal(*outs)


# ---------------------------------------------------------------------------
# Prompts
# ---------------------------------------------------------------------------

def _prefill(query, cache, w_kv, tables, starts, context, scale, max_new=None, max_context=None,
             status=None, out=None):
    from paged_kv_cache_415_b200 import binding as B
    t, h, _ = query.shape
    lens = [b - a for a, b in zip(starts.tolist(), starts.tolist()[1:])]
    max_new = max(lens) if max_new is None else max_new
    top = max(context.tolist()) if max_context is None else max_context
    ws = torch.full((B.pa_latent_prefill_workspace_size(len(context), h, cache.shape[2] - 64,
                                                        cache.shape[1], top),), 0xff,
                    dtype=torch.uint8, device="cuda")
    if out is None:
        out = torch.full((t, h, 128), 9.0, dtype=query.dtype, device="cuda")
    B.pa_latent_prefill(out, query.cuda(), cache.cuda(), w_kv.cuda(), tables.cuda(), starts.cuda(),
                        context.cuda(), max_new, top, scale, ws, d_status=status)
    return out


def _prompt(heads, lat, block, new, old, dtype, seed, extra=0, fill=float("nan")):
    g = torch.Generator().manual_seed(seed)
    context = [a + b for a, b in zip(new, old)]
    cache, tables = _pool(context, block, lat, dtype, g, fill=fill)
    starts = torch.tensor([0] + torch.tensor(new).cumsum(0).tolist(), dtype=torch.int32)
    query = torch.randn(sum(new) + extra, heads, 192, generator=g).to(dtype)
    w = (torch.randn(heads, 256, lat, generator=g) * lat ** -0.5).to(dtype)
    return query, cache, w, tables, starts, torch.tensor(context, dtype=torch.int32)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("heads,lat,block,new,old", [
    (1, 512, 16, [1], [0]),
    (3, 256, 8, [5, 0, 130], [0, 9, 1]),
    (2, 512, 16, [127, 128, 129, 1], [0, 0, 0, 255]),
    (8, 512, 32, [17, 300], [300, 0]),
    (5, 256, 64, [64, 65, 63], [64, 63, 1]),
    (20, 512, 64, [2, 31], [500, 97]),
    (1, 512, 16, [513], [0]),
])
def test_prefill(dtype, heads, lat, block, new, old):
    x = _prompt(heads, lat, block, new, old, dtype, seed=sum(new) + heads, extra=3)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = _prefill(*x, 192 ** -0.5, status=status)
    ref, bound = latent_prefill(*x, 192 ** -0.5)
    n = sum(new)
    assert_within(out.cpu()[:n], ref[:n], bound[:n], "prefill")
    assert (out[n:] == 9).all()                        # rows behind the last sequence
    assert int(status) == 0


def test_prefill_moving_maximum():
    """Scores in the hundreds that rise along the context."""
    query, cache, w, tables, starts, ctx = _prompt(2, 256, 16, [300], [100], torch.bfloat16, 3)
    t = torch.arange(400)
    cache[tables[0][t // 16].long(), t % 16, 256:] += ((t / 40)[:, None]
                                                       * query[0, 0, 128:].float()).bfloat16()
    out = _prefill(query, cache, w, tables, starts, ctx, 0.3)
    ref, bound = latent_prefill(query, cache, w, tables, starts, ctx, 0.3)
    assert_within(out.cpu(), ref, bound, "prefill")


@pytest.mark.parametrize("fill", [float("inf"), float("nan")])
def test_prefill_bad_blocks_and_lengths(fill):
    new, old = [40, 30, 20, 10, 25], [100, 0, 10, 0, 3]
    query, cache, w, tables, starts, ctx = _prompt(3, 512, 16, new, old, torch.float16, 5,
                                                   fill=fill)
    tables[0, 2], tables[1, 0] = -1, cache.shape[0]
    ctx = ctx.clone()
    ctx[2], ctx[3] = 19, 1 << 20                       # shorter than its new tokens; too long
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = _prefill(query, cache, w, tables, starts, ctx, 0.07, max_context=140, status=status)
    good = ctx.clone()
    good[2] = good[3] = 0
    ref, bound = latent_prefill(query, cache, w, tables, starts, good, 0.07)
    assert_within(out.cpu(), ref, bound, "prefill")
    assert (out[70:100] == 0).all()
    assert (out[40:56] == 0).all()                     # these rows see the bad block alone
    assert int(status) == (BAD_BLOCK | BAD_CONTEXT)
    # starts that decrease, pass the tokens, or are longer than the grid: rows left as they were
    status.zero_()
    starts = torch.tensor([0, 40, 30, 50, 126, 126], dtype=torch.int32)
    ctx = torch.tensor([140, 30, 30, 13, 28], dtype=torch.int32)
    out = _prefill(query, cache, w, tables, starts, ctx, 0.07, max_new=40, max_context=140,
                   status=status)
    assert (out[50:] == 9).all() and int(status) & BAD_CONTEXT


def test_prefill_repeats_from_a_graph_and_on_two_streams():
    from paged_kv_cache_415_b200 import binding as B
    x = [t.cuda() for t in _prompt(4, 512, 16, [200, 70], [0, 64], torch.bfloat16, 7)]
    query, cache, w, tables, starts, ctx = x
    n = B.pa_latent_prefill_workspace_size(2, 4, 512, 16, 200)
    spaces = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(2)]
    outs = [torch.empty(270, 4, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    first = _prefill(*x, 0.07)
    torch.cuda.synchronize()
    for _ in range(4):
        for o, s, st in zip(outs, spaces, (torch.cuda.Stream(), torch.cuda.Stream())):
            B.pa_latent_prefill(o, query, cache, w, tables, starts, ctx, 200, 200, 0.07, s,
                                stream=st)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], first) and torch.equal(outs[1], first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.pa_latent_prefill(outs[0], query, cache, w, tables, starts, ctx, 200, 200, 0.07,
                            spaces[0])
    query.mul_(0.5)
    graph.replay()
    assert torch.equal(outs[0], _prefill(*x, 0.07))


# ---------------------------------------------------------------------------
# Together: a prompt, then decode steps
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_prompt_then_steps(dtype):
    """Two sequences: their prompts appended and attended to (expanded), then
    three decode steps (append, absorbed attention) through LatentDecodeStep.
    The decode of a prompt's last token, its value projection applied to the
    latent output, is what the expanded form gives for it."""
    from paged_kv_cache_415_b200 import binding as B
    from paged_kv_cache_415_b200.step import LatentDecodeStep
    g = torch.Generator().manual_seed(12)
    heads, lat, block, prompt, steps = 6, 256, 16, [70, 5], 3
    longest = max(prompt) + steps
    blocks_each = -(-longest // block)
    tables = torch.randperm(2 * blocks_each + 2, generator=g)[:2 * blocks_each].view(2, -1).int()
    cache = torch.full((2 * blocks_each + 2, block, lat + 64), float("nan"), dtype=dtype).cuda()
    table = angle_table(longest, 64)
    w_kv = (torch.randn(heads, 256, lat, generator=g) * lat ** -0.5).to(dtype)
    weight = (torch.randn(lat, generator=g) * 0.2 + 1).to(dtype)
    scale = 192 ** -0.5

    def slot(s, t):
        return int(tables[s, t // block]) * block + t % block

    pos = torch.cat([torch.arange(n) for n in prompt])
    owner = [s for s, n in enumerate(prompt) for _ in range(n)]
    slots = torch.tensor([slot(s, int(t)) for s, t in zip(owner, pos)])
    rows = torch.randn(len(pos), lat + 64, generator=g).to(dtype)
    query = torch.randn(len(pos), heads, 192, generator=g).to(dtype)
    q = query.cuda()
    B.pa_latent_append(q[..., 128:], q[..., 128:], rows.cuda(), cache, slots.cuda(), pos.cuda(),
                       table.cuda(), weight=weight.cuda())
    starts = torch.tensor([0, 70, 75], dtype=torch.int32)
    ctx = torch.tensor(prompt, dtype=torch.int32)
    out = _prefill(q, cache, w_kv, tables, starts, ctx, scale)
    pool = cache.cpu()
    ref, bound = latent_prefill(q.cpu(), pool, w_kv, tables, starts, ctx, scale)
    assert_within(out.cpu(), ref, bound, "prompt")
    # the appended rows are the definition's
    c = normed(rows[:, :lat], weight, 1e-6)
    got = pool.flatten(0, 1)[slots].to(F64)
    assert ((got[:, :lat] - c).abs() <= c.abs() * (half_step(dtype) + 2.0 ** -19) + 2.0 ** -25).all()

    last = starts[1:].long() - 1
    absorbed = torch.einsum("she,hel->shl", q.cpu()[last][..., :128].to(F64),
                            w_kv[:, :128].to(F64)).to(dtype)
    dq = torch.cat([absorbed, q.cpu()[last][..., 128:]], -1)
    lat_out = _decode(dq, pool, tables, ctx, scale)
    value = torch.einsum("shl,hel->she", lat_out.cpu().to(F64), w_kv[:, 128:].to(F64))
    # the roundings of the absorbed query and the latent output, and both forms' own
    diff = (value - out.cpu()[last].to(F64)).abs()
    assert diff.max() <= 40 * half_step(dtype) * value.abs().max()

    stepper = LatentDecodeStep(cache, 2, heads, longest)
    for i in range(steps):
        ctx = ctx + 1
        p = ctx.long() - 1
        new_rows = torch.randn(2, lat + 64, generator=g).to(dtype)
        sq = torch.randn(2, heads, lat + 64, generator=g).to(dtype)
        s_map = torch.tensor([slot(s, int(p[s])) for s in range(2)])
        dev_q = sq.cuda()
        got = stepper(dev_q, tables.cuda(), ctx.cuda(), scale, new_latent=new_rows.cuda(),
                      slot_mapping=s_map.cuda(), positions=p.cuda(), cos_sin=table.cuda(),
                      weight=weight.cuda())
        turned, _ = rotated(sq[..., lat:].to(F64), table, p, False)
        assert ((dev_q.cpu()[..., lat:].to(F64) - turned).abs() <= 2 * half_step(dtype)
                * sq[..., lat:].abs().max()).all()
        ref, bound = latent_decode(dev_q.cpu(), cache.cpu(), tables, ctx, scale)
        assert_within(got.cpu(), ref, bound, f"step {i}")
    assert int(stepper.d_status) == 0


def test_attend_bound_is_tight_enough_to_fail():
    """The oracle with a planted mistake (one token too many) leaves the bound."""
    g = torch.Generator().manual_seed(0)
    rows = torch.randn(40, 320, generator=g, dtype=F64)
    q = torch.randn(4, 320, generator=g, dtype=F64)
    seen = torch.ones(4, 40, dtype=torch.bool)
    ref, bound = attend(q, rows, rows[:, :256], seen, 0.05, torch.float16)
    seen[:, 39] = False
    wrong, _ = attend(q, rows, rows[:, :256], seen, 0.05, torch.float16)
    with pytest.raises(AssertionError):
        assert_within(wrong, ref, bound, "planted")


# ---------------------------------------------------------------------------
# Wide groups, nothing to do, values that are not finite
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("heads,lat", [(64, 256), (128, 256), (48, 512), (17, 256)])
def test_decode_group_widths(heads, lat):
    g = torch.Generator().manual_seed(heads + lat)
    context = [333, 64, 2, 1025]
    cache, tables = _pool(context, 16, lat, torch.bfloat16, g)
    query = torch.randn(len(context), heads, lat + 64, generator=g).to(torch.bfloat16)
    ctx = torch.tensor(context, dtype=torch.int32)
    out = _decode(query, cache, tables, ctx, 0.05)
    ref, bound = latent_decode(query, cache, tables, ctx, 0.05)
    assert_within(out.cpu(), ref, bound, "decode")


def test_nothing_to_do():
    """Empty contexts alone, no sequences, no new tokens."""
    from paged_kv_cache_415_b200 import binding as B
    g = torch.Generator().manual_seed(9)
    cache, tables = _pool([0, 0, 0], 16, 512, torch.float16, g)
    query = torch.randn(3, 20, 576, generator=g).to(torch.float16)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    empty = torch.zeros(3, dtype=torch.int32)
    assert B.pa_latent_decode_workspace_size(3, 20, 512, 16, 0) == 0
    assert (_decode(query, cache, tables, empty, 0.1, max_context=0, status=status) == 0).all()
    assert (_decode(query, cache, tables, empty, 0.1, max_context=900, status=status) == 0).all()
    assert _decode(query[:0], cache, tables[:0], empty[:0], 0.1, max_context=64).shape[0] == 0
    q = torch.randn(4, 2, 192, generator=g).to(torch.float16)
    w = torch.randn(2, 256, 512, generator=g).to(torch.float16)
    starts = torch.zeros(4, dtype=torch.int32)
    out = _prefill(q, cache, w, tables, starts, empty, 0.1, max_new=4, max_context=16,
                   status=status)
    assert (out == 9).all()
    out = _prefill(q, cache, w, tables, starts, empty, 0.1, max_new=0, max_context=0, status=status)
    assert (out == 9).all() and int(status) == 0


@pytest.mark.parametrize("masked", [1, 64, 100, 200])
def test_decode_scores_of_minus_infinity(masked):
    """The first `masked` tokens score minus infinity (through their rotated
    part): they weigh nothing, whichever tile the first finite score is in."""
    g = torch.Generator().manual_seed(masked)
    cache, tables = _pool([300], 16, 256, torch.bfloat16, g)
    query = torch.randn(1, 16, 320, generator=g).to(torch.bfloat16)
    query[..., 256] = query[..., 256].abs() + 0.5
    t = torch.arange(masked)
    cache[tables[0][t // 16].long(), t % 16, 256] = 0
    ctx = torch.tensor([300], dtype=torch.int32)
    rows, _ = context_rows(cache, tables[0], 300)
    seen = (torch.arange(300) >= masked).expand(16, 300)
    ref, bound = attend(query[0].to(F64), rows, rows[:, :256], seen, 0.05, torch.bfloat16)
    cache[tables[0][t // 16].long(), t % 16, 256] = -float("inf")
    out = _decode(query, cache, tables, ctx, 0.05)
    assert_within(out.cpu()[0], ref, bound, "decode")


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("worst", [float("inf"), float("nan")])
def test_prefill_later_tokens_do_not_reach_back(dtype, worst):
    """Tokens that are not finite: queries before them are what they are
    without them, those that see them are not finite."""
    x = _prompt(3, 256, 16, [200, 90], [100, 0], dtype, 21)
    query, cache, w, tables, starts, ctx = x
    first = {0: 250, 1: 40}                            # of the new ones, 150 and 40
    for s, t in first.items():
        cache[tables[s, t // 16], t % 16] = 0
        cache[tables[s, (t + 9) // 16], (t + 9) % 16] = 0
    ref, bound = latent_prefill(*x, 0.07)
    for s, t in first.items():
        cache[tables[s, t // 16], t % 16, :256] = worst
        cache[tables[s, (t + 9) // 16], (t + 9) % 16, 7] = worst
    out = _prefill(*x, 0.07).cpu()
    for rows in (slice(0, 150), slice(200, 240)):
        assert_within(out[rows], ref[rows], bound[rows], "before")
    for rows in (slice(150, 200), slice(240, 290)):
        assert not torch.isfinite(out[rows]).all(-1).any()


def test_prefill_value_past_the_type():
    """A value past fp16, that its context's mean is not: as any other."""
    x = _prompt(2, 512, 32, [60], [40], torch.float16, 22)
    query, cache, w, tables, starts, ctx = x
    # head 0's value element 5 of token 20 is about 300 * 512 * 0.8, of others 300 * 512^0.5
    w[0, 128 + 5] = torch.where(cache[tables[0, 0], 20, :512] < 0, -300.0, 300.0).half()
    out = _prefill(*x, 0.07).cpu()
    ref, bound = latent_prefill(*x, 0.07)
    assert ref.abs().max() < 60000
    assert_within(out, ref, bound, "prefill")


@pytest.mark.parametrize("power", [-40, 40])
def test_prefill_follows_the_values_scale(power):
    """Values times a power of two give outputs times it, and are of no account
    for the other heads."""
    x = _prompt(3, 256, 16, [150, 33], [20, 70], torch.bfloat16, 23)
    query, cache, w, tables, starts, ctx = x
    out = _prefill(*x, 0.07)
    ref, bound = latent_prefill(*x, 0.07)
    w[1, 128:] = torch.ldexp(w[1, 128:].float(), torch.tensor(power)).bfloat16()
    got = _prefill(query, cache, w, tables, starts, ctx, 0.07)
    assert torch.equal(got[:, ::2], out[:, ::2])
    assert_within(torch.ldexp(got[:, 1].cpu().to(F64), torch.tensor(-power)), ref[:, 1],
                  bound[:, 1], "scaled")


def test_prefill_values_of_uneven_size():
    """Tokens whose values differ by powers of two up to 2^12, within the 32
    that share one and between them; a context whose values are all zero."""
    x = _prompt(2, 256, 16, [200, 20], [30, 0], torch.bfloat16, 24)
    query, cache, w, tables, starts, ctx = x
    t = torch.arange(230)
    grow = torch.where(t < 100, t % 7, t % 13).float()
    rows = cache[tables[0][t // 16].long(), t % 16]
    rows[:, :256] = (rows[:, :256].float() * 2.0 ** grow[:, None] / 64).bfloat16()
    cache[tables[0][t // 16].long(), t % 16] = rows
    w[:, :128] /= 64                                   # (scores of an ordinary size)
    cache[tables[1, 0], :, :256] = 0
    cache[tables[1, 1], :4, :256] = 0
    out = _prefill(*x, 0.07).cpu()
    ref, bound = latent_prefill(*x, 0.07)
    assert_within(out, ref, bound, "prefill")
    assert (out[200:] == 0).all()


@pytest.mark.parametrize("heads,new,old", [
    (20, [1, 300, 300, 0, 513, 129, 17], [0, 40, 40, 0, 3, 400, 290]),    # ranked by size, with ties
    (40, [3, 2, 1, 4], [70, 0, 200, 5]),                                  # a pair a sequence
    (2, [1 + i % 5 for i in range(150)], [i % 3 for i in range(150)]),    # too many to rank
])
def test_prefill_many_blocks(heads, new, old):
    """More blocks than fit at once: the order in which they are taken is of
    no account, a bad length among them neither."""
    x = _prompt(heads, 256, 16, new, old, torch.bfloat16, 31)
    ctx = x[-1].clone()
    ctx[1] = -7
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    top = int(x[-1].max())
    out = _prefill(*x[:-1], ctx, 192 ** -0.5, max_context=top, status=status).cpu()
    first = new[0]
    assert (out[first:first + new[1]] == 0).all() and int(status) == BAD_CONTEXT
    ctx[1] = 0
    ref, bound = latent_prefill(*x[:-1], ctx, 192 ** -0.5)
    assert_within(out, ref, bound, "prefill")
