"""pa_rope_append and pa_latent_append against their 64-bit definitions."""
import pytest
import torch

from tests.latent_reference import (F64, angle_table, assert_rounded, half_step, normed, rotated)

pytestmark = pytest.mark.gpu
BAD_SLOT, BAD_POSITION = 2, 32


def _inputs(tokens, hq, hkv, d, dtype, block, rot, seed=0, blocks=None, positions=64):
    g = torch.Generator().manual_seed(seed)
    rows = (torch.randn(tokens, (hq + 2 * hkv) * d, generator=g) * 2).to(dtype)
    blocks = blocks or -(-tokens // block) + 2
    return dict(
        rows=rows, q=rows[:, :hq * d].unflatten(1, (hq, d)),
        k=rows[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d)),
        v=rows[:, (hq + hkv) * d:].unflatten(1, (hkv, d)),
        pools=[torch.randn(blocks, block, hkv, d, generator=g).to(dtype) for _ in range(2)],
        slots=torch.randperm(blocks * block, generator=g)[:tokens],
        pos=torch.randint(0, positions, (tokens,), generator=g),
        table=angle_table(positions, rot),
        qw=(torch.randn(d, generator=g) * 0.3 + 1).to(dtype),
        kw=(torch.randn(d, generator=g) * 0.3 + 1).to(dtype))


def _device(x, hq, hkv, d):
    rows = x["rows"].cuda()
    return dict(q=rows[:, :hq * d].unflatten(1, (hq, d)),
                k=rows[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d)),
                v=rows[:, (hq + hkv) * d:].unflatten(1, (hkv, d)),
                pools=[p.cuda() for p in x["pools"]], slots=x["slots"].cuda(),
                pos=x["pos"].cuda(), table=x["table"].cuda(), qw=x["qw"].cuda(), kw=x["kw"].cuda(),
                status=torch.zeros(1, dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("tokens,hq,hkv,d,rot,block,norm,interleaved", [
    (1, 1, 1, 64, 64, 16, True, False),
    (3, 8, 2, 128, 128, 8, True, True),
    (17, 5, 5, 128, 64, 32, False, False),
    (5, 3, 1, 64, 16, 16, True, False),
    (4, 7, 3, 128, 48, 16, True, False),
    (4, 2, 2, 64, 0, 16, True, True),
    (9, 33, 11, 64, 32, 16, False, True),
    (700, 32, 8, 128, 128, 16, True, False),       # several rows a lane group
    (701, 64, 4, 64, 64, 32, True, True),
])
def test_rope_append(dtype, tokens, hq, hkv, d, rot, block, norm, interleaved):
    from paged_kv_cache_415_b200 import binding as B
    x = _inputs(tokens, hq, hkv, d, dtype, block, rot, seed=tokens + hq)
    if tokens > 4:                                  # padding, no slot, bad slot, bad position
        x["pos"][1], x["slots"][2] = -1, -7
        x["slots"][3], x["pos"][4] = x["pools"][0].shape[0] * block, x["table"].shape[0]
    c = _device(x, hq, hkv, d)
    qw, kw = (c["qw"], c["kw"]) if norm else (None, None)
    out = torch.full((tokens, hq, d), 7.0, dtype=dtype, device="cuda")
    B.pa_rope_append(out, c["q"], c["k"], c["v"], *c["pools"], c["slots"], c["pos"], c["table"],
                     q_weight=qw, k_weight=kw, eps=1e-5, interleaved=interleaved,
                     d_status=c["status"])
    live = (x["pos"] >= 0) & (x["pos"] < x["table"].shape[0])
    q, q_off = rotated(normed(x["q"], x["qw"] if norm else None, 1e-5), x["table"], x["pos"],
                       interleaved)
    k, k_off = rotated(normed(x["k"], x["kw"] if norm else None, 1e-5), x["table"], x["pos"],
                       interleaved)
    assert_rounded(out.cpu()[live], q[live], q_off[live], dtype, "queries")
    assert (out.cpu()[~live] == 7).all()
    total = x["pools"][0].shape[0] * block
    put = live & (x["slots"] >= 0) & (x["slots"] < total)
    kc, vc = (p.cpu().flatten(0, 1) for p in c["pools"])
    assert_rounded(kc[x["slots"][put]], k[put], k_off[put], dtype, "keys")
    assert torch.equal(vc[x["slots"][put]], x["v"][put])
    kept = torch.ones(total, dtype=torch.bool)
    kept[x["slots"][put]] = False
    for got, was in zip((kc, vc), x["pools"]):
        assert torch.equal(got[kept], was.flatten(0, 1)[kept])
    assert int(c["status"]) == ((BAD_SLOT | BAD_POSITION) if tokens > 4 else 0)


def test_rope_append_in_place_and_on_a_stream():
    """query_out may be the query inside the fused projection; a second pass
    over the same state on another stream repeats the first bit for bit."""
    from paged_kv_cache_415_b200 import binding as B
    x = _inputs(33, 8, 2, 128, torch.bfloat16, 16, 128, seed=3)
    c = _device(x, 8, 2, 128)
    out = torch.empty(33, 8, 128, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    B.pa_rope_append(out, c["q"], c["k"], c["v"], *c["pools"], c["slots"], c["pos"], c["table"],
                     stream=side)
    side.synchronize()
    k_first = c["k"].clone()
    pools = [p.clone() for p in c["pools"]]
    with torch.cuda.stream(side):
        B.pa_rope_append(c["q"], c["q"], c["k"], c["v"], *c["pools"], c["slots"], c["pos"],
                         c["table"])
    side.synchronize()
    assert torch.equal(c["q"], out) and torch.equal(c["k"], k_first)
    assert all(torch.equal(a, b) for a, b in zip(pools, c["pools"]))


@pytest.mark.parametrize("codes", ["e4m3", "int8"])
@pytest.mark.parametrize("row_scaled", [False, True])
@pytest.mark.parametrize("d,block", [(64, 8), (128, 16)])
def test_rope_append_one_byte_pools(codes, row_scaled, d, block):
    from paged_kv_cache_415_b200 import binding as B
    tokens, hq, hkv = 21, 4, 2
    x = _inputs(tokens, hq, hkv, d, torch.bfloat16, block, d, seed=11)
    x["rows"][5, hq * d:(hq + hkv) * d] = 0                         # a key row of zeros
    x["rows"][6, (hq + hkv) * d:] *= 1000                           # values past the top code
    c = _device(x, hq, hkv, d)
    blocks = x["pools"][0].shape[0]
    kind = torch.float8_e4m3fn if codes == "e4m3" else torch.int8
    pools = [torch.zeros(blocks, block, hkv, d, dtype=kind, device="cuda") for _ in range(2)]
    scales = [torch.full((blocks, hkv, block), -1.0, device="cuda") for _ in range(2)]
    ks, vs = (0.011, 0.07)
    out = torch.empty(tokens, hq, d, dtype=torch.bfloat16, device="cuda")
    more = dict(k_scales=scales[0], v_scales=scales[1]) if row_scaled \
        else dict(k_scale=ks, v_scale=vs)
    B.pa_rope_append(out, c["q"], c["k"], c["v"], *pools, c["slots"], c["pos"], c["table"], **more)
    top = 448.0 if codes == "e4m3" else 127.0
    low = -448.0 if codes == "e4m3" else -128.0
    k, k_off = rotated(x["k"].to(F64), x["table"], x["pos"], False)
    v = x["v"].to(F64)
    for ref, off, pool, scale, table in ((k, k_off, pools[0], ks, scales[0]),
                                         (v, torch.zeros_like(v), pools[1], vs, scales[1])):
        got = pool.float().cpu().to(F64).flatten(0, 1)[x["slots"]]
        if row_scaled:
            stored = table.cpu().to(F64)[x["slots"] // block, :, x["slots"] % block]
            want = ref.abs().amax(-1) / top
            assert ((stored - want).abs() <= want * 2.0 ** -23 + off.amax(-1) / top).all()
            scale = stored[..., None]
            got_value = got * scale
        else:
            got_value = got * scale
            ref = ref.clamp(low * scale, top * scale)
        # half a step of the code, the fp32 error before it, and the product with 1 / scale
        step = (half_step(kind) * ref.abs() + 2.0 ** -10 * scale) if codes == "e4m3" \
            else 0.5 * scale
        bound = step + off + ref.abs() * 2.0 ** -21
        assert ((got_value - ref).abs() <= bound).all(), (codes, row_scaled)
    zero = pools[0].float().cpu().flatten(0, 1)[x["slots"][5]]
    assert (zero == 0).all()
    if row_scaled:
        untouched = torch.ones(blocks * block, dtype=torch.bool)
        untouched[x["slots"]] = False
        flat = scales[0].cpu().transpose(1, 2).flatten(0, 1)
        assert (flat[untouched] == -1).all()


def test_rope_append_then_decode_uses_the_rotated_rows():
    """A step as a layer runs it: append with rotation, then attention over
    the pool, against the same step on rows rotated beforehand."""
    from paged_kv_cache_415_b200 import binding as B
    s, hq, hkv, d, block = 3, 8, 2, 128, 16
    x = _inputs(s, hq, hkv, d, torch.float16, block, d, seed=5, blocks=8)
    c = _device(x, hq, hkv, d)
    ctx = torch.tensor([1, 16, 37], dtype=torch.int32)
    tables = torch.tensor([[0, 0, 0], [1, 0, 0], [2, 3, 4]], dtype=torch.int32)
    slots = torch.tensor([int(tables[i, (n - 1) // block]) * block + (n - 1) % block
                          for i, n in enumerate(ctx.tolist())])
    pools2 = [p.clone() for p in c["pools"]]
    q = torch.empty(s, hq, d, dtype=torch.float16, device="cuda")
    B.pa_rope_append(q, c["q"], c["k"], c["v"], *c["pools"], slots.cuda(), c["pos"], c["table"],
                     q_weight=c["qw"], k_weight=c["kw"])
    out = torch.empty_like(q)
    B.pa_paged_decode(out, q, *c["pools"], tables.cuda(), ctx.cuda(), 37, d ** -0.5)
    k_rot = c["pools"][0].flatten(0, 1)[slots.cuda()].contiguous()
    B.pa_reshape_and_cache(k_rot, c["v"].contiguous(), *pools2, slots.cuda())
    out2 = torch.empty_like(q)
    B.pa_paged_decode(out2, q, *pools2, tables.cuda(), ctx.cuda(), 37, d ** -0.5)
    assert torch.equal(out, out2)


def _latent_inputs(tokens, heads, lat, block, dtype, seed, blocks=None):
    g = torch.Generator().manual_seed(seed)
    blocks = blocks or -(-tokens // block) + 2
    return dict(q=(torch.randn(tokens, heads, 128 + 64, generator=g) * 2).to(dtype),
                rows=(torch.randn(tokens, lat + 64 + 8, generator=g) * 2).to(dtype),
                cache=torch.randn(blocks, block, lat + 64, generator=g).to(dtype),
                slots=torch.randperm(blocks * block, generator=g)[:tokens],
                pos=torch.randint(0, 50, (tokens,), generator=g), table=angle_table(50, 64),
                weight=(torch.randn(lat, generator=g) * 0.3 + 1).to(dtype))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("tokens,heads,lat,block,norm,interleaved", [
    (1, 1, 512, 16, True, True), (6, 3, 256, 8, True, False), (19, 16, 512, 64, False, True),
    (7, 128, 256, 32, True, False), (1500, 61, 512, 16, True, True),
])
def test_latent_append(dtype, tokens, heads, lat, block, norm, interleaved):
    from paged_kv_cache_415_b200 import binding as B
    x = _latent_inputs(tokens, heads, lat, block, dtype, seed=tokens)
    if tokens > 4:
        x["pos"][1], x["slots"][2] = -1, -1
        x["slots"][3], x["pos"][4] = x["cache"].shape[0] * block, 50
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cache, q = x["cache"].cuda(), x["q"].cuda()
    query = torch.full((tokens, heads, lat + 64), 3.0, dtype=dtype, device="cuda")
    rows = x["rows"].cuda()[:, :lat + 64]                            # strided
    B.pa_latent_append(query[..., lat:], q[..., 128:], rows, cache, x["slots"].cuda(),
                       x["pos"].cuda(), x["table"].cuda(),
                       weight=x["weight"].cuda() if norm else None, eps=1e-6,
                       interleaved=interleaved, d_status=status)
    live = (x["pos"] >= 0) & (x["pos"] < 50)
    ref, off = rotated(x["q"][..., 128:].to(F64), x["table"], x["pos"], interleaved)
    got = query.cpu()
    assert_rounded(got[live][..., lat:], ref[live], off[live], dtype, "queries")
    assert (got[..., :lat] == 3).all() and (got[~live] == 3).all()
    total = x["cache"].shape[0] * block
    put = live & (x["slots"] >= 0) & (x["slots"] < total)
    flat = cache.cpu().flatten(0, 1)
    c = normed(x["rows"][:, :lat], x["weight"] if norm else None, 1e-6)
    # sum of squares: 16 fmas and 5 shuffle steps, halved by the root; rsqrtf; two products
    c_off = c.abs() * 2.0 ** -20 if norm else torch.zeros_like(c)
    assert_rounded(flat[x["slots"][put], :lat], c[put], c_off[put], dtype, "latent")
    k, k_off = rotated(x["rows"][:, None, lat:lat + 64].to(F64), x["table"], x["pos"], interleaved)
    assert_rounded(flat[x["slots"][put], lat:], k[put, 0], k_off[put, 0], dtype, "key part")
    kept = torch.ones(total, dtype=torch.bool)
    kept[x["slots"][put]] = False
    assert torch.equal(flat[kept], x["cache"].flatten(0, 1)[kept])
    assert int(status) == ((BAD_SLOT | BAD_POSITION) if tokens > 4 else 0)


def test_latent_append_without_queries_and_in_place():
    from paged_kv_cache_415_b200 import binding as B
    x = _latent_inputs(5, 4, 256, 16, torch.bfloat16, seed=9)
    args = (x["slots"].cuda(), x["pos"].cuda(), x["table"].cuda())
    rows = x["rows"].cuda()[:, :320]
    caches = [x["cache"].cuda() for _ in range(2)]
    B.pa_latent_append(None, None, rows, caches[0], *args)
    q = x["q"].cuda()
    apart = torch.empty(5, 4, 64, dtype=torch.bfloat16, device="cuda")
    B.pa_latent_append(apart, q[..., 128:], rows, caches[1], *args)
    assert torch.equal(caches[0], caches[1])
    B.pa_latent_append(q[..., 128:], q[..., 128:], rows, caches[1], *args)
    assert torch.equal(q[..., 128:], apart) and torch.equal(q[..., :128].cpu(), x["q"][..., :128])


@pytest.mark.slow
def test_appends_past_32_bit_offsets():
    """Slots whose element offsets pass 2^31."""
    from paged_kv_cache_415_b200 import binding as B
    dtype, block = torch.bfloat16, 16
    x = _latent_inputs(4, 2, 512, block, dtype, seed=2)
    blocks = (1 << 31) // (block * 576) + 3
    cache = torch.empty(blocks, block, 576, dtype=dtype, device="cuda")
    slots = torch.tensor([0, blocks * block - 1, blocks * block - 2, blocks * block - 33])
    rows = x["rows"].cuda()[:, :576]
    B.pa_latent_append(None, None, rows, cache, slots.cuda(), x["pos"].cuda(), x["table"].cuda())
    got = cache.flatten(0, 1)[slots.cuda()].cpu()
    assert torch.equal(got[:, :512], x["rows"][:, :512])
    del cache
    blocks = (1 << 31) // (block * 8 * 128) + 3
    x = _inputs(4, 8, 8, 128, dtype, block, 0, seed=4, blocks=1)
    c = _device(x, 8, 8, 128)
    pools = [torch.empty(blocks, block, 8, 128, dtype=dtype, device="cuda") for _ in range(2)]
    slots = torch.tensor([0, blocks * block - 1, blocks * block - 2, blocks * block - 33])
    out = torch.empty(4, 8, 128, dtype=dtype, device="cuda")
    B.pa_rope_append(out, c["q"], c["k"], c["v"], *pools, slots.cuda(), c["pos"], c["table"])
    for pool, want in zip(pools, (x["k"], x["v"])):
        assert torch.equal(pool.flatten(0, 1)[slots.cuda()].cpu(), want)




@pytest.mark.parametrize("pool", ["16-bit", "e4m3", "int8 rows"])
def test_decode_step_with_a_rotation(pool):
    """DecodeStep given a Rotation: the same result as rotating first and
    taking the step on rotated rows; captured into a graph as well."""
    from paged_kv_cache_415_b200 import binding as B
    from paged_kv_cache_415_b200.step import DecodeStep, Rotation
    s, hq, hkv, d, block = 3, 8, 2, 128, 16
    dtype = torch.bfloat16
    x = _inputs(s, hq, hkv, d, dtype, block, d, seed=21, blocks=8)
    c = _device(x, hq, hkv, d)
    ctx = torch.tensor([1, 16, 37], dtype=torch.int32, device="cuda")
    tables = torch.tensor([[0, 0, 0], [1, 0, 0], [2, 3, 4]], dtype=torch.int32, device="cuda")
    slots = torch.tensor([0, 16 + 15, 4 * 16 + 4], device="cuda")
    kind = {"16-bit": dtype, "e4m3": torch.uint8, "int8 rows": torch.int8}[pool]
    make = lambda: [torch.zeros(8, block, hkv, d, dtype=kind, device="cuda") for _ in range(2)]
    scales = lambda: dict(k_scales=torch.zeros(8, hkv, block, device="cuda"),
                          v_scales=torch.zeros(8, hkv, block, device="cuda")) \
        if pool == "int8 rows" else dict(k_scale=0.02, v_scale=0.02)
    pools, direct = make(), make()
    rot = Rotation(c["table"], c["qw"], c["kw"], 1e-6, False)
    more, more_direct = scales(), scales()
    q = torch.empty(s, hq, d, dtype=dtype, device="cuda")
    B.pa_rope_append(q, c["q"], c["k"], c["v"], *direct, slots, c["pos"], c["table"], c["qw"],
                     c["kw"], **more_direct)
    want = DecodeStep(*direct, s, hq, 37, **more_direct)(q, tables, ctx, d ** -0.5)
    step = DecodeStep(*pools, s, hq, 37, **more)
    before = c["q"].clone()
    got = step(c["q"], tables, ctx, d ** -0.5, new_key=c["k"], new_value=c["v"],
               slot_mapping=slots, positions=c["pos"], rotation=rot)
    assert torch.equal(got, want) and torch.equal(c["q"], before)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(pools, direct))
    out = torch.empty_like(got)
    graph = step.graph(c["q"], tables, ctx, d ** -0.5, out, new_key=c["k"], new_value=c["v"],
                       slot_mapping=slots, positions=c["pos"], rotation=rot)
    out.zero_()
    graph.replay()
    assert torch.equal(out, want) and int(step.d_status) == 0
    with pytest.raises(ValueError):
        step(c["q"], tables, ctx, 1.0, new_key=c["k"], new_value=c["v"], slot_mapping=slots,
             positions=c["pos"], rotation=rot, fused_append=True)
