"""Rotating decode steps of several batch sizes through one DecodeStep."""
import pytest
import torch

from tests.latent_reference import angle_table

pytestmark = pytest.mark.gpu
HQ, HKV, D, BLOCK = 8, 2, 128, 16


def _batch(seqs, seed, dtype):
    g = torch.Generator().manual_seed(seed)
    ctx = torch.tensor([1 + (11 * i) % 40 for i in range(seqs)], dtype=torch.int32)
    tables = torch.arange(3 * seqs, dtype=torch.int32).view(seqs, 3)
    p = ctx.long() - 1
    slots = tables[torch.arange(seqs), p // BLOCK].long() * BLOCK + p % BLOCK
    x = dict(query=torch.randn(seqs, HQ, D, generator=g).to(dtype),
             new_key=torch.randn(seqs, HKV, D, generator=g).to(dtype),
             new_value=torch.randn(seqs, HKV, D, generator=g).to(dtype),
             block_tables=tables, context_lens=ctx, slot_mapping=slots, positions=p)
    return {k: v.cuda() for k, v in x.items()}


def _want(b, pools, rotation):
    """Rotate first, then the step on rotated rows, over copies of the pools."""
    from paged_kv_cache_415_b200 import binding as B
    from paged_kv_cache_415_b200.step import DecodeStep
    pools = [p.clone() for p in pools]
    q = torch.empty_like(b["query"])
    B.pa_rope_append(q, b["query"], b["new_key"], b["new_value"], *pools, b["slot_mapping"],
                     b["positions"], rotation.cos_sin)
    return DecodeStep(*pools, q.shape[0], HQ, 48)(q, b["block_tables"], b["context_lens"], 0.1)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_graphs_of_several_batch_sizes(dtype):
    """A graph each of two batch sizes, an eager step of a third and tensors
    allocated in between; replayed in turn with new queries, each gives its
    own batch's result and no other tensor changes."""
    from paged_kv_cache_415_b200.step import DecodeStep, Rotation
    pools = [torch.randn(32, BLOCK, HKV, D, device="cuda").to(dtype) for _ in range(2)]
    rotation = Rotation(angle_table(64, D).cuda())
    step = DecodeStep(*pools, 7, HQ, 48)
    batches = [_batch(s, 10 + s, dtype) for s in (3, 7)]
    outs, graphs, bystanders = [], [], []
    others = lambda: [torch.full((n, HQ, D), 5.0, dtype=dtype, device="cuda")
                      for n in (1, 2, 3, 5, 7) for _ in range(4)]
    for b in batches:
        rows = {k: v for k, v in b.items() if k not in ("query", "block_tables", "context_lens")}
        outs.append(torch.zeros_like(b["query"]))
        graphs.append(step.graph(b["query"], b["block_tables"], b["context_lens"], 0.1, outs[-1],
                                 rotation=rotation, **rows))
        bystanders += others()
    third = _batch(5, 99, dtype)
    want = _want(third, pools, rotation)
    rows = {k: third[k] for k in ("new_key", "new_value", "slot_mapping", "positions")}
    got = step(third["query"], third["block_tables"], third["context_lens"], 0.1,
               rotation=rotation, **rows)
    assert torch.equal(got, want)
    bystanders += others()
    assert all(g.step is step for g in graphs)
    del step
    bystanders += others()
    for turn in range(3):
        for b, out, graph in zip(batches, outs, graphs):
            b["query"].mul_(-0.75)
            want = _want(b, pools, rotation)
            out.zero_()
            graph.replay()
            assert torch.equal(out, want), turn
    assert all((t == 5).all() for t in bystanders)


def _host(b):
    return {k: v.cpu().pin_memory() for k, v in b.items()}


def test_rotating_steps_fed_from_the_host():
    """run_from_host, and HostPipeline eagerly and from graphs: what the step
    gives on the same inputs on the device."""
    from paged_kv_cache_415_b200.step import DecodeStep, HostPipeline, Rotation
    dtype, seqs = torch.bfloat16, 5
    pools = [torch.randn(32, BLOCK, HKV, D, device="cuda").to(dtype) for _ in range(2)]
    rotation = Rotation(angle_table(64, D).cuda())
    step = DecodeStep(*pools, seqs, HQ, 48)
    batches = [_batch(seqs, 70 + i, dtype) for i in range(6)]
    want = []
    for b in batches:
        rows = {k: v for k, v in b.items() if k not in ("query", "block_tables", "context_lens")}
        want.append(step(b["query"], b["block_tables"], b["context_lens"], 0.1, rotation=rotation,
                         **rows).cpu())
    host = _host(batches[0]) | {"out": torch.empty(seqs, HQ, D, dtype=dtype).pin_memory()}
    dev = {k: torch.empty_like(v, device="cuda") for k, v in host.items()}
    out = step.run_from_host(host, dev, 0.1, rotation=rotation)
    torch.cuda.synchronize()
    assert torch.equal(out, want[0])
    like = batches[0] | {"out": batches[0]["query"]}
    for graphs in (False, True):
        pipe = HostPipeline(step, like, use_graphs=graphs, rotation=rotation)
        outs = [torch.zeros(seqs, HQ, D, dtype=dtype).pin_memory() for _ in batches]
        packed = []
        for b in batches:
            buf, views = pipe.host_buffer()
            for name, t in b.items():
                views[name].copy_(t)
            packed.append(buf)
        for buf, o in zip(packed, outs):
            pipe.submit(buf, 0.1, o)
        pipe.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want)), graphs
    assert int(step.d_status) == 0
    with pytest.raises(ValueError, match="positions"):
        HostPipeline(step, {k: v for k, v in like.items() if k != "positions"}, rotation=rotation)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_latent_steps_repeat(dtype):
    """A step that rotates from query_rope can be taken again and captured:
    the same rows and outputs each time, those of rotating in place once."""
    from paged_kv_cache_415_b200.step import LatentDecodeStep
    seqs, heads, lat = 4, 20, 256
    g = torch.Generator().manual_seed(5)
    ctx = torch.tensor([1, 16, 70, 33], dtype=torch.int32)
    tables = torch.arange(5 * seqs, dtype=torch.int32).view(seqs, 5)
    pool = torch.randn(24, BLOCK, lat + 64, generator=g).to(dtype).cuda()
    p = ctx.long() - 1
    slots = tables[torch.arange(seqs), p // BLOCK].long() * BLOCK + p % BLOCK
    tables, ctx = tables.cuda(), ctx.cuda()
    rows = dict(new_latent=torch.randn(seqs, lat + 64, generator=g).to(dtype).cuda(),
                slot_mapping=slots.cuda(), positions=p.cuda(), cos_sin=angle_table(80, 64).cuda(),
                weight=(torch.rand(lat, generator=g) + 0.5).to(dtype).cuda())
    projected = torch.randn(seqs, heads, 192, generator=g).to(dtype).cuda()
    turned = projected[..., 128:]                    # as the projection leaves them
    absorbed = torch.randn(seqs, heads, lat + 64, generator=g).to(dtype).cuda()

    in_place = absorbed.clone()
    in_place[..., lat:] = turned
    pools = [pool.clone() for _ in range(2)]
    want = LatentDecodeStep(pools[0], seqs, heads, 80)(in_place, tables, ctx, 0.05, **rows)
    step = LatentDecodeStep(pools[1], seqs, heads, 80)
    query = absorbed.clone()
    for bound in (None, 80, 70):
        got = step(query, tables, ctx, 0.05, query_rope=turned, max_context_len=bound, **rows)
        assert torch.equal(got, want) and torch.equal(query, in_place)
        assert torch.equal(*pools)
    out = torch.zeros_like(want)
    query = absorbed.clone()
    graph = step.graph(query, tables, ctx, 0.05, out, query_rope=turned, **rows)
    for _ in range(2):
        out.zero_()
        graph.replay()
        assert torch.equal(out, want) and torch.equal(query, in_place) and torch.equal(*pools)
    assert int(step.d_status) == 0
    with pytest.raises(ValueError, match="query_rope"):
        step.graph(query, tables, ctx, 0.05, out, **rows)
    with pytest.raises(ValueError, match="new_latent"):
        step(query, tables, ctx, 0.05, query_rope=turned)
