"""Host-side refusals and size queries of the rotating appends and the latent
pool's calls (CPU only: no call here reaches a kernel launch)."""
import pytest
import torch

FAKE = 1 << 20                       # 16-byte aligned, never dereferenced
OK, INVALID, UNSUPPORTED = 0, 1, 2


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_415_b200 import build
    build.build()
    from paged_kv_cache_415_b200 import binding
    return binding


def _rope(pa, **kw):
    args = dict(query_out=FAKE, query=FAKE, key=FAKE, value=FAKE, k_cache=FAKE, v_cache=FAKE,
                k_scales=None, v_scales=None, slot_mapping=FAKE, positions=FAKE, cos_sin=FAKE,
                q_weight=None, k_weight=None, eps=1e-6, num_tokens=4, num_q_heads=8,
                num_kv_heads=2, head_dim=128, rot_dim=128, max_position=100, interleaved=0,
                query_out_stride=1024, query_stride=1536, key_stride=1536, value_stride=1536,
                block_size=16, num_blocks=10, dtype=0, pool_dtype=0, k_scale=1.0, v_scale=1.0,
                d_status=None, stream=None)
    assert set(kw) <= set(args)
    args.update(kw)
    return pa.LIB.pa_rope_append(*args.values())


@pytest.mark.parametrize("kw,code", [
    (dict(num_tokens=0), OK),
    (dict(num_tokens=-1), INVALID), (dict(query=None), INVALID), (dict(query_out=None), INVALID),
    (dict(key=None), INVALID), (dict(v_cache=None), INVALID), (dict(slot_mapping=None), INVALID),
    (dict(positions=None), INVALID), (dict(cos_sin=None), INVALID),
    (dict(query=FAKE + 8), INVALID), (dict(positions=FAKE + 4), INVALID),
    (dict(cos_sin=FAKE + 4), INVALID), (dict(q_weight=FAKE + 2), INVALID),
    (dict(d_status=FAKE + 1), INVALID), (dict(eps=-1e-6), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(num_q_heads=0), INVALID), (dict(num_kv_heads=0), INVALID), (dict(num_blocks=0), INVALID),
    (dict(max_position=0), INVALID), (dict(rot_dim=-16), INVALID), (dict(rot_dim=144), INVALID),
    (dict(rot_dim=24), UNSUPPORTED), (dict(head_dim=96), UNSUPPORTED),
    (dict(block_size=64), UNSUPPORTED), (dict(dtype=4), UNSUPPORTED),
    (dict(pool_dtype=1), UNSUPPORTED), (dict(pool_dtype=4), UNSUPPORTED),
    (dict(query_out_stride=1016), INVALID), (dict(query_stride=1028), INVALID),
    (dict(key_stride=128), INVALID), (dict(value_stride=0), INVALID),
    (dict(pool_dtype=2, k_scale=0.0), INVALID), (dict(pool_dtype=3, v_scale=float("inf")), INVALID),
    (dict(pool_dtype=2, k_scales=FAKE), INVALID), (dict(k_scales=FAKE, v_scales=FAKE), INVALID),
    (dict(pool_dtype=3, k_scales=FAKE, v_scales=FAKE + 4), INVALID),
])
def test_rope_append_refusals(pa, kw, code):
    assert _rope(pa, **kw) == code


def _append(pa, **kw):
    args = dict(query_out=FAKE, query_rope=FAKE, latent=FAKE, cache=FAKE, slot_mapping=FAKE,
                positions=FAKE, cos_sin=FAKE, weight=None, eps=1e-6, num_tokens=4, num_heads=8,
                latent_dim=512, rope_dim=64, max_position=100, interleaved=0,
                query_out_stride=8 * 576, query_out_head_stride=576, query_stride=8 * 192,
                query_head_stride=192, latent_stride=576, block_size=16, num_blocks=10, dtype=0,
                d_status=None, stream=None)
    assert set(kw) <= set(args)
    args.update(kw)
    return pa.LIB.pa_latent_append(*args.values())


@pytest.mark.parametrize("kw,code", [
    (dict(num_tokens=0), OK),
    (dict(num_tokens=0, num_heads=0, query_out=None, query_rope=None), OK),
    (dict(num_tokens=-1), INVALID), (dict(num_heads=-1), INVALID), (dict(latent=None), INVALID),
    (dict(cache=None), INVALID), (dict(query_out=None), INVALID), (dict(cos_sin=None), INVALID),
    (dict(latent=FAKE + 8), INVALID), (dict(query_rope=FAKE + 8), INVALID),
    (dict(slot_mapping=FAKE + 4), INVALID), (dict(weight=FAKE + 8), INVALID),
    (dict(eps=-1.0), INVALID), (dict(latent_stride=568), INVALID), (dict(latent_stride=580), INVALID),
    (dict(query_head_stride=56), INVALID), (dict(query_out_head_stride=68), INVALID),
    (dict(query_stride=192), INVALID), (dict(query_out_stride=576), INVALID),
    (dict(num_blocks=0), INVALID), (dict(max_position=0), INVALID),
    (dict(latent_dim=384), UNSUPPORTED), (dict(rope_dim=32), UNSUPPORTED),
    (dict(block_size=12), UNSUPPORTED), (dict(dtype=2), UNSUPPORTED),
])
def test_latent_append_refusals(pa, kw, code):
    assert _append(pa, **kw) == code


def _decode(pa, **kw):
    args = dict(out=FAKE, query=FAKE, cache=FAKE, block_tables=FAKE, context_lens=FAKE, num_seqs=4,
                num_heads=16, latent_dim=512, rope_dim=64, block_size=16, max_blocks_per_seq=8,
                num_blocks=64, max_context_len=100, scale=0.1, workspace=FAKE,
                workspace_bytes=1 << 30, dtype=0, d_status=None, stream=None)
    assert set(kw) <= set(args)
    args.update(kw)
    return pa.LIB.pa_latent_decode(*args.values())


@pytest.mark.parametrize("kw,code", [
    (dict(num_seqs=0), OK),
    (dict(num_seqs=-1), INVALID), (dict(out=None), INVALID), (dict(query=None), INVALID),
    (dict(cache=None), INVALID), (dict(block_tables=None), INVALID),
    (dict(context_lens=None), INVALID), (dict(out=FAKE + 8), INVALID),
    (dict(cache=FAKE + 8), INVALID), (dict(context_lens=FAKE + 2), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(max_context_len=-1), INVALID), (dict(max_blocks_per_seq=0), INVALID),
    (dict(num_blocks=0), INVALID), (dict(num_heads=0), INVALID), (dict(d_status=FAKE + 2), INVALID),
    (dict(num_heads=129), UNSUPPORTED), (dict(latent_dim=128), UNSUPPORTED),
    (dict(rope_dim=128), UNSUPPORTED), (dict(block_size=48), UNSUPPORTED),
    (dict(dtype=4), UNSUPPORTED), (dict(num_seqs=65536), UNSUPPORTED),
])
def test_latent_decode_refusals(pa, kw, code):
    assert _decode(pa, **kw) == code


def test_latent_decode_refuses_a_short_workspace(pa):
    need = pa.pa_latent_decode_workspace_size(4, 16, 512, 16, 4096)
    if need:
        kw = dict(max_context_len=4096, max_blocks_per_seq=256)
        assert _decode(pa, workspace=None, workspace_bytes=0, **kw) == INVALID
        assert _decode(pa, workspace_bytes=need - 1, **kw) == INVALID
        assert _decode(pa, workspace=FAKE + 8, workspace_bytes=need, **kw) == INVALID


def _prefill(pa, **kw):
    args = dict(out=FAKE, query=FAKE, cache=FAKE, w_kv=FAKE, block_tables=FAKE, query_starts=FAKE,
                context_lens=FAKE, num_seqs=2, num_tokens=20, num_heads=16, latent_dim=512,
                rope_dim=64, nope_dim=128, value_dim=128, block_size=16, max_blocks_per_seq=8,
                num_blocks=64, max_query_len=20, max_context_len=100, scale=0.1, workspace=FAKE,
                workspace_bytes=1 << 30, dtype=0, d_status=None, stream=None)
    assert set(kw) <= set(args)
    args.update(kw)
    return pa.LIB.pa_latent_prefill(*args.values())


@pytest.mark.parametrize("kw,code", [
    (dict(num_seqs=0), OK), (dict(num_tokens=0), OK), (dict(max_query_len=0), OK),
    (dict(num_seqs=-1), INVALID), (dict(num_tokens=-1), INVALID), (dict(out=None), INVALID),
    (dict(w_kv=None), INVALID), (dict(query_starts=None), INVALID), (dict(w_kv=FAKE + 8), INVALID),
    (dict(query_starts=FAKE + 2), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(max_query_len=-1), INVALID), (dict(max_context_len=-1), INVALID),
    (dict(workspace=None, workspace_bytes=0), INVALID), (dict(workspace_bytes=1000), INVALID),
    (dict(workspace=FAKE + 8), INVALID), (dict(num_blocks=0), INVALID),
    (dict(nope_dim=64), UNSUPPORTED), (dict(value_dim=64), UNSUPPORTED),
    (dict(latent_dim=1024), UNSUPPORTED), (dict(num_heads=200), UNSUPPORTED),
    (dict(block_size=4), UNSUPPORTED), (dict(dtype=3), UNSUPPORTED),
])
def test_latent_prefill_refusals(pa, kw, code):
    assert _prefill(pa, **kw) == code


def test_workspace_sizes(pa):
    ws = pa.pa_latent_prefill_workspace_size
    # the expanded K and V of every head, at least
    for s, h, lat, ctx in ((1, 8, 512, 100), (3, 128, 256, 5000)):
        assert ws(s, h, lat, 16, ctx) >= s * h * 256 * 2 * ctx
    assert ws(1, 8, 300, 16, 100) == 0 and ws(1, 129, 512, 16, 100) == 0
    # no overflow of 32 bits on the way
    assert ws(64, 128, 512, 64, 131072) > 1 << 38
    assert pa.pa_latent_decode_workspace_size(4, 200, 512, 16, 100) == 0
    assert pa.pa_latent_decode_workspace_size(-1, 16, 512, 16, 100) == 0


def test_binding_checks_what_the_library_cannot_see(pa):
    """Wrong element types, shapes and strides, tensors that are not on a
    CUDA device: refused before the library is called."""
    t = torch.zeros
    h = torch.float16
    good = dict(query_out=t(4, 8, 128, dtype=h), query=t(4, 8, 128, dtype=h),
                key=t(4, 2, 128, dtype=h), value=t(4, 2, 128, dtype=h),
                k_cache=t(3, 16, 2, 128, dtype=h), v_cache=t(3, 16, 2, 128, dtype=h),
                slot_mapping=t(4, dtype=torch.int64), positions=t(4, dtype=torch.int64),
                cos_sin=t(10, 128))
    bad = dict(query=t(4, 8, 128), key=t(4, 2, 64, dtype=h), value=t(3, 2, 128, dtype=h),
               v_cache=t(3, 16, 2, 128), slot_mapping=t(4, dtype=torch.int32),
               positions=t(4, 2, dtype=torch.int64)[:, 0], cos_sin=t(10, 128, dtype=h),
               query_out=t(4, 128, 8, dtype=h).transpose(1, 2), k_cache=t(4, 16, 2, 128, dtype=h))
    for name, value in bad.items():
        with pytest.raises(ValueError):
            pa.pa_rope_append(**{**good, name: value})
    with pytest.raises(ValueError, match="CUDA"):
        pa.pa_rope_append(**good)
    good = dict(out=t(2, 4, 512, dtype=h), query=t(2, 4, 576, dtype=h),
                cache=t(3, 16, 576, dtype=h), block_tables=t(2, 3, dtype=torch.int32),
                context_lens=t(2, dtype=torch.int32), max_context_len=40, scale=1.0)
    bad = dict(out=t(2, 4, 512), cache=t(3, 16, 512, dtype=h), context_lens=t(2, dtype=torch.int64),
               block_tables=t(3, 3, dtype=torch.int32), query=t(2, 8, 576, dtype=h)[:, ::2])
    for name, value in bad.items():
        with pytest.raises(ValueError):
            pa.pa_latent_decode(**{**good, name: value})
    with pytest.raises(ValueError, match="CUDA"):
        pa.pa_latent_decode(**good)


def test_empty_calls_take_null_tensors(pa):
    """Tensors of no elements have no address."""
    none = dict.fromkeys(("query_out", "query", "key", "value", "slot_mapping", "positions"))
    assert _rope(pa, num_tokens=0, **none) == OK
    none = dict.fromkeys(("query_out", "query_rope", "latent", "slot_mapping", "positions"))
    assert _append(pa, num_tokens=0, **none) == OK
    none = dict.fromkeys(("out", "query", "block_tables", "context_lens", "workspace"))
    assert _decode(pa, num_seqs=0, **none) == OK
    assert _prefill(pa, num_seqs=0, **none) == OK
    assert _prefill(pa, num_tokens=0, out=None, query=None) == OK


def test_sizes_past_the_limits(pa):
    assert pa.LIB.pa_latent_decode_workspace_size(65536, 16, 512, 16, 4096) == 0
    assert pa.LIB.pa_latent_prefill_workspace_size(65536, 16, 512, 16, 4096) == 0
    assert _decode(pa, num_seqs=65536) == UNSUPPORTED
    assert _prefill(pa, num_seqs=65536) == UNSUPPORTED
