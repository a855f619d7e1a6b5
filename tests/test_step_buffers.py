"""The buffers that a decode step owns, on the CPU: the library's calls are
replaced by recorders, as nothing is launched here."""
import pytest
import torch

H, D, BLOCK = 4, 64, 16


@pytest.fixture
def calls(monkeypatch):
    from paged_kv_cache_415_b200 import build
    build.build()
    from paged_kv_cache_415_b200 import binding as B
    seen = []
    monkeypatch.setattr(B, "pa_rope_append", lambda *a: seen.append(("append", a)))
    monkeypatch.setattr(B, "pa_paged_decode", lambda *a: seen.append(("decode", a)))
    return seen


def _step(num_seqs):
    from paged_kv_cache_415_b200.step import DecodeStep
    pools = [torch.zeros(8, BLOCK, 2, D, dtype=torch.float16) for _ in range(2)]
    return DecodeStep(*pools, num_seqs, H, 64)


def _take(step, seqs, dtype=torch.float16):
    from paged_kv_cache_415_b200.step import Rotation
    long = torch.zeros(seqs, dtype=torch.int64)
    return step(torch.zeros(seqs, H, D, dtype=dtype), None, None, 1.0,
                new_key=torch.zeros(seqs, 2, D, dtype=dtype),
                new_value=torch.zeros(seqs, 2, D, dtype=dtype), slot_mapping=long, positions=long,
                rotation=Rotation(torch.zeros(4, D)))


def test_rotated_queries_keep_their_place(calls):
    """Steps of several batch sizes and both types rotate into one buffer that
    lives as long as the step: a graph captured at one size replays into it."""
    step = _step(5)
    for seqs, dtype in ((3, torch.float16), (5, torch.float16), (1, torch.bfloat16),
                        (3, torch.float16)):
        _take(step, seqs, dtype)
    rotated = [a[0] for kind, a in calls if kind == "append"]
    assert [tuple(t.shape) for t in rotated] == [(s, H, D) for s in (3, 5, 1, 3)]
    assert len({t.untyped_storage().data_ptr() for t in rotated}) == 1
    assert len({t.data_ptr() for t in rotated}) == 1
    # the decode reads what the append wrote
    assert [a[1].data_ptr() for kind, a in calls if kind == "decode"] \
        == [t.data_ptr() for t in rotated]


def test_rotating_more_than_the_step_is_made_for_is_refused(calls):
    step = _step(2)
    with pytest.raises(ValueError, match="at most 2 sequences"):
        _take(step, 3)
    with pytest.raises(ValueError, match="16-bit"):
        _take(step, 1, torch.float32)
    assert not calls
