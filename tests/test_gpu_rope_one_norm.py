"""pa_rope_append with a norm for the queries or for the keys alone."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("d,hq,hkv,tokens", [(64, 5, 3, 9), (128, 32, 8, 700)])
def test_one_norm_alone(dtype, d, hq, hkv, tokens):
    """Each side is what it is with both norms, or with none."""
    from paged_kv_cache_415_b200 import binding as B
    g = torch.Generator(device="cuda").manual_seed(d)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dtype)
    q, k, v = rand(tokens, hq, d), rand(tokens, hkv, d), rand(tokens, hkv, d)
    weights = [(torch.rand(d, generator=g, device="cuda") + 0.5).to(dtype) for _ in range(2)]
    slots = torch.randperm(tokens, generator=g, device="cuda")
    pos = torch.arange(tokens, device="cuda") % 50
    table = torch.rand(50, d, generator=g, device="cuda")

    def take(qw, kw):
        pools = [torch.zeros(-(-tokens // 16), 16, hkv, d, dtype=dtype, device="cuda")
                 for _ in range(2)]
        out = torch.empty_like(q)
        B.pa_rope_append(out, q, k, v, *pools, slots, pos, table, q_weight=qw, k_weight=kw)
        return out, *pools

    both, none = take(*weights), take(None, None)
    assert not torch.equal(both[0], none[0]) and not torch.equal(both[1], none[1])
    got = take(weights[0], None)
    assert torch.equal(got[0], both[0]) and torch.equal(got[1], none[1])
    got = take(None, weights[1])
    assert torch.equal(got[0], none[0]) and torch.equal(got[1], both[1])
    assert torch.equal(got[2], none[2])
