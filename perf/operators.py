"""The operators around a rotated and a latent key-value cache, as they are measured.

Four operators, each with its plain form (elementary torch operations in 32 bits) and with the
library's own call:

  rope_append     queries and keys normalised for each head and rotated by position, keys and
                  values written to their slots of the paged pools
  latent_append   the shared latent vector of each token normalised, its key part rotated, both
                  written to their slot of the paged latent pool; the queries' rotated part
  latent_decode   one query a sequence over the latent pool, with the projections absorbed into
                  the query and the output
  latent_prefill  the new tokens of each prompt over the latent pool, with keys and values of each
                  head expanded from the latent vectors

``own`` chooses the form that ``run`` takes; ``exact`` gives the same outputs in 64 bits.
"""
import math
import random

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
_NOPE = 128          # features of a head's expanded key that carry no position
_VALUE = 128         # features of a head's expanded value


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one decode step of a batch with grouped heads: a token a sequence, latency counts
        dict(name="rope decode step", op="rope_append", type="bf16", pool="bf16", tokens=64,
             q_heads=32, kv_heads=8, dim=128, rot=128, block=16, norm=True, pairs=False),
        # a long prompt's chunk with a key head for each query head, no norms
        dict(name="rope prompt", op="rope_append", type="fp16", pool="fp16", tokens=8192,
             q_heads=32, kv_heads=32, dim=128, rot=128, block=16, norm=False, pairs=False),
        # a ragged prompt into 8-bit pools: small heads, half of each head rotated, adjacent pairs
        dict(name="rope prompt e4m3", op="rope_append", type="bf16", pool="e4m3", tokens=4099,
             q_heads=20, kv_heads=4, dim=64, rot=32, block=32, norm=True, pairs=True),
        # one decode step's append to a latent pool, all heads on one device
        dict(name="latent append step", op="latent_append", type="bf16", tokens=100, heads=128,
             latent=512, rope=64, block=16, norm=True, pairs=True),
        # a prompt's append, heads split over devices
        dict(name="latent append prompt", op="latent_append", type="fp16", tokens=8191, heads=32,
             latent=512, rope=64, block=64, norm=True, pairs=False),
        # one user with a long document: few heads, the work is split along the context
        dict(name="latent decode one long", op="latent_decode", type="bf16", seqs=1, heads=16,
             latent=512, rope=64, block=16, low=32773, top=32773),
        # a serving batch with all heads on one device: many products for each byte of the pool
        dict(name="latent decode all heads", op="latent_decode", type="bf16", seqs=64, heads=128,
             latent=512, rope=64, block=32, low=1, top=4096),
        # short ragged conversations of a smaller model, an odd number of heads
        dict(name="latent decode short ragged", op="latent_decode", type="fp16", seqs=33, heads=40,
             latent=256, rope=64, block=16, low=1, top=700),
        # a large batch with the heads split over devices: reading the pool is all there is
        dict(name="latent decode large batch", op="latent_decode", type="bf16", seqs=256, heads=16,
             latent=512, rope=64, block=64, low=3500, top=4500),
        # one whole prompt
        dict(name="latent prefill prompt", op="latent_prefill", type="bf16", seqs=1, heads=32,
             latent=512, rope=64, block=16, new_low=4096, new_top=4096, old_low=0, old_top=0),
        # chunks of several prompts behind cached prefixes
        dict(name="latent prefill chunks", op="latent_prefill", type="fp16", seqs=7, heads=20,
             latent=512, rope=64, block=32, new_low=1, new_top=700, old_low=0, old_top=2300),
        # the last few tokens of one prompt behind its cached prefix
        dict(name="latent prefill tail", op="latent_prefill", type="bf16", seqs=1, heads=8,
             latent=256, rope=64, block=16, new_low=17, new_top=17, old_low=300, old_top=300),
    ]


def _spread(rng, low, top):
    """A whole number in [low, top], evenly over its logarithm."""
    return min(top, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(top + 1)))))))


def draw(rng):
    op = rng.choice(["rope_append", "latent_append", "latent_decode", "latent_prefill"])
    kind = rng.choice(["bf16", "fp16"])
    if op == "rope_append":
        kv = rng.choice([1, 2, 4, 8, 32])
        dim = rng.choice([64, 128])
        return dict(op=op, type=kind, pool=rng.choice([kind, kind, "e4m3"]),
                    tokens=_spread(rng, 1, 8192), q_heads=kv * rng.choice([1, 2, 4, 5, 8])
                    if kv < 32 else 32, kv_heads=kv, dim=dim, rot=rng.choice([dim, dim, dim // 2]),
                    block=rng.choice([8, 16, 32]), norm=rng.random() < 0.5,
                    pairs=rng.random() < 0.5)
    if op == "latent_append":
        return dict(op=op, type=kind, tokens=_spread(rng, 1, 8192),
                    heads=rng.choice([1, 8, 16, 20, 32, 64]), latent=rng.choice([256, 512]),
                    rope=64, block=rng.choice([8, 16, 32, 64]), norm=rng.random() < 0.8,
                    pairs=rng.random() < 0.5)
    if op == "latent_decode":
        seqs = _spread(rng, 1, 256)
        top = _spread(rng, 1, min(65536, 1 << 20 if seqs < 8 else (1 << 20) // seqs))
        return dict(op=op, type=kind, seqs=seqs,
                    heads=rng.choice([1, 8, 16, 20, 32, 40, 64, 96, 128]) if seqs * top < 200000
                    else rng.choice([8, 16, 32]), latent=rng.choice([256, 512]), rope=64,
                    block=rng.choice([8, 16, 32, 64]), low=rng.randint(1, top), top=top)
    seqs = _spread(rng, 1, 12)
    new = _spread(rng, 1, 2048 // seqs)
    old = rng.choice([0, _spread(rng, 1, 4096 // seqs)])
    return dict(op=op, type=kind, seqs=seqs, heads=rng.choice([1, 8, 20, 32]),
                latent=rng.choice([256, 512]), rope=64, block=rng.choice([8, 16, 32, 64]),
                new_low=rng.randint(1, new), new_top=new, old_low=rng.randint(0, old), old_top=old)


def _lengths(count, low, top, salt):
    """The ragged lengths of a case: they belong to the case, not to the seed."""
    rng = random.Random(count * 1000003 + low * 101 + top * 7 + salt)
    got = [rng.randint(low, top) for _ in range(count)]
    got[rng.randrange(count)] = top
    return got


def _case_lengths(case):
    """(new tokens, context with them) of each sequence of an attention case."""
    if case["op"] == "latent_decode":
        context = _lengths(case["seqs"], case["low"], case["top"], 1)
        return [1] * case["seqs"], context
    new = _lengths(case["seqs"], case["new_low"], case["new_top"], 2)
    old = _lengths(case["seqs"], case["old_low"], case["old_top"], 3)
    return new, [a + b for a, b in zip(new, old)]


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

class _Maker:
    def __init__(self, seed):
        self.dev = torch.device("cuda")
        self.gen = torch.Generator(device=self.dev)
        self.gen.manual_seed(seed * 2654435761 % (1 << 62))

    def normal(self, *shape, kind, scale=1.0):
        x = torch.randn(*shape, generator=self.gen, device=self.dev, dtype=torch.float32)
        return (x * scale).to(kind)

    def order(self, n):
        return torch.randperm(n, generator=self.gen, device=self.dev)

    def below(self, top, *shape):
        return torch.randint(0, top, shape, generator=self.gen, device=self.dev)


def _angles(positions, rot):
    """float32 [positions][rot]: the cosines of the rot / 2 angles of each position, then the
    sines; the angles themselves in 64 bits."""
    half = rot // 2
    dev = torch.device("cuda")
    rate = 10000.0 ** (-torch.arange(half, device=dev, dtype=torch.float64) / half)
    at = torch.arange(positions, device=dev, dtype=torch.float64)[:, None] * rate
    return torch.cat([at.cos(), at.sin()], 1).float()


_POSITIONS = 16384       # positions of the angle table that the append cases rotate by


def prepare(case, seed):
    op, kind = case["op"], _TYPES[case["type"]]
    m = _Maker(seed)
    if op == "rope_append":
        t, hq, hkv, d, b = (case[k] for k in ("tokens", "q_heads", "kv_heads", "dim", "block"))
        blocks = -(-t // b) + 5
        # queries, keys and values side by side, as one projection leaves them
        rows = m.normal(t, (hq + 2 * hkv) * d, kind=kind, scale=2.0)
        q = rows[:, :hq * d].unflatten(1, (hq, d))
        k = rows[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
        v = rows[:, (hq + hkv) * d:].unflatten(1, (hkv, d))
        pools = [m.normal(blocks, b, hkv, d, kind=kind) for _ in range(2)]
        if case["pool"] == "e4m3":
            pools = [p.to(torch.float8_e4m3fn) for p in pools]
        return dict(case=case, query=q, key=k, value=v, k_cache=pools[0], v_cache=pools[1],
                    query_out=torch.zeros(t, hq, d, device=m.dev, dtype=kind),
                    slots=m.order(blocks * b)[:t].contiguous(), positions=m.below(_POSITIONS, t),
                    cos_sin=_angles(_POSITIONS, case["rot"]),
                    q_weight=m.normal(d, kind=kind, scale=0.2) + 1 if case["norm"] else None,
                    k_weight=m.normal(d, kind=kind, scale=0.2) + 1 if case["norm"] else None)
    if op == "latent_append":
        t, h, lat, r, b = (case[k] for k in ("tokens", "heads", "latent", "rope", "block"))
        blocks = -(-t // b) + 5
        q = m.normal(t, h, _NOPE + r, kind=kind, scale=2.0)       # the queries' projection
        return dict(case=case, query_rope=q[..., _NOPE:],
                    query=torch.zeros(t, h, lat + r, device=m.dev, dtype=kind),
                    rows=m.normal(t, lat + r, kind=kind, scale=2.0),
                    cache=m.normal(blocks, b, lat + r, kind=kind),
                    slots=m.order(blocks * b)[:t].contiguous(), positions=m.below(_POSITIONS, t),
                    cos_sin=_angles(_POSITIONS, r),
                    weight=m.normal(lat, kind=kind, scale=0.2) + 1 if case["norm"] else None)
    new, context = _case_lengths(case)
    s, h, lat, r, b = (case[k] for k in ("seqs", "heads", "latent", "rope", "block"))
    need = [-(-c // b) for c in context]
    width = max(need)
    blocks = sum(need) + 3
    order = m.order(blocks).to(torch.int32)
    tables = torch.full((s, width), -1, device=m.dev, dtype=torch.int32)
    at = 0
    for i, n in enumerate(need):
        tables[i, :n] = order[at:at + n]
        at += n
    state = dict(case=case, cache=m.normal(blocks, b, lat + r, kind=kind), tables=tables,
                 context=torch.tensor(context, device=m.dev, dtype=torch.int32),
                 max_context=max(context))
    if op == "latent_decode":
        # the scores' standard deviation is about 1 for such queries
        state |= dict(query=m.normal(s, h, lat + r, kind=kind), scale=(lat + r) ** -0.5,
                      out=torch.zeros(s, h, lat, device=m.dev, dtype=kind))
        return state
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    # positions of the padded form: row i of sequence s is token rows[s][i] of the batch
    state |= dict(query=m.normal(starts[-1], h, _NOPE + r, kind=kind),
                  w_kv=m.normal(h, _NOPE + _VALUE, lat, kind=kind, scale=lat ** -0.5),
                  starts=torch.tensor(starts, device=m.dev, dtype=torch.int32),
                  max_new=max(new), scale=(_NOPE + r) ** -0.5,
                  out=torch.zeros(starts[-1], h, _VALUE, device=m.dev, dtype=kind))
    return state


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------

def _normed(x, weight):
    x = x.float()
    if weight is None:
        return x
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * weight.float()


def _turned(x, cos_sin, positions, pairs):
    """x [T][H][D] with its first R features rotated by the angles of each token's position."""
    rot = cos_sin.shape[1]
    angle = cos_sin[positions][:, None, :]
    c, s = angle[..., :rot // 2], angle[..., rot // 2:]
    a, rest = x[..., :rot], x[..., rot:]
    if pairs:
        lo, hi = a[..., 0::2], a[..., 1::2]
        turned = torch.stack([lo * c - hi * s, hi * c + lo * s], -1).flatten(-2)
    else:
        lo, hi = a[..., :rot // 2], a[..., rot // 2:]
        turned = torch.cat([lo * c - hi * s, hi * c + lo * s], -1)
    return torch.cat([turned, rest], -1)


def _plain_rope(st):
    case = st["case"]
    q = _turned(_normed(st["query"], st["q_weight"]), st["cos_sin"], st["positions"], case["pairs"])
    k = _turned(_normed(st["key"], st["k_weight"]), st["cos_sin"], st["positions"], case["pairs"])
    v = st["value"]
    pool = st["k_cache"].dtype
    if case["pool"] == "e4m3":
        top = torch.finfo(pool).max
        k, v = k.clamp(-top, top), v.float().clamp(-top, top)
    # index by bytes: an 8-bit float pool is written as its codes
    view = torch.uint8 if case["pool"] == "e4m3" else pool
    st["query_out"].copy_(q)
    st["k_cache"].view(view).flatten(0, 1)[st["slots"]] = k.to(pool).view(view)
    st["v_cache"].view(view).flatten(0, 1)[st["slots"]] = v.to(pool).view(view)
    return st["query_out"], st["k_cache"], st["v_cache"]


def _plain_latent_append(st):
    case = st["case"]
    lat = case["latent"]
    c = _normed(st["rows"][:, :lat], st["weight"])
    k = _turned(st["rows"][:, None, lat:].float(), st["cos_sin"], st["positions"], case["pairs"])
    q = _turned(st["query_rope"].float(), st["cos_sin"], st["positions"], case["pairs"])
    st["query"][..., lat:] = q.to(st["query"].dtype)
    st["cache"].flatten(0, 1)[st["slots"]] = torch.cat([c, k[:, 0]], 1).to(st["cache"].dtype)
    return st["query"][..., lat:], st["cache"]


def _context_rows(st):
    """float32 [S][tokens][width]: each sequence's cached rows, in order; and which of them count."""
    cache, tables = st["cache"], st["tables"].long()
    at = torch.arange(st["max_context"], device=cache.device)
    slot = tables[:, at // cache.shape[1]] * cache.shape[1] + at % cache.shape[1]
    counts = at[None, :] < st["context"][:, None]
    return cache.flatten(0, 1)[torch.where(counts, slot, 0)].float(), counts


def _weights(score, seen):
    """Softmax over the last axis among the places that `seen` allows."""
    score = score.masked_fill(~seen, -math.inf)
    p = torch.exp(score - score.amax(-1, keepdim=True))
    return p / p.sum(-1, keepdim=True)


def _plain_latent_decode(st):
    rows, counts = _context_rows(st)
    score = torch.matmul(st["query"].float(), rows.transpose(1, 2)) * st["scale"]
    p = _weights(score, counts[:, None, :])
    st["out"].copy_(torch.matmul(p, rows[..., :st["case"]["latent"]]))
    return st["out"]


def _plain_latent_prefill(st):
    rows, counts = _context_rows(st)
    lat = st["case"]["latent"]
    starts, context = st["starts"].long(), st["context"].long()
    new = starts[1:] - starts[:-1]
    kv = torch.einsum("stl,hel->shte", rows[..., :lat], st["w_kv"].float())
    key = torch.cat([kv[..., :_NOPE], rows[:, None, :, lat:].expand(-1, kv.shape[1], -1, -1)], -1)
    i = torch.arange(st["max_new"], device=rows.device)
    token = (starts[:-1, None] + i).clamp(max=st["query"].shape[0] - 1)
    q = st["query"].float()[token].transpose(1, 2)                       # [S][H][new][D]
    score = torch.matmul(q, key.transpose(2, 3)) * st["scale"]
    at = (context - new)[:, None] + i                                    # positions of the queries
    # rows of the padding attend to token 0 alone: they are not taken below
    at = torch.where(i < new[:, None], at, 0)
    seen = torch.arange(rows.shape[1], device=rows.device)[None, None, :] <= at[:, :, None]
    out = torch.matmul(_weights(score, seen[:, None]), kv[..., _NOPE:])
    # the place of each token of the batch in the padded form
    t = torch.arange(st["query"].shape[0], device=rows.device)
    s = torch.searchsorted(starts[1:].contiguous(), t, right=True)
    st["out"].copy_(out[s, :, t - starts[s]])
    return st["out"]


def _own(st):
    from paged_kv_cache_415_b200 import binding as B
    case = st["case"]
    op = case["op"]
    if op == "rope_append":
        B.pa_rope_append(st["query_out"], st["query"], st["key"], st["value"], st["k_cache"],
                         st["v_cache"], st["slots"], st["positions"], st["cos_sin"],
                         q_weight=st["q_weight"], k_weight=st["k_weight"], eps=1e-6,
                         interleaved=case["pairs"])
        return st["query_out"], st["k_cache"], st["v_cache"]
    if op == "latent_append":
        tail = st["query"][..., case["latent"]:]
        B.pa_latent_append(tail, st["query_rope"], st["rows"], st["cache"], st["slots"],
                           st["positions"], st["cos_sin"], weight=st["weight"], eps=1e-6,
                           interleaved=case["pairs"])
        return tail, st["cache"]
    if op == "latent_decode":
        if "workspace" not in st:                    # kept from step to step, as DecodeStep does
            n = B.pa_latent_decode_workspace_size(case["seqs"], case["heads"], case["latent"],
                                                  case["block"], st["max_context"])
            st["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
        B.pa_latent_decode(st["out"], st["query"], st["cache"], st["tables"], st["context"],
                           st["max_context"], st["scale"], workspace=st["workspace"])
        return st["out"]
    if "workspace" not in st:
        n = B.pa_latent_prefill_workspace_size(case["seqs"], case["heads"], case["latent"],
                                               case["block"], st["max_context"])
        st["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    B.pa_latent_prefill(st["out"], st["query"], st["cache"], st["w_kv"], st["tables"],
                        st["starts"], st["context"], st["max_new"], st["max_context"],
                        st["scale"], st["workspace"])
    return st["out"]


_PLAIN = {"rope_append": _plain_rope, "latent_append": _plain_latent_append,
          "latent_decode": _plain_latent_decode, "latent_prefill": _plain_latent_prefill}


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# Work
# ---------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "rope_append":
        t, hq, hkv, d = (case[k] for k in ("tokens", "q_heads", "kv_heads", "dim"))
        stored = 1 if case["pool"] == "e4m3" else 2
        per = 2 * hq * d * 2 + 2 * hkv * d * (2 + stored) + case["rot"] * 4 + 16
        return {"bytes": t * per, "flops": t * (hq + hkv) * d * (4 if case["norm"] else 0)
                + t * (hq + hkv) * case["rot"] * 3}
    if op == "latent_append":
        t, h, w, r = case["tokens"], case["heads"], case["latent"] + case["rope"], case["rope"]
        return {"bytes": t * (2 * h * r * 2 + 2 * w * 2 + r * 4 + 16),
                "flops": t * (case["latent"] * (4 if case["norm"] else 0) + (h + 1) * r * 3)}
    new, context = _case_lengths(case)
    h, lat, w = case["heads"], case["latent"], case["latent"] + case["rope"]
    blocks = sum(-(-c // case["block"]) for c in context)
    if op == "latent_decode":
        return {"bytes": sum(context) * w * 2 + case["seqs"] * h * (w + lat) * 2 + blocks * 4,
                "flops": sum(context) * h * 2 * (w + lat)}
    seen = sum(n * (c - n) + n * (n + 1) // 2 for n, c in zip(new, context))
    d = _NOPE + case["rope"]
    return {"bytes": sum(context) * w * 2 + sum(new) * h * (d + _VALUE) * 2
            + h * (_NOPE + _VALUE) * lat * 2 + blocks * 4,
            "flops": sum(context) * h * 2 * lat * (_NOPE + _VALUE) + seen * h * 2 * (d + _VALUE)}


# ---------------------------------------------------------------------------
# The definitions in 64 bits, a head or a sequence at a time
# ---------------------------------------------------------------------------

def _rotation(cos_sin, positions, pairs, width):
    """float64 [T][width][width]: the rotation of each token as a matrix."""
    t, rot = positions.shape[0], cos_sin.shape[1]
    half = rot // 2
    full = torch.eye(width, dtype=torch.float64, device="cuda").repeat(t, 1, 1)
    for j in range(half):
        a, b = (2 * j, 2 * j + 1) if pairs else (j, j + half)
        c, s = cos_sin[positions, j].double(), cos_sin[positions, half + j].double()
        full[:, a, a], full[:, a, b], full[:, b, a], full[:, b, b] = c, -s, s, c
    return full


def _unit(x, weight):
    x = x.double()
    if weight is None:
        return x
    n = x.shape[-1]
    return x * weight.double() / torch.sqrt(torch.linalg.vecdot(x, x)[..., None] / n + 1e-6)


def _rotated(x, st, pairs):
    """float64: x [T][H][D] times the rotation matrix of each token, some tokens at a time."""
    got = torch.empty(x.shape, dtype=torch.float64, device="cuda")
    for i in range(0, x.shape[0], 1024):
        turn = _rotation(st["cos_sin"], st["positions"][i:i + 1024], pairs, x.shape[-1])
        got[i:i + 1024] = torch.einsum("tij,thj->thi", turn, x[i:i + 1024])
    return got


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "rope_append":
        q = _rotated(_unit(st["query"], st["q_weight"]), st, case["pairs"])
        k = _rotated(_unit(st["key"], st["k_weight"]), st, case["pairs"])
        kc, vc = st["k_cache"].double(), st["v_cache"].double()
        kc.view(-1, *kc.shape[2:]).index_copy_(0, st["slots"], k)
        vc.view(-1, *vc.shape[2:]).index_copy_(0, st["slots"], st["value"].double())
        return q, kc, vc
    if op == "latent_append":
        lat = case["latent"]
        q = _rotated(st["query_rope"].double(), st, case["pairs"])
        k = _rotated(st["rows"][:, None, lat:].double(), st, case["pairs"])[:, 0]
        pool = st["cache"].double()
        flat = pool.view(-1, pool.shape[-1])
        flat[:, :lat].index_copy_(0, st["slots"], _unit(st["rows"][:, :lat], st["weight"]))
        flat[:, lat:].index_copy_(0, st["slots"], k)
        return q, pool
    new, context = _case_lengths(case)
    if op == "latent_prefill" and work(case)["flops"] > 2e12:
        return None
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for i, (n, c) in enumerate(zip(new, context)):
        pages = st["tables"][i, :-(-c // case["block"])].long()
        rows = st["cache"][pages].flatten(0, 1)[:c].double()
        if op == "latent_decode":
            p = torch.softmax(st["query"][i].double() @ rows.T * st["scale"], -1)
            out[i] = p @ rows[:, :case["latent"]]
            continue
        later = torch.ones(n, c, dtype=torch.bool, device="cuda").triu(c - n + 1)
        for h in range(case["heads"]):
            w = st["w_kv"][h].double()
            key = torch.cat([rows[:, :case["latent"]] @ w[:_NOPE].T, rows[:, case["latent"]:]], 1)
            score = st["query"][at:at + n, h].double() @ key.T * st["scale"]
            p = torch.softmax(score.masked_fill(later, -math.inf), -1)
            out[at:at + n, h] = p @ (rows[:, :case["latent"]] @ w[_NOPE:].T)
        at += n
    return out
