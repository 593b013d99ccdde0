"""Cases of rotary positions and of latent attention: what a serving step of a
model whose layers keep one latent vector a token runs before it calls the FFN,
and the rotation that grouped-query layers need beside their cache.

  rotate         q and k rows turned by their positions (moe_rope_apply)
  rotate_append  the same, with k and v into the paged cache (moe_rope_append)
  latent_append  the latent row and its turned key part into the paged latent
                 cache, q's part turned beside it (moe_latent_append)
  latent_prompt  expanded form: causal attention over packed prompts, keys of
                 128 elements a head and 64 that the heads share (moe_latent_prompt)
  latent_tree    absorbed form: attention of single tokens or drafted trees over
                 the paged latent cache (moe_latent_tree)

``run`` computes a case in plain torch operations, or with ``own`` set
through the library's entry points.  The requests' lengths follow from the case
(falling by a constant factor from the given longest one); a seed orders them and
makes everything else."""
import math

import torch

own = False
DEV = "cuda:0"
TREE = 64                                  # tokens of a drafted tree at most: the bits of a mask word
LATENT, ROPE, NOPE, VALUE = 512, 64, 128, 128
SCALE = (NOPE + ROPE) ** -0.5
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # One decoded token of a grouped-query layer: latency counts.
        dict(name="rotate, 1 row", op="rotate", dtype="bf16", rows=1, q_heads=32, kv_heads=8, head_dim=128, dims=128, interleaved=False,
             scaling="plain", theta=10000.0, far=1000),
        # The rows of a long prompt's part at far positions: half of each head turns, interleaved pairs, a stretched context.
        dict(name="rotate, 8192 rows", op="rotate", dtype="f16", rows=8192, q_heads=24, kv_heads=4, head_dim=128, dims=64,
             interleaved=True, scaling="yarn", theta=50000.0, far=1000000),
        # The verify step of 7 streams with 8 drafted rows each, out of a fused projection.
        dict(name="rotate + append, 56 rows", op="rotate_append", dtype="bf16", rows=56, q_heads=32, kv_heads=8, head_dim=128, dims=128,
             interleaved=False, scaling="bands", theta=500000.0, far=4000, page=16),
        # A large batch of prompts; every 29th row belongs to no request (the padding of a fixed-size step).
        dict(name="rotate + append, 16384 rows", op="rotate_append", dtype="bf16", rows=16384, q_heads=16, kv_heads=8, head_dim=128,
             dims=128, interleaved=False, scaling="linear", theta=10000.0, far=30000, page=64),
        # One decoded token of each of 7 streams.
        dict(name="latent append, 7 rows", op="latent_append", dtype="bf16", rows=7, heads=16, interleaved=True, scaling="yarn",
             theta=50000.0, far=100000, page=16),
        # A large batch of prompts, with the padding of a fixed-size step.
        dict(name="latent append, 16384 rows", op="latent_append", dtype="bf16", rows=16384, heads=64, interleaved=True, scaling="yarn",
             theta=50000.0, far=30000, page=64),
        # One prompt of 512 tokens, the length of the layer's prefill workload.
        dict(name="latent prompt, 512", op="latent_prompt", dtype="bf16", requests=1, longest=512, ragged=False, heads=16),
        # A batch of short and middling prompts with odd lengths, odd heads.
        dict(name="latent prompt, 17 ragged", op="latent_prompt", dtype="f16", requests=17, longest=1501, ragged=True, heads=7),
        # One long document.
        dict(name="latent prompt, 8192", op="latent_prompt", dtype="bf16", requests=1, longest=8192, ragged=False, heads=32),
        # One stream, one token, a short context: the smallest decode.
        dict(name="latent tree, 1 token at 1000", op="latent_tree", dtype="bf16", requests=1, cached=1000, fresh=1, tree=False, heads=16,
             page=16),
        # The verify step: trees of up to 8 in 8 streams of up to a few thousand tokens.
        dict(name="latent tree, 8 x 8 at 4000", op="latent_tree", dtype="bf16", requests=8, cached=4000, fresh=8, tree=True, heads=64,
             page=64),
        # Decode of 16 streams of up to 100 thousand tokens.
        dict(name="latent tree, 16 tokens at 100000", op="latent_tree", dtype="bf16", requests=16, cached=100000, fresh=1, tree=False,
             heads=64, page=32),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def _turn(rng):
    return dict(interleaved=rng.random() < 0.5, scaling=rng.choice(["plain", "linear", "base", "yarn", "bands"]),
                theta=rng.choice([10000.0, 50000.0, 500000.0, 1000000.0]), far=_log(rng, 1, 1000000))


def _drawn(rng):
    op = rng.choice(["rotate", "rotate_append", "latent_append", "latent_prompt", "latent_prompt", "latent_tree", "latent_tree", "latent_tree"])
    case = dict(op=op, dtype=rng.choice(["bf16", "f16"]))
    if op.startswith("rotate"):
        kv, d = rng.choice([1, 2, 3, 4, 8]), rng.choice([64, 128])
        case.update(rows=_log(rng, 1, 16384), kv_heads=kv, q_heads=kv * rng.choice([1, 2, 3, 4, 5, 8]), head_dim=d,
                    dims=rng.choice([d, d, d // 2, d // 4]), **_turn(rng))
        if op == "rotate_append":
            case["page"] = rng.choice([16, 32, 64, 128])
        return case
    case["heads"] = rng.choice([1, 2, 3, 5, 8, 12, 16, 20, 32, 40, 64, 96, 128])
    if op == "latent_append":
        case.update(rows=_log(rng, 1, 16384), page=rng.choice([16, 32, 64, 128]), **_turn(rng))
    elif op == "latent_prompt":
        case.update(requests=_log(rng, 1, 64), longest=_log(rng, 1, 8192), ragged=rng.random() < 0.7)
    else:
        case.update(requests=_log(rng, 1, 64), cached=_log(rng, 1, 100000), fresh=rng.choice([1, _log(rng, 2, TREE)]), tree=rng.random() < 0.7,
                    page=rng.choice([16, 32, 64, 128]))
    return case


def _fits(case):
    """No dearer than the largest listed case of its operator, in the plain form either."""
    op = case["op"]
    if op.startswith("rotate"):
        return case["rows"] * (case["q_heads"] + 2 * case["kv_heads"]) * case["head_dim"] <= 16384 * 32 * 128
    if op == "latent_append":
        return case["rows"] * (576 + case["heads"] * ROPE) <= 16384 * (576 + 64 * ROPE)
    if op == "latent_prompt":
        n, L, h = case["requests"], case["longest"], case["heads"]
        return n * h * L * L <= 32 * 8192 ** 2 and n * L * h <= 32 * 8192
    n = case["requests"] * (case["cached"] + case["fresh"])
    return n <= 16 * 100001 and n * case["heads"] * case["fresh"] <= 16 * 100001 * 64


def draw(rng):
    while True:
        case = _drawn(rng)
        if _fits(case):
            return case


def _falling(n, longest, span):
    """n lengths from `longest` down to a span-th of it (one at least)."""
    return [max(1, int(longest * span ** (-i / max(1, n - 1)))) for i in range(n)]


def _fresh(case):
    return _falling(case["requests"], case["fresh"], 4.0)


def _cached(case):
    return _falling(case["requests"], case["cached"], 8.0)


def _prompts(case):
    return _falling(case["requests"], case["longest"], 24.0 if case["ragged"] else 1.0)


def _ceil(a, b):
    return -(-a // b)


def work(case):
    """Each input once, each output once; products of visible (query, key) pairs."""
    op = case["op"]
    if op.startswith("rotate"):
        n, d, q, kv = case["rows"], case["head_dim"], case["q_heads"], case["kv_heads"]
        live = n - (n // 29 if op == "rotate_append" else 0)
        turned = live * (q + kv)
        return {"bytes": 4 * n + 4 * d * (turned + (live * kv if op == "rotate_append" else 0)) + (4 * n if op == "rotate_append" else 0),
                "flops": 3 * turned * case["dims"]}
    if op == "latent_append":
        live = case["rows"] - case["rows"] // 29
        return {"bytes": 8 * case["rows"] + live * 4 * (LATENT + ROPE + case["heads"] * ROPE), "flops": 3 * live * ROPE * (1 + case["heads"])}
    h = case["heads"]
    if op == "latent_prompt":
        n = _prompts(case)
        return {"bytes": sum(n) * (2 * h * (NOPE + ROPE + NOPE + 2 * VALUE) + 2 * ROPE + 4 * h),
                "flops": sum((NOPE + ROPE + VALUE) * h * a * (a + 1) for a in n)}
    f, c = _fresh(case), _cached(case)
    rows, context = sum(f), sum(f) + sum(c)
    pages = sum(_ceil(a + b, case["page"]) for a, b in zip(f, c))
    return {"bytes": context * 2 * (LATENT + ROPE) + rows * h * (2 * (LATENT + ROPE) + 2 * LATENT + 4) + 4 * pages + (8 * rows if case["tree"] else 0),
            "flops": sum(2 * (2 * LATENT + ROPE) * h * a * (b + (a + 1) / 2) for a, b in zip(f, c))}


# ---------------------------------------------------------------- the inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(shape, dtype, g):
    return torch.randn(shape, generator=g, device=DEV, dtype=dtype)


def _shuffled(values, g):
    return torch.tensor(values, dtype=torch.int32, device=DEV)[torch.randperm(len(values), generator=g, device=DEV)]


def _offsets(fresh):
    cu = torch.zeros(fresh.numel() + 1, dtype=torch.int32, device=DEV)
    cu[1:] = torch.cumsum(fresh, 0)
    return cu


def _stretch(case):
    """The parameters of a case's scaling, as a model's configuration gives them."""
    return {"plain": {}, "linear": dict(factor=4.0), "base": dict(factor=8.0),
            "yarn": dict(factor=32.0, original=4096, low=1.0, high=32.0, attn_factor=0.1 * math.log(32.0) + 1.0),
            "bands": dict(factor=8.0, original=8192, low=1.0, high=4.0)}[case["scaling"]]


def _frequencies(case):
    """Radians a position, of each pair (64 bits); what the program keeps beside its weights."""
    n, theta, s = case.get("dims", ROPE), case["theta"], _stretch(case)
    i = torch.arange(n // 2, dtype=torch.float64, device=DEV)
    if case["scaling"] == "base":
        theta = theta * s["factor"] ** (n / (n - 2))
    f = theta ** (-2 * i / n)
    if case["scaling"] == "linear":
        return f / s["factor"]
    if case["scaling"] == "yarn":              # whole turns over the original context choose between the two
        at = [n * math.log(s["original"] / (turns * 2 * math.pi)) / (2 * math.log(theta)) for turns in (s["high"], s["low"])]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), n - 1)
        ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        return f / s["factor"] * ramp + f * (1 - ramp)
    if case["scaling"] == "bands":
        smooth = ((s["original"] * f / (2 * math.pi) - s["low"]) / (s["high"] - s["low"])).clamp(0, 1)
        return f * (smooth + (1 - smooth) / s["factor"])
    return f


def _rope(case):
    from quantized_moe_expert_router_gb300 import moe
    kind = {"plain": moe.ROPE_PLAIN, "linear": moe.ROPE_LINEAR, "base": moe.ROPE_BASE, "yarn": moe.ROPE_YARN, "bands": moe.ROPE_BANDS}
    return moe.Rope(case.get("dims", ROPE), theta=case["theta"], layout=moe.ROPE_INTERLEAVED if case["interleaved"] else moe.ROPE_HALF,
                    scaling=kind[case["scaling"]], dtype=TYPES[case["dtype"]], **_stretch(case))


def _latent(case, pool, width):
    from quantized_moe_expert_router_gb300 import moe
    return moe.LatentAttention(case["heads"], case.get("page", 16), pool, width, TYPES[case["dtype"]], softmax_scale=SCALE)


def _slots(case, s, g):
    """Slots of a shuffled pool for the rows; every 29th row belongs to no request (no slot, no position)."""
    rows, page = case["rows"], case["page"]
    pool = _ceil(rows, page) + 2
    s["slots"] = torch.randperm(pool * page, generator=g, device=DEV)[:rows].int()
    s["slots"][28::29] = -1
    s["positions"][28::29] = -1
    return pool


def _parents(cu, rows, g):
    """A random tree per request: a token's parent is an earlier one, near ones more often; -1 hangs it from the context."""
    _, local = _requests(cu, rows)
    u = torch.rand(rows, generator=g, device=DEV)
    return ((local + 1).float() * u.sqrt()).floor().clamp(max=local).int() - 1


def prepare(case, seed):
    g = _gen(seed)
    op, dt = case["op"], TYPES[case["dtype"]]
    s = dict(op=op, case=case)
    if "scaling" in case:
        s["positions"] = torch.randint(0, case["far"] + 1, (case["rows"],), generator=g, device=DEV, dtype=torch.int32)
        s["turn"] = _rope(case) if own else (_frequencies(case), _stretch(case).get("attn_factor", 1.0))
    if op.startswith("rotate"):
        rows, d, q, kv = case["rows"], case["head_dim"], case["q_heads"], case["kv_heads"]
        x = _normal((rows, (q + 2 * kv) * d), dt, g)               # one projection's output
        s["q"], s["k"], s["v"] = x[:, :q * d].view(rows, q, d), x[:, q * d:(q + kv) * d].view(rows, kv, d), x[:, (q + kv) * d:].view(rows, kv, d)
        s["q_out"] = torch.zeros((rows, q, d), dtype=dt, device=DEV)
        if op == "rotate":
            s["k_out"] = torch.zeros((rows, kv, d), dtype=dt, device=DEV)
            return s
        pool = _slots(case, s, g)
        s["k_cache"], s["v_cache"] = (torch.zeros((pool, kv, case["page"], d), dtype=dt, device=DEV) for _ in range(2))
        if own:
            from quantized_moe_expert_router_gb300 import moe
            s["attn"] = moe.Attention(q, kv, d, case["page"], pool, pool, dt)
        return s
    h = case["heads"]
    if op == "latent_append":
        rows = case["rows"]
        x = _normal((rows, LATENT + ROPE), dt, g)                  # the projection to the latent, and q's
        s["c"], s["k_rope"] = x[:, :LATENT], x[:, LATENT:]
        s["q_rope"] = _normal((rows, h, NOPE + ROPE), dt, g)[:, :, NOPE:]
        s["q_out"] = torch.zeros((rows, h, ROPE), dtype=dt, device=DEV)
        pool = _slots(case, s, g)
        s["cache"] = torch.zeros((pool, case["page"], LATENT + ROPE), dtype=dt, device=DEV)
        if own:
            s["lat"] = _latent(case, pool, pool)
        return s
    if op == "latent_prompt":
        s["cu"] = _offsets(_shuffled(_prompts(case), g))
        rows, s["longest"] = sum(_prompts(case)), max(_prompts(case))
        s["q"] = _normal((rows, h, NOPE + ROPE), dt, g)
        x = _normal((rows, h, NOPE + VALUE), dt, g)                # the latent's expansion: keys and values of each head
        s["k"], s["v"] = x[:, :, :NOPE], x[:, :, NOPE:]
        s["k_rope"] = _normal((rows, LATENT + ROPE), dt, g)[:, LATENT:]
        pool, width, d = 1, 1, VALUE
    else:
        s["cached"], s["fresh"] = _shuffled(_cached(case), g), _shuffled(_fresh(case), g)
        s["cu"] = _offsets(s["fresh"])
        rows, s["longest"] = sum(_fresh(case)), max(_fresh(case))
        page = case["page"]
        need = (s["cached"] + s["fresh"] + page - 1) // page
        width, pool = int(need.max()), int(need.sum()) + 3
        order = torch.randperm(pool, generator=g, device=DEV).int()
        col = torch.arange(width, device=DEV)
        at = (torch.cumsum(need, 0) - need)[:, None] + col
        s["table"] = torch.where(col < need[:, None], order[at.clamp(max=pool - 1)], -1).int().contiguous()
        s["mask"] = _reach(_parents(s["cu"], rows, g), s["cu"]) if case["tree"] else None
        s["q"] = _normal((h, rows, LATENT), dt, g).transpose(0, 1)    # of a product per head
        s["q_rope"] = _normal((rows, h, NOPE + ROPE), dt, g)[:, :, NOPE:]
        s["cache"] = _normal((pool, page, LATENT + ROPE), dt, g)
        d = LATENT
    s["rows"] = rows
    s["out"] = torch.empty((rows, h, d), dtype=dt, device=DEV)
    s["lse"] = torch.empty((rows, h), dtype=torch.float32, device=DEV)
    if own:
        from quantized_moe_expert_router_gb300 import moe
        s["lat"] = _latent(case, pool, width)
        s["ws"] = moe.alloc_latent_workspace(s["lat"], case["requests"], rows)
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    if own:
        return _call(s)
    return {"rotate": _rotate, "rotate_append": _rotate_append, "latent_append": _latent_append, "latent_prompt": _latent_prompt,
            "latent_tree": _latent_tree}[s["op"]](s)


def _call(s):
    from quantized_moe_expert_router_gb300 import moe
    op = s["op"]
    if op == "rotate":
        moe.moe_rope_apply(s["turn"], s["positions"], s["q"], s["q_out"], s["k"], s["k_out"])
        return [s["q_out"], s["k_out"]]
    if op == "rotate_append":
        moe.moe_rope_append(s["attn"], s["turn"], s["q"], s["k"], s["v"], s["positions"], s["slots"], s["q_out"], s["k_cache"], s["v_cache"])
        return [s["q_out"], s["k_cache"], s["v_cache"]]
    if op == "latent_append":
        moe.moe_latent_append(s["lat"], s["turn"], s["c"], s["k_rope"], s["positions"], s["slots"], s["cache"], q=s["q_rope"], q_out=s["q_out"])
        return [s["q_out"], s["cache"]]
    if op == "latent_prompt":
        moe.moe_latent_prompt(s["lat"], s["q"], s["k"], s["k_rope"], s["v"], s["cu"], s["out"], s["ws"], lse=s["lse"])
    else:
        moe.moe_latent_tree(s["lat"], s["q"], s["q_rope"], s["cu"], s["cached"], s["table"], s["cache"], s["out"], s["ws"],
                            tree_mask=s["mask"], lse=s["lse"])
    return [s["out"], s["lse"]]


def _turned(s, x):
    """x [rows][heads][d] with the first elements of each head turned; the angles in 64 bits, for far positions."""
    freq, factor = s["turn"]
    angle = s["positions"].double()[:, None] * freq
    cos, sin = (angle.cos() * factor).float()[:, None], (angle.sin() * factor).float()[:, None]
    n, y = 2 * freq.numel(), x.float()
    if s["case"]["interleaved"]:
        a, b = y[..., 0:n:2], y[..., 1:n:2]
        y = torch.cat([torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2), y[..., n:]], -1)
    else:
        a, b = y[..., :n // 2], y[..., n // 2:n]
        y = torch.cat([a * cos - b * sin, a * sin + b * cos, y[..., n:]], -1)
    return y.to(x.dtype)


def _rotate(s):
    s["q_out"].copy_(_turned(s, s["q"]))
    s["k_out"].copy_(_turned(s, s["k"]))
    return [s["q_out"], s["k_out"]]


def _rotate_append(s):
    page, live = s["case"]["page"], s["positions"] >= 0
    s["q_out"][live] = _turned(s, s["q"])[live]
    at = s["slots"][live].long()
    s["k_cache"][at // page, :, at % page] = _turned(s, s["k"])[live]
    s["v_cache"][at // page, :, at % page] = s["v"][live]
    return [s["q_out"], s["k_cache"], s["v_cache"]]


def _latent_append(s):
    page, live = s["case"]["page"], s["positions"] >= 0
    s["q_out"][live] = _turned(s, s["q_rope"])[live]
    at = s["slots"][live].long()
    s["cache"][at // page, at % page] = torch.cat([s["c"], _turned(s, s["k_rope"][:, None])[:, 0]], -1)[live]
    return [s["q_out"], s["cache"]]


def _requests(cu, rows):
    """Of each row: its request and its place in it."""
    t = torch.arange(rows, device=DEV)
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True).clamp(max=cu.numel() - 2)
    return b, t - cu[b]


def _reach(parents, cu):
    """The ancestor word of each row: a token sees itself and what it hangs from."""
    b, local = _requests(cu, parents.numel())
    a = torch.eye(TREE, device=DEV).repeat(cu.numel() - 1, 1, 1)
    up = parents >= 0
    a[b[up], local[up], parents[up].long()] = 1.0
    for _ in range(6):                                             # paths of up to 64 steps
        a = (a @ a > 0).float()
    return (a[b, local].long() << torch.arange(TREE, device=DEV)).sum(1)


def _padded(x, cu, longest):
    """[rows][heads][d] of packed requests -> 32-bit [requests][heads][longest][d]."""
    at = cu[:-1, None] + torch.arange(longest, device=DEV)
    return x[at.clamp(max=x.shape[0] - 1)].float().transpose(1, 2)


def _softmax(x, visible):
    """Weights over the last axis and the logarithm of their sum; a row that sees nothing has weights of zero."""
    x = x.masked_fill_(~visible, -math.inf)
    top = x.amax(-1, keepdim=True)
    p = x.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)).exp_()
    z = p.sum(-1, keepdim=True)
    return p.div_(torch.where(z == 0, torch.ones_like(z), z)), (top + z.log()).squeeze(-1)


def _unpadded(s, o, lse):
    b, local = _requests(s["cu"], s["rows"])
    return [o[b, :, local].to(s["q"].dtype), lse[b, :, local]]


def _latent_prompt(s):
    n, cu = s["longest"], s["cu"]
    q = _padded(s["q"], cu, n) * SCALE
    shared = _padded(s["k_rope"][:, None], cu, n)
    x = q[..., :NOPE] @ _padded(s["k"], cu, n).transpose(-1, -2)
    x += q[..., NOPE:] @ shared.transpose(-1, -2)
    i = torch.arange(n, device=DEV)
    length = cu[1:] - cu[:-1]
    p, lse = _softmax(x, ((i <= i[:, None]) & (i < length[:, None, None]))[:, None])
    return _unpadded(s, p @ _padded(s["v"], cu, n), lse)


def _latent_tree(s):
    n, h = s["longest"], s["case"]["heads"]
    kv = s["cache"][s["table"].clamp(min=0).long()].float().flatten(1, 2)      # [requests][key][latent and key part]
    q = torch.cat([_padded(s["q"], s["cu"], n), _padded(s["q_rope"], s["cu"], n)], -1) * SCALE
    x = (q.flatten(1, 2) @ kv.transpose(-1, -2)).view(q.shape[0], h, n, -1)
    j, i = torch.arange(kv.shape[1], device=DEV), torch.arange(n, device=DEV)
    fresh = s["cu"][1:] - s["cu"][:-1]
    new = (j - s["cached"][:, None])[:, None, :]                   # place among the fresh tokens [requests][1][key]
    if s["mask"] is None:
        seen = new <= i[:, None]
    else:
        row = (s["cu"][:-1, None] + i).clamp(max=s["rows"] - 1)
        seen = (new < 0) | ((s["mask"][row][:, :, None] >> new.clamp(0, TREE - 1)) & 1).bool()
    p, lse = _softmax(x, (seen & (new < fresh[:, None, None]))[:, None])
    o = (p.flatten(1, 2) @ kv[..., :LATENT]).view(q.shape[0], h, n, LATENT)
    return _unpadded(s, o, lse)


# ---------------------------------------------------------------- in 64 bits

def _exact_angles(case):
    """cos and sin of every row's pairs, the frequencies written out one by one."""
    n, theta, p = case.get("dims", ROPE), case["theta"], _stretch(case)
    f = []
    for i in range(n // 2):
        base = theta
        if case["scaling"] == "base":
            base *= p["factor"] ** (n / (n - 2))
        w = math.exp(-2 * i / n * math.log(base))
        if case["scaling"] == "linear":
            w /= p["factor"]
        elif case["scaling"] == "yarn":
            first = max(0, math.floor(n / 2 * math.log(p["original"] / (2 * math.pi * p["high"]), theta)))
            last = min(n - 1, math.ceil(n / 2 * math.log(p["original"] / (2 * math.pi * p["low"]), theta)))
            share = 0.0 if i <= first else (1.0 if i >= last else (i - first) / (last - first))
            w *= 1 - share + share / p["factor"]
        elif case["scaling"] == "bands":
            turns = p["original"] * w / (2 * math.pi)
            if turns < p["low"]:
                w /= p["factor"]
            elif turns <= p["high"]:
                share = (turns - p["low"]) / (p["high"] - p["low"])
                w = (1 - share) * w / p["factor"] + share * w
        f.append(w)
    return torch.tensor(f, dtype=torch.float64, device=DEV), p.get("attn_factor", 1.0)


def _exact_turn(case, positions, x):
    f, factor = _exact_angles(case)
    turn = torch.polar(torch.full_like(positions, 1).double()[:, None] * torch.full_like(f, factor), positions.double()[:, None] * f)[:, None]
    n, y = 2 * f.numel(), x.double().clone()
    part = y[..., :n].unflatten(-1, (n // 2, 2) if case["interleaved"] else (2, n // 2))
    if not case["interleaved"]:
        part = part.transpose(-1, -2)
    z = torch.view_as_real(torch.view_as_complex(part.contiguous()) * turn)
    y[..., :n] = (z if case["interleaved"] else z.transpose(-1, -2)).flatten(-2)
    return y


def exact(case, seed):
    """The definition in 64 bits; attention one request and one head at a time."""
    s = prepare(case, seed)
    op = case["op"]
    if "scaling" in case:
        dead = (s["positions"] < 0)[:, None, None]
        q = torch.where(dead, 0.0, _exact_turn(case, s["positions"], s["q"] if "q" in s else s["q_rope"]))
        if op == "rotate":
            return [q, _exact_turn(case, s["positions"], s["k"])]
        if op == "rotate_append":
            rows = [_exact_turn(case, s["positions"], s["k"]), s["v"].double()]
        else:
            rows = [torch.cat([s["c"].double()[:, None], _exact_turn(case, s["positions"], s["k_rope"][:, None])], -1)]
        caches = []
        for x in rows:
            pool = (s["cache"] if op == "latent_append" else s["k_cache"]).shape[0]
            by_token = torch.zeros((pool * case["page"] + 1, *x.shape[1:]), dtype=torch.float64, device=DEV)
            by_token[s["slots"].long()] = x                        # rows without a slot go to the last place, which is dropped
            by_page = by_token[:-1].unflatten(0, (pool, case["page"]))
            caches.append(by_page.transpose(1, 2).contiguous() if op == "rotate_append" else by_page[:, :, 0].contiguous())
        return [q] + caches
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device=DEV)
    cu = s["cu"].tolist()
    cached = s["cached"].tolist() if op == "latent_tree" else [0] * case["requests"]
    for b in range(case["requests"]):
        lo, hi, c = cu[b], cu[b + 1], cached[b]
        if op == "latent_tree":
            all_keys = s["cache"][s["table"][b, :_ceil(c + hi - lo, case["page"])].long()].flatten(0, 1)[:c + hi - lo].double()
        sees = torch.ones((hi - lo, hi - lo), dtype=torch.bool, device=DEV).tril()
        if s.get("mask") is not None:
            sees = torch.stack([(s["mask"][lo:hi] >> j) & 1 for j in range(hi - lo)], 1).bool()
        for h in range(case["heads"]):
            if op == "latent_tree":
                k, v = all_keys, all_keys[:, :LATENT]
                q = torch.cat([s["q"][lo:hi, h], s["q_rope"][lo:hi, h]], -1).double()
            else:
                k = torch.cat([s["k"][lo:hi, h], s["k_rope"][lo:hi]], -1).double()
                v, q = s["v"][lo:hi, h].double(), s["q"][lo:hi, h].double()
            for r0 in range(0, hi - lo, 4096):                     # rows in parts: keys past a part's last row are not looked at
                r1 = min(hi - lo, r0 + 4096)
                last = c + (r1 if s.get("mask") is None else hi - lo)
                x = q[r0:r1] @ k[:last].T * SCALE
                x[:, c:] = torch.where(sees[r0:r1, :last - c], x[:, c:], -math.inf)
                lse[lo + r0:lo + r1, h] = torch.logsumexp(x, -1)
                out[lo + r0:lo + r1, h] = torch.softmax(x, -1).nan_to_num(0.0) @ v[:last]
    return [out, lse]
