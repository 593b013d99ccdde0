"""Cases of the attention beside the routed MoE FFN: what a serving step runs
over a paged key/value cache before it calls the FFN.

  plan     block tables, slot maps, positions and tree masks from the
           requests' lengths (moe_kv_plan)
  append   the step's key and value rows into their cache slots (moe_kv_append)
  prompt   causal attention over whole prompts, packed (moe_attn_prompt)
  tree     attention of drafted trees, or of single tokens, over the cache
           (moe_attn_tree)

``run`` computes a case in plain torch operations, or with ``own`` set
through the library's entry points.  A request's context is the ``cached``
tokens that are in the cache already and the ``fresh`` ones of this step.
The requests' lengths follow from the case (falling by a constant factor from
the given longest one); a seed orders them and makes everything else."""
import math

import torch

own = False
DEV = "cuda:0"
TREE = 64          # tokens of a drafted tree at most: the bits of a mask word
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # The verify step of 7 streams with a drafted tree of up to 8 tokens each: a small step, latency counts.
        dict(name="plan, 7 trees", op="plan", requests=7, cached=4000, fresh=8, tree=True, page=16),
        # Admission of a batch of prompts of ragged lengths: every page is new.
        dict(name="plan, 48 prompts", op="plan", requests=48, cached=0, fresh=1900, tree=False, page=32),
        # The rows of that verify step, out of a fused projection's output.
        dict(name="append, 56 rows", op="append", dtype="bf16", tokens=56, kv_heads=8, group=4, head_dim=128, page=16),
        # The rows of a large batch of prompts; every 29th row has no slot (the padding of a fixed-size step).
        dict(name="append, 16384 rows", op="append", dtype="f16", tokens=16384, kv_heads=8, group=2, head_dim=128, page=64),
        # One prompt of 512 tokens, the length of the layer's prefill workload.
        dict(name="prompt, 512", op="prompt", dtype="bf16", requests=1, longest=512, ragged=False, kv_heads=8, group=4,
             head_dim=128),
        # A batch of short and middling prompts, with odd lengths and an odd group.
        dict(name="prompt, 17 ragged", op="prompt", dtype="f16", requests=17, longest=1501, ragged=True, kv_heads=8, group=3,
             head_dim=64),
        # Four prompts of a few thousand tokens.
        dict(name="prompt, 4 x 4096", op="prompt", dtype="bf16", requests=4, longest=4096, ragged=False, kv_heads=4, group=8,
             head_dim=128),
        # One long document.
        dict(name="prompt, 16384", op="prompt", dtype="bf16", requests=1, longest=16384, ragged=False, kv_heads=2, group=8,
             head_dim=128),
        # One stream, one token, a short context: the smallest decode.
        dict(name="tree, 1 token at 1000", op="tree", dtype="bf16", requests=1, cached=1000, fresh=1, tree=False, kv_heads=8,
             group=4, head_dim=128, page=16),
        # The verify step: trees of up to 8 in 8 streams of up to a few thousand tokens.
        dict(name="tree, 8 x 8 at 4000", op="tree", dtype="bf16", requests=8, cached=4000, fresh=8, tree=True, kv_heads=8,
             group=4, head_dim=128, page=64),
        # Wide trees of up to 64 drafted tokens over long contexts: many query rows to a key.
        dict(name="tree, 4 x 64 at 9000", op="tree", dtype="f16", requests=4, cached=9000, fresh=64, tree=True, kv_heads=4,
             group=8, head_dim=128, page=128),
        # Decode of 16 streams of up to 100 thousand tokens: the cache is read once and nothing else counts.
        dict(name="tree, 16 tokens at 100000", op="tree", dtype="bf16", requests=16, cached=100000, fresh=1, tree=False,
             kv_heads=8, group=8, head_dim=128, page=32),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def _drawn(rng):
    op = rng.choice(["plan", "append", "prompt", "prompt", "tree", "tree"])
    heads = dict(dtype=rng.choice(["bf16", "f16"]), kv_heads=rng.choice([1, 2, 3, 4, 8]),
                 group=rng.choice([1, 2, 3, 4, 5, 6, 8, 12, 16]), head_dim=rng.choice([64, 128]))
    page = rng.choice([16, 32, 64, 128])
    if op == "plan":
        if rng.random() < 0.5:
            return dict(op=op, requests=_log(rng, 1, 256), cached=_log(rng, 1, 20000), fresh=_log(rng, 1, TREE), tree=True, page=page)
        return dict(op=op, requests=_log(rng, 1, 256), cached=rng.choice([0, _log(rng, 1, 20000)]), fresh=_log(rng, 1, 1900), tree=False,
                    page=page)
    if op == "append":
        return dict(op=op, tokens=_log(rng, 1, 16384), page=page, **heads)
    if op == "prompt":
        return dict(op=op, requests=_log(rng, 1, 64), longest=_log(rng, 1, 16384), ragged=rng.random() < 0.7, **heads)
    return dict(op=op, requests=_log(rng, 1, 64), cached=_log(rng, 1, 100000), fresh=rng.choice([1, _log(rng, 2, TREE)]),
                tree=rng.random() < 0.7, page=page, **heads)


def _fits(case):
    """No dearer than the largest listed case of its operator, in the plain form either."""
    if case["op"] == "prompt":
        L, q = case["longest"], case["kv_heads"] * case["group"]
        return case["requests"] * q * L * L <= 16 * 16384 ** 2 and case["requests"] * L * q <= 16384 * 32
    if case["op"] == "tree":
        n, kv = case["requests"] * (case["cached"] + case["fresh"]), case["kv_heads"] * case["head_dim"]
        return n * kv <= 16 * 100000 * 1024 and n * kv * case["group"] * case["fresh"] <= 4 * 9000 * 64 * 32 * 128
    if case["op"] == "plan":
        return sum(_fresh(case)) <= 48 * 1900
    return True


def draw(rng):
    while True:
        case = _drawn(rng)
        if _fits(case):
            return case


def _falling(n, longest, span):
    """n lengths from `longest` down to a span-th of it (one at least)."""
    return [max(1, int(longest * span ** (-i / max(1, n - 1)))) for i in range(n)]


def _fresh(case):
    return _falling(case["requests"], case["fresh"], 16.0 if not case["tree"] else 4.0)


def _cached(case):
    return _falling(case["requests"], case["cached"], 8.0) if case["cached"] else [0] * case["requests"]


def _prompts(case):
    return _falling(case["requests"], case["longest"], 24.0 if case["ragged"] else 1.0)


def _ceil(a, b):
    return -(-a // b)


def work(case):
    """Each input once, each output once; products of visible (query, key) pairs."""
    op = case["op"]
    if op == "plan":
        f, c = _fresh(case), _cached(case)
        new = sum(_ceil(a + b, case["page"]) - _ceil(b, case["page"]) for a, b in zip(f, c))
        return {"bytes": 4 * (3 * case["requests"] + 1) + 8 * new + sum(f) * (8 + (12 if case["tree"] else 0)) + 16, "flops": 0}
    d, kv, g = case["head_dim"], case["kv_heads"], case["group"]
    if op == "append":
        return {"bytes": case["tokens"] * (4 + 2 * 2 * 2 * kv * d), "flops": 0}
    if op == "prompt":
        n = _prompts(case)
        return {"bytes": sum(n) * (2 * d * (2 * kv * g + 2 * kv) + 4 * kv * g), "flops": sum(2 * d * kv * g * a * (a + 1) for a in n)}
    f, c = _fresh(case), _cached(case)
    rows, context = sum(f), sum(f) + sum(c)
    pages = sum(_ceil(a + b, case["page"]) for a, b in zip(f, c))
    return {"bytes": context * 2 * 2 * kv * d + rows * kv * g * (4 * d + 4) + 4 * pages + (8 * rows if case["tree"] else 0),
            "flops": sum(4 * d * kv * g * a * (b + (a + 1) / 2) for a, b in zip(f, c))}


# ---------------------------------------------------------------- the inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _shuffled(values, g):
    return _ints(values)[torch.randperm(len(values), generator=g, device=DEV)]


def _offsets(fresh):
    cu = torch.zeros(fresh.numel() + 1, dtype=torch.int32, device=DEV)
    cu[1:] = torch.cumsum(fresh, 0)
    return cu


def _parents(cu, rows, g):
    """A random tree per request: a token's parent is an earlier one, near ones more often; -1 hangs it from the context."""
    t = torch.arange(rows, device=DEV)
    local = t - cu[torch.searchsorted(cu[1:-1].contiguous(), t, right=True)] if cu.numel() > 2 else t
    u = torch.rand(rows, generator=g, device=DEV)
    return ((local + 1).float() * u.sqrt()).floor().clamp(max=local).int() - 1


def _pages(case, cached, fresh, g, new):
    """A shuffled pool of pages: the requests' own first (all of the context's, or the cached tokens' only), the rest free."""
    page = case["page"]
    need = (cached + fresh + page - 1) // page
    have = (cached + page - 1) // page if new else need
    width = int(need.max())
    pool = int(need.sum()) + 3
    order = torch.randperm(pool, generator=g, device=DEV).int()
    col = torch.arange(width, device=DEV)
    first = torch.cumsum(have, 0) - have
    at = first[:, None] + col
    table = torch.where(col < have[:, None], order[at.clamp(max=pool - 1)], -1).int()
    return table.contiguous(), order[int(have.sum()):].contiguous(), pool


def _library(case, pool, width):
    from quantized_moe_expert_router_gb300 import moe
    return moe.Attention(case.get("kv_heads", 1) * case.get("group", 1), case.get("kv_heads", 1), case.get("head_dim", 64), case.get("page", 16),
                         pool, width, TYPES[case.get("dtype", "bf16")])


def _fused(case, rows, g):
    """q, k, v as views of one projection's output [rows][(q_heads + 2 kv_heads) * head_dim]."""
    d, kv, q = case["head_dim"], case["kv_heads"], case["kv_heads"] * case["group"]
    x = torch.randn((rows, (q + 2 * kv) * d), generator=g, device=DEV, dtype=torch.float32).to(TYPES[case["dtype"]])
    return (x[:, :q * d].view(rows, q, d), x[:, q * d:(q + kv) * d].view(rows, kv, d), x[:, (q + kv) * d:].view(rows, kv, d))


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = dict(op=op, case=case)
    if op == "plan":
        s["cached"], s["fresh"] = _shuffled(_cached(case), g), _shuffled(_fresh(case), g)
        rows = _ceil(sum(_fresh(case)), 8) * 8                     # a fixed-size step: some rows stay empty
        s["table"], s["free"], pool = _pages(case, s["cached"], s["fresh"], g, True)
        s["parents"] = _parents(_offsets(s["fresh"]), rows, g) if case["tree"] else None
        s["cu"] = torch.empty(case["requests"] + 1, dtype=torch.int32, device=DEV)
        s["slots"], s["positions"] = (torch.empty(rows, dtype=torch.int32, device=DEV) for _ in range(2))
        s["mask"] = torch.empty(rows, dtype=torch.int64, device=DEV) if case["tree"] else None
        s["info"] = torch.zeros(4, dtype=torch.int32, device=DEV)
        if own:
            s["attn"] = _library(case, pool, s["table"].shape[1])
        return s
    dt, d, kv = TYPES[case["dtype"]], case["head_dim"], case["kv_heads"]
    if op == "append":
        rows, page = case["tokens"], case["page"]
        pool = _ceil(rows, page) + 2
        s["slots"] = torch.randperm(pool * page, generator=g, device=DEV)[:rows].int()
        s["slots"][28::29] = -1
        _, s["k"], s["v"] = _fused(case, rows, g)
        s["k_cache"], s["v_cache"] = (torch.zeros((pool, kv, page, d), dtype=dt, device=DEV) for _ in range(2))
        if own:
            s["attn"] = _library(case, pool, pool)
        return s
    if op == "prompt":
        s["cu"] = _offsets(_shuffled(_prompts(case), g))
        rows = sum(_prompts(case))
        s["q"], s["k"], s["v"] = _fused(case, rows, g)
        s["longest"] = max(_prompts(case))
        pool, width = 1, 1
    else:
        s["cached"], s["fresh"] = _shuffled(_cached(case), g), _shuffled(_fresh(case), g)
        s["cu"] = _offsets(s["fresh"])
        rows = sum(_fresh(case))
        s["table"], _, pool = _pages(case, s["cached"], s["fresh"], g, False)
        width = s["table"].shape[1]
        s["mask"] = _reach(_parents(s["cu"], rows, g), s["cu"])[0] if case["tree"] else None
        s["q"] = _fused(case, rows, g)[0]
        s["k_cache"], s["v_cache"] = (torch.randn((pool, kv, case["page"], d), generator=g, device=DEV, dtype=dt) for _ in range(2))
        s["longest"] = max(_fresh(case))
    s["rows"] = rows
    s["out"] = torch.empty((rows, kv * case["group"], d), dtype=dt, device=DEV)
    s["lse"] = torch.empty((rows, kv * case["group"]), dtype=torch.float32, device=DEV)
    if own:
        from quantized_moe_expert_router_gb300 import moe
        s["attn"] = _library(case, pool, width)
        s["ws"] = moe.alloc_attn_workspace(s["attn"], case["requests"], rows)
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    if own:
        return _call(s)
    return {"plan": _plan, "append": _append, "prompt": _prompt, "tree": _tree}[s["op"]](s)


def _call(s):
    from quantized_moe_expert_router_gb300 import moe
    if s["op"] == "plan":
        moe.moe_kv_plan(s["attn"], s["cached"], s["fresh"], s["free"], s["table"], s["cu"], s["slots"], s["positions"], s["info"],
                        parents=s["parents"], tree_mask=s["mask"])
        return [s["table"], s["cu"], s["slots"], s["positions"], s["info"], s["mask"]]
    if s["op"] == "append":
        moe.moe_kv_append(s["attn"], s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"])
        return [s["k_cache"], s["v_cache"]]
    if s["op"] == "prompt":
        moe.moe_attn_prompt(s["attn"], s["q"], s["k"], s["v"], s["cu"], s["out"], s["ws"], lse=s["lse"])
    else:
        moe.moe_attn_tree(s["attn"], s["q"], s["cu"], s["cached"], s["table"], s["k_cache"], s["v_cache"], s["out"], s["ws"],
                          tree_mask=s["mask"], lse=s["lse"])
    return [s["out"], s["lse"]]


def _requests(cu, rows):
    """Of each row: its request, its place in it, and whether it belongs to one."""
    t = torch.arange(rows, device=DEV)
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    real = t < cu[-1]
    b = b.clamp(max=cu.numel() - 2)
    return b, t - cu[b], real


def _twice(r):
    return (r @ r > 0).float()


def _reach(parents, cu):
    """Ancestor words (a token sees itself and what it hangs from) and the number of ancestors, of each row."""
    b, local, real = _requests(cu, parents.numel())
    a = torch.eye(TREE, device=DEV).repeat(cu.numel() - 1, 1, 1)
    up = real & (parents >= 0)
    a[b[up], local[up], parents[up].long()] = 1.0
    a = _twice(_twice(_twice(_twice(_twice(_twice(a))))))          # paths of up to 64 steps
    bits = torch.ones(TREE, dtype=torch.int64, device=DEV) << torch.arange(TREE, device=DEV)
    rows = a[b, local.clamp(0, TREE - 1)] * real[:, None]
    return (rows.long() * bits).sum(1), (rows.sum(1) - 1).int()


def _plan(s):
    page, cached, fresh = s["case"]["page"], s["cached"].long(), s["fresh"].long()
    cu = _offsets(fresh)
    need, have = (cached + fresh + page - 1) // page, (cached + page - 1) // page
    first = torch.cumsum(need - have, 0) - (need - have)
    col = torch.arange(s["table"].shape[1], device=DEV)
    at = (first[:, None] + col - have[:, None]).clamp(0, s["free"].numel() - 1)
    table = torch.where((col >= have[:, None]) & (col < need[:, None]), s["free"][at], s["table"])
    b, local, real = _requests(cu, s["slots"].numel())
    place = (cached[b] + local).clamp(max=table.shape[1] * page - 1)
    slots = torch.where(real, table[b, place // page].long() * page + place % page, -1).int()
    mask, depth = _reach(s["parents"], cu) if s["parents"] is not None else (None, local)
    positions = torch.where(real, cached[b] + depth, -1).int()
    info = torch.stack([cu[-1].long(), (need - have).sum(), (cached + fresh).max(), torch.zeros_like(cu[-1]).long()]).int()
    return [table, cu, slots, positions, info, mask]


def _append(s):
    page, keep = s["case"]["page"], s["slots"] >= 0
    at = s["slots"][keep].long()
    s["k_cache"][at // page, :, at % page] = s["k"][keep]
    s["v_cache"][at // page, :, at % page] = s["v"][keep]
    return [s["k_cache"], s["v_cache"]]


def _softmax(x, visible):
    """Weights over the last axis and the logarithm of their sum; a row that sees nothing has weights of zero."""
    x = x.masked_fill_(~visible, -math.inf)
    top = x.amax(-1, keepdim=True)
    p = x.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)).exp_()
    z = p.sum(-1, keepdim=True)
    return p.div_(torch.where(z == 0, torch.ones_like(z), z)), (top + z.log()).squeeze(-1)


def _padded(x, cu, longest):
    """[rows][heads][d] of packed requests -> 32-bit [requests][heads][longest][d]."""
    at = cu[:-1, None] + torch.arange(longest, device=DEV)
    return x[at.clamp(max=x.shape[0] - 1)].float().transpose(1, 2)


def _attend(s, k, v, visible):
    """Softmax attention of the packed queries over 32-bit k, v [requests][kv_heads][keys][d] where visible [requests][row][key]."""
    case = s["case"]
    d, kv, group, n = case["head_dim"], case["kv_heads"], case["group"], s["longest"]
    q = _padded(s["q"], s["cu"], n)                                # [requests][q_heads][n][d]
    q = q.reshape(q.shape[0], kv, group * n, d) / math.sqrt(d)
    x = (q @ k.transpose(-1, -2)).view(q.shape[0], kv, group, n, -1)
    p, lse = _softmax(x, visible[:, None, None])
    o = (p.view(q.shape[0], kv, group * n, -1) @ v).view(q.shape[0], kv * group, n, d)
    b, local, _ = _requests(s["cu"], s["rows"])
    return [o[b, :, local].to(s["q"].dtype), lse.view(q.shape[0], kv * group, n)[b, :, local]]


def _prompt(s):
    n = s["longest"]
    k, v = _padded(s["k"], s["cu"], n), _padded(s["v"], s["cu"], n)
    i = torch.arange(n, device=DEV)
    length = s["cu"][1:] - s["cu"][:-1]
    visible = (i <= i[:, None]) & (i < length[:, None, None])
    return _attend(s, k, v, visible)


def _tree(s):
    case = s["case"]
    at = s["table"].clamp(min=0).long()
    k, v = (c[at].float().transpose(1, 2).reshape(at.shape[0], case["kv_heads"], -1, case["head_dim"]) for c in (s["k_cache"], s["v_cache"]))
    j = torch.arange(k.shape[2], device=DEV)
    i = torch.arange(s["longest"], device=DEV)
    fresh = s["cu"][1:] - s["cu"][:-1]
    new = (j - s["cached"][:, None])[:, None, :]                   # place among the fresh tokens [requests][1][key]
    if s["mask"] is None:
        seen = new <= i[:, None]
    else:
        row = (s["cu"][:-1, None] + i).clamp(max=s["rows"] - 1)
        seen = (new < 0) | ((s["mask"][row][:, :, None] >> new.clamp(0, TREE - 1)) & 1).bool()
    return _attend(s, k, v, seen & (new < fresh[:, None, None]))


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    """The definition in 64 bits, one request and one head at a time; a plan computes no numbers."""
    if case["op"] == "plan":
        return None
    s = prepare(case, seed)
    d, kv, group, page = case["head_dim"], case["kv_heads"], case["group"], case.get("page")
    if case["op"] == "append":
        caches = []
        for x, c in ((s["k"], s["k_cache"]), (s["v"], s["v_cache"])):
            by_token = torch.zeros((c.shape[0] * page + 1, kv, d), dtype=torch.float64, device=DEV)
            by_token[s["slots"].long()] = x.double()               # rows without a slot go to the last place, which is dropped
            caches.append(by_token[:-1].view(-1, page, kv, d).transpose(1, 2).contiguous())
        return caches
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device=DEV)
    cu = s["cu"].tolist()
    cached = s["cached"].tolist() if case["op"] == "tree" else [0] * case["requests"]
    for b in range(case["requests"]):
        lo, hi, c = cu[b], cu[b + 1], cached[b]
        for h in range(kv):
            if case["op"] == "prompt":
                k, v = s["k"][lo:hi, h].double(), s["v"][lo:hi, h].double()
            else:
                own_pages = s["table"][b, :_ceil(c + hi - lo, page)].long()
                k, v = (x[own_pages, h].reshape(-1, d)[:c + hi - lo].double() for x in (s["k_cache"], s["v_cache"]))
            sees = torch.ones((hi - lo, hi - lo), dtype=torch.bool, device=DEV).tril()
            if s.get("mask") is not None:
                sees = torch.stack([(s["mask"][lo:hi] >> j) & 1 for j in range(hi - lo)], 1).bool()
            for r0 in range(0, hi - lo, 4096):                     # rows in parts: keys past a part's last row are not looked at
                r1 = min(hi - lo, r0 + 4096)
                last = c + (r1 if s.get("mask") is None else hi - lo)
                for head in range(h * group, (h + 1) * group):
                    x = s["q"][lo + r0:lo + r1, head].double() @ k[:last].T / math.sqrt(d)
                    x[:, c:] = torch.where(sees[r0:r1, :last - c], x[:, c:], -math.inf)
                    lse[lo + r0:lo + r1, head] = torch.logsumexp(x, -1)
                    w = torch.softmax(x, -1).nan_to_num(0.0)
                    out[lo + r0:lo + r1, head] = w @ v[:last]
    return [out, lse]
