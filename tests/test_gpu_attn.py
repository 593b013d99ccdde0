"""The attention beside the FFN on the GPU: plan, append, prompt and tree
attention against their definitions in 64 bits (``attn_ref``)."""
import math

import numpy as np
import pytest
import torch

import attn_ref as ref
from quantized_moe_expert_router_gb300 import moe

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_moe_expert_router_gb300 import build
    build.build()
    moe.load_library()


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def randn(shape, dt, seed, scale=1.0):
    return (torch.randn(shape, generator=gen(seed), device=DEV) * scale).to(dt)


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def offsets(lengths):
    return ints(np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32).tolist())


# ---------------------------------------------------------------- prompts

def prompt_ref(q, k, v, lengths, scale, lo=0):
    parts = []
    for n in lengths:
        vis = torch.ones((n, n), dtype=torch.bool, device=DEV).tril()
        parts.append(ref.attend(q[lo:lo + n], k[lo:lo + n], v[lo:lo + n], vis, scale))
        lo += n
    return [torch.cat([p[i] for p in parts]) for i in range(4)]


def run_prompt(attn, q, k, v, lengths, lse=True):
    out = torch.empty(q.shape, dtype=q.dtype, device=DEV)
    l = torch.empty(q.shape[:2], dtype=torch.float32, device=DEV) if lse else None
    moe.moe_attn_prompt(attn, q, k, v, offsets(lengths), out, moe.alloc_attn_workspace(attn, len(lengths), q.shape[0]), lse=l)
    torch.cuda.synchronize()
    return out, l


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("hk,g,d,lengths", [
    (1, 1, 64, [1]), (2, 4, 128, [2, 1, 3]), (2, 3, 64, [0, 5, 0, 17, 0]), (1, 8, 128, [127, 128, 129]),
    (8, 1, 64, [63, 64, 65, 200]), (1, 16, 128, [300]), (1, 128, 64, [9, 1, 30]), (2, 5, 128, [511, 33]),
    (1, 12, 64, [1000, 7]), (3, 2, 128, [1, 640, 385]), (1, 48, 128, [70, 11]), (1, 1, 128, [257, 1025]),
])
def test_prompt_parity(dt, hk, g, d, lengths):
    T = sum(lengths)
    attn = moe.Attention(hk * g, hk, d, 16, 1, 1, TYPES[dt])
    q, k, v = randn((T, hk * g, d), TYPES[dt], 1, 1.5), randn((T, hk, d), TYPES[dt], 2), randn((T, hk, d), TYPES[dt], 3)
    out, lse = run_prompt(attn, q, k, v, lengths)
    ref.check(out, lse, prompt_ref(q, k, v, lengths, d ** -0.5))


def test_prompt_many_requests():
    lengths = [(7 * i) % 23 for i in range(1024)]
    T, dt = sum(lengths), torch.bfloat16
    attn = moe.Attention(4, 2, 64, 16, 1, 1, dt)
    q, k, v = randn((T, 4, 64), dt, 1), randn((T, 2, 64), dt, 2), randn((T, 2, 64), dt, 3)
    out, lse = run_prompt(attn, q, k, v, lengths)
    ref.check(out, lse, prompt_ref(q, k, v, lengths, 0.125))


@pytest.mark.parametrize("order", ["fused", "heads_first", "gaps"])
def test_prompt_strides(order):
    hk, g, d, lengths, dt = 2, 3, 64, [150, 45], torch.bfloat16
    T, hq = sum(lengths), hk * g
    attn = moe.Attention(hq, hk, d, 16, 1, 1, dt)
    if order == "fused":
        x = randn((T, (hq + 2 * hk) * d), dt, 4)
        q, k, v = x[:, :hq * d].view(T, hq, d), x[:, hq * d:(hq + hk) * d].view(T, hk, d), x[:, (hq + hk) * d:].view(T, hk, d)
        out = torch.full((T, 2 * hq * d), 7.0, dtype=dt, device=DEV)
        o = out[:, hq * d:].view(T, hq, d)
    elif order == "heads_first":
        q, k, v = (randn((h, T, d), dt, 5 + i).transpose(0, 1) for i, h in enumerate((hq, hk, hk)))
        o = torch.empty((hq, T, d), dtype=dt, device=DEV).transpose(0, 1)
    else:
        q, k, v = (randn((2 * T, h + 1, d + 8), dt, 5 + i)[::2, 1:, :d] for i, h in enumerate((hq, hk, hk)))
        o = torch.empty((T, hq, d + 24), dtype=dt, device=DEV)[:, :, 8:d + 8]
    moe.moe_attn_prompt(attn, q, k, v, offsets(lengths), o, moe.alloc_attn_workspace(attn, 2, T))
    torch.cuda.synchronize()
    ref.check(o, None, prompt_ref(q, k, v, lengths, d ** -0.5))
    if order == "fused":
        assert (out[:, :hq * d] == 7.0).all()


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("d,dt", [(64, "bf16"), (128, "f16"), (128, "bf16")])
def test_prompt_unseen_rows_have_no_effect(d, dt, bad):
    """Rows after a row, other requests' rows and rows of no request hold anything."""
    dt, hk, g, lengths = TYPES[dt], 2, 2, [130, 75, 300]
    pad0, pad1 = 5, 40
    T = pad0 + sum(lengths) + pad1
    attn = moe.Attention(hk * g, hk, d, 16, 1, 1, dt)
    q, k, v = (randn((T, h, d), dt, 10 + i) for i, h in enumerate((hk * g, hk, hk)))
    clean = [x.clone() for x in (q, k, v)]
    cu = offsets(lengths) + pad0
    poisoned = []
    for b, last in enumerate([129, 60, 170]):            # from this row on, the request is poisoned
        lo = int(cu[b])
        for x in (q, k, v):
            x[lo + last:lo + lengths[b]] = bad
        poisoned.append((lo, lo + last))
    for x in (q, k, v):
        x[:pad0] = bad
        x[T - pad1:] = bad
    out = torch.full((T, hk * g, d), 3.0, dtype=dt, device=DEV)
    moe.moe_attn_prompt(attn, q, k, v, cu, out, moe.alloc_attn_workspace(attn, 3, T))
    torch.cuda.synchronize()
    want = prompt_ref(*(x for x in clean), lengths, d ** -0.5, pad0)
    for b, (lo, hi) in enumerate(poisoned):
        at = slice(lo - pad0, hi - pad0)
        ref.check(out[lo:hi], None, [w[at] for w in want], f"request {b}")
        assert torch.isnan(out[hi:int(cu[b + 1])].float()).all(), "rows that see a poisoned row"
    assert (out[:pad0] == 3.0).all() and (out[T - pad1:] == 3.0).all()


@pytest.mark.parametrize("where", ["v_inf", "k_nan"])
def test_prompt_one_bad_token_reaches_the_rows_that_see_it(where):
    d, n, at, dt = 128, 300, 140, torch.bfloat16
    attn = moe.Attention(2, 1, d, 16, 1, 1, dt)
    q, k, v = (randn((n, h, d), dt, 20 + i) for i, h in enumerate((2, 1, 1)))
    if where == "v_inf":
        v[at, 0, 3] = math.inf
    else:
        k[at, 0, 3] = math.nan
    out, _ = run_prompt(attn, q, k, v, [n])
    vis = torch.ones((at, at), dtype=torch.bool, device=DEV).tril()
    ref.check(out[:at], None, ref.attend(q[:at], k[:at], v[:at], vis, d ** -0.5))
    if where == "v_inf":
        assert (out[at:, :, 3] == math.inf).all()
        assert torch.isfinite(out[at:, :, :3]).all() and torch.isfinite(out[at:, :, 4:]).all()
    else:
        assert torch.isnan(out[at:].float()).all()


def test_prompt_large_scores():
    """Scores of several hundred: one weight is 1, the maximum jumps from tile to tile."""
    d, n, dt = 128, 700, torch.bfloat16
    attn = moe.Attention(4, 1, d, 16, 1, 1, dt)
    q, k, v = randn((n, 4, d), dt, 30, 20.0), randn((n, 1, d), dt, 31, 3.0), randn((n, 1, d), dt, 32)
    k = (k.float() * torch.linspace(0.1, 3, n, device=DEV)[:, None, None]).to(dt)
    out, lse = run_prompt(attn, q, k, v, [n])
    ref.check(out, lse, prompt_ref(q, k, v, [n], d ** -0.5))


@pytest.mark.parametrize("hk,g,d,lengths", [(1, 12, 64, [1000, 7]), (2, 8, 64, [1500]), (1, 3, 128, [900, 300])])
def test_prompt_fresh_data_every_call(hk, g, d, lengths):
    """Other values in every call: what an earlier call left in shared memory is of no use.  The key tiles of the long
    requests go round the ring more than once before their masked tiles come."""
    T, dt = sum(lengths), torch.float16
    attn = moe.Attention(hk * g, hk, d, 16, 1, 1, dt)
    for rep in range(8):
        q, k, v = (randn((T, h, d), dt, 50 + 3 * rep + i, 1.5 if i == 0 else 1.0) for i, h in enumerate((hk * g, hk, hk)))
        want = prompt_ref(q, k, v, lengths, d ** -0.5)
        ref.check(*run_prompt(attn, q, k, v, lengths), want, f"call {rep}")


def test_prompt_scale_and_slope():
    """A small softmax_scale: near-uniform weights; v of large magnitude."""
    d, n, dt = 64, 333, torch.float16
    attn = moe.Attention(2, 2, d, 16, 1, 1, dt, softmax_scale=0.001)
    q, k, v = randn((n, 2, d), dt, 33), randn((n, 2, d), dt, 34), randn((n, 2, d), dt, 35, 100.0)
    out, lse = run_prompt(attn, q, k, v, [n])
    ref.check(out, lse, prompt_ref(q, k, v, [n], 0.001))


# ---------------------------------------------------------------- the cache

class Cache:
    """A cache with shuffled pages, filled for the given contexts; everything else in it is NaN."""

    def __init__(self, hq, hk, d, page, dt, cached, fresh, seed=0, spare=3, extra_cols=2):
        self.hk, self.d, self.page, self.dt = hk, d, page, dt
        rng = np.random.default_rng(seed)
        ctx = [c + f for c, f in zip(cached, fresh)]
        need = [-(-n // page) for n in ctx]
        pool = sum(need) + spare
        width = max(need, default=0) + extra_cols
        order = rng.permutation(pool).astype(np.int32)
        table = np.full((len(ctx), width), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            at += n
        self.attn = moe.Attention(hq, hk, d, page, pool, width, dt)
        self.table, self.cached, self.fresh = ints(table.tolist()).view(len(ctx), width), ints(list(cached)), list(fresh)
        self.cu = offsets(fresh)
        self.k, self.v = (torch.full((pool, hk, page, d), math.nan, dtype=dt, device=DEV) for _ in range(2))
        self.rows = []
        for b, n in enumerate(ctx):
            kv = [randn((n, hk, d), dt, 1000 * seed + 2 * b + i) for i in range(2)]
            self.rows.append(kv)
            p = torch.arange(n, device=DEV)
            pg = self.table[b, p // page].long()
            self.k[pg, :, p % page] = kv[0]
            self.v[pg, :, p % page] = kv[1]
        self.T = sum(fresh)
        self.q = randn((self.T, hq, d), dt, 1000 * seed + 999, 1.5)

    def run(self, mask=None, lse=True, **kw):
        out = torch.full(self.q.shape, 9.0, dtype=self.dt, device=DEV)
        l = torch.empty(self.q.shape[:2], dtype=torch.float32, device=DEV) if lse else None
        ws = moe.alloc_attn_workspace(self.attn, len(self.fresh), self.T)
        moe.moe_attn_tree(self.attn, kw.get("q", self.q), self.cu, self.cached, self.table, self.k, self.v, out, ws, tree_mask=mask, lse=l)
        torch.cuda.synchronize()
        return out, l

    def want(self, mask=None, unseen=None):
        parts, lo = [], 0
        for b, f in enumerate(self.fresh):
            c = int(self.cached[b])
            vis = torch.ones((f, c + f), dtype=torch.bool, device=DEV)
            vis[:, c:] = torch.ones((f, f), dtype=torch.bool, device=DEV).tril() if mask is None \
                else ref.words_to_visible(mask[lo:lo + f], f)
            if unseen is not None:
                vis &= ~unseen[b][None, :c + f]
            parts.append(ref.attend(self.q[lo:lo + f], *self.rows[b], vis, self.d ** -0.5))
            lo += f
        return [torch.cat([p[i] for p in parts]) for i in range(4)]


def random_words(fresh, seed, empty=False):
    """Random ancestor-like words: bits up to the row's own, every 5th row empty."""
    rng = np.random.default_rng(seed)
    out = []
    for f in fresh:
        for i in range(f):
            w = int(rng.integers(0, 2 ** 63)) & ((1 << min(i + 1, 64)) - 1)
            w |= 1 << i if i < 64 and not empty else 0
            out.append(0 if empty and i % 5 == 0 else (w - 2 ** 64 if w >= 2 ** 63 else w))
    return torch.tensor(out, dtype=torch.int64, device=DEV)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("hk,g,d,page,cached,fresh", [
    (1, 1, 64, 16, [0], [1]), (2, 4, 128, 16, [5, 0, 16, 31], [1, 1, 1, 1]), (8, 8, 64, 32, [1000, 63, 64, 65], [1, 1, 1, 1]),
    (2, 3, 128, 64, [127, 128, 129, 3000], [8, 5, 1, 3]), (1, 16, 128, 16, [500], [8]), (1, 128, 64, 16, [40, 7], [3, 1]),
    (4, 8, 128, 128, [900, 17, 0], [64, 33, 64]), (2, 5, 64, 128, [4096, 1], [7, 64]), (1, 4, 128, 32, [20000], [1]),
    (3, 1, 128, 64, [255, 256, 257], [64, 2, 30]), (2, 12, 64, 16, [77, 300], [0, 11]),
])
def test_tree_parity(dt, hk, g, d, page, cached, fresh):
    c = Cache(hk * g, hk, d, page, TYPES[dt], cached, fresh, seed=hk + g + d)
    ref.check(*c.run(), c.want(), "causal")
    for empty in (False, True):
        mask = random_words(fresh, 3, empty)
        ref.check(*c.run(mask), c.want(mask), f"masked, empty {empty}")


@pytest.mark.parametrize("d,page", [(64, 16), (128, 128)])
def test_tree_continues_a_prompt(d, page):
    """More than 64 fresh rows without a mask: the next part of a prompt."""
    c = Cache(6, 2, d, page, torch.bfloat16, [300, 0, 41], [200, 129, 1], seed=5)
    ref.check(*c.run(), c.want())


def test_tree_rows_past_the_64th_are_seen_by_none():
    c = Cache(4, 2, 64, 16, torch.bfloat16, [20], [70], seed=6)
    mask = random_words([70], 4)
    mask[64:] = -1
    ref.check(*c.run(mask), c.want(mask))


def test_tree_nothing_cached_and_empty_words():
    c = Cache(8, 2, 128, 16, torch.bfloat16, [0, 0], [4, 9], seed=7)
    out, lse = c.run(torch.zeros(13, dtype=torch.int64, device=DEV))
    assert (out == 0).all() and (lse == -math.inf).all()


@pytest.mark.parametrize("entry", [-1, 10 ** 6])
@pytest.mark.parametrize("fresh", [[1, 3], [40, 64]])
def test_tree_table_entries_out_of_range_are_not_seen(entry, fresh):
    page, cached = 16, [70, 200]
    c = Cache(8, 2, 128, page, torch.bfloat16, cached, fresh, seed=8)
    c.table[0, 1] = entry
    c.table[1, 0] = entry
    c.table[1, 9] = entry
    unseen = []
    for b in range(2):
        p = torch.arange(cached[b] + fresh[b], device=DEV) // page
        unseen.append(p == 1 if b == 0 else (p == 0) | (p == 9))
    ref.check(*c.run(), c.want(unseen=unseen))


@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_tree_unseen_drafted_rows_have_no_effect(bad):
    """Row 2 of the tree is poisoned: rows that do not descend from it stay exact."""
    fresh = [7, 40]
    c = Cache(8, 1, 128, 64, torch.float16, [130, 50], fresh, seed=9)
    words = random_words(fresh, 5)
    words &= ~4
    lo = 0
    for b, f in enumerate(fresh):
        p = int(c.cached[b]) + 2
        pg, at = int(c.table[b, p // 64]), p % 64
        c.k[pg, :, at] = bad
        c.v[pg, :, at] = bad
        words[lo + 5] |= 4
        lo += f
    out, _ = c.run(words)
    want = c.want(words)
    sees = ((words >> 2) & 1).bool()
    ref.check(out[~sees], None, [w[~sees] for w in want])
    assert torch.isnan(out[sees].float()).all()


def test_tree_strides_and_untouched_rows():
    c = Cache(6, 3, 64, 32, torch.bfloat16, [33, 500], [2, 8], seed=10)
    T, hq, d = c.q.shape
    wide = torch.full((hq, T + 5, 2 * d), 9.0, dtype=c.dt, device=DEV)
    q = torch.full((T + 5, 2 * hq, d), math.nan, dtype=c.dt, device=DEV)
    q[:T, ::2] = c.q
    o = wide[:, :, d:].transpose(0, 1)
    moe.moe_attn_tree(c.attn, q[:, ::2], c.cu, c.cached, c.table, c.k, c.v, o, moe.alloc_attn_workspace(c.attn, 2, T + 5))
    torch.cuda.synchronize()
    ref.check(o[:T], None, c.want())
    assert (o[T:] == 9.0).all() and (wide[:, :, :d] == 9.0).all()


def test_tree_offsets_past_32_bits():
    """Pages at the end of a cache of 2^32 + elements."""
    hk, d, page, dt = 4, 128, 128, torch.bfloat16
    pool = 2 ** 32 // (hk * d * page) + 8
    attn = moe.Attention(16, hk, d, page, pool, 4, dt)
    kc, vc = (torch.empty((pool, hk, page, d), dtype=dt, device=DEV) for _ in range(2))
    n, c = 300, 296
    pages = [pool - 1, 2, pool - 5]
    table = ints(pages + [-1]).view(1, 4)
    k, v = randn((n, hk, d), dt, 40), randn((n, hk, d), dt, 41)
    p = torch.arange(n, device=DEV)
    pg = table[0, p // page].long()
    slots = (pg * page + p % page).int()
    moe.moe_kv_append(attn, k, v, slots, kc, vc)
    q = randn((n - c, 16, d), dt, 42)
    out = torch.empty_like(q)
    moe.moe_attn_tree(attn, q, ints([0, n - c]), ints([c]), table, kc, vc, out, moe.alloc_attn_workspace(attn, 1, n - c))
    torch.cuda.synchronize()
    vis = torch.ones((n, n), dtype=torch.bool, device=DEV).tril()[c:]
    ref.check(out, None, ref.attend(q, k, v, vis, d ** -0.5))


def test_tree_and_prompt_repeat_bitwise():
    c = Cache(16, 2, 128, 32, torch.bfloat16, [5000, 30, 1200], [8, 64, 1], seed=11)
    a, b = c.run(), c.run()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    attn = moe.Attention(8, 2, 128, 16, 1, 1)
    q, k, v = randn((900, 8, 128), torch.bfloat16, 1), randn((900, 2, 128), torch.bfloat16, 2), randn((900, 2, 128), torch.bfloat16, 3)
    a, b = run_prompt(attn, q, k, v, [700, 200]), run_prompt(attn, q, k, v, [700, 200])
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_tree_in_a_graph_follows_its_lengths():
    """A captured step, replayed after the lengths on the device have changed (and on another stream)."""
    c = Cache(8, 2, 128, 16, torch.bfloat16, [700, 90], [1, 1], seed=12)
    ws = moe.alloc_attn_workspace(c.attn, 2, 2)
    out = torch.empty_like(c.q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            moe.moe_attn_tree(c.attn, c.q, c.cu, c.cached, c.table, c.k, c.v, out, ws)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            moe.moe_attn_tree(c.attn, c.q, c.cu, c.cached, c.table, c.k, c.v, out, ws)
        g.replay()
    side.synchronize()
    ref.check(out, None, c.want())
    c.cached.copy_(ints([10, 33]))
    c.rows = [[x[:n] for x in kv] for kv, n in zip(c.rows, (11, 34))]
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    ref.check(out, None, c.want())


# ---------------------------------------------------------------- plan and append

def run_plan(attn, cached, fresh, free, table, T, parents=None, info=None):
    i32 = torch.int32
    t = {"table": ints(table).view(len(cached), attn.cfg.max_pages), "cu": torch.full((len(cached) + 1,), -7, dtype=i32, device=DEV),
         "slots": torch.full((T,), -7, dtype=i32, device=DEV), "positions": torch.full((T,), -7, dtype=i32, device=DEV),
         "words": torch.full((T,), -7, dtype=torch.int64, device=DEV) if parents is not None else None,
         "info": torch.zeros(4, dtype=i32, device=DEV) if info is None else info}
    moe.moe_kv_plan(attn, ints(cached), ints(fresh), ints(free), t["table"], t["cu"], t["slots"], t["positions"], t["info"],
                    parents=None if parents is None else ints(parents), tree_mask=t["words"])
    torch.cuda.synchronize()
    return [None if x is None else x.cpu().numpy() for x in t.values()]


def compare_plan(got, want):
    for name, a, b in zip(("table", "cu", "slots", "positions", "words", "info"), got, want):
        if a is not None:
            np.testing.assert_array_equal(a, b, err_msg=name)


def plan_case(seed, B, page, longest, tree, free_short=0):
    rng = np.random.default_rng(seed)
    cached = rng.integers(0, longest, B)
    fresh = rng.integers(0, 65 if tree else longest, B)
    cached[rng.random(B) < 0.2] = 0
    fresh[rng.random(B) < 0.2] = 0
    need, have = -(-(cached + fresh) // page), -(-cached // page)
    width = int(need.max()) + 1
    pool = int(need.sum()) + 2
    order = rng.permutation(pool)
    table = np.full((B, width), -1, np.int64)
    at = 0
    for b in range(B):
        table[b, :have[b]] = order[at:at + have[b]]
        at += have[b]
    T = int(fresh.sum()) + int(rng.integers(0, 9))
    parents = None
    if tree:
        parents = np.concatenate([[int(rng.integers(-1, i)) if i else -1 for i in range(f)] for f in fresh] + [[0] * (T - fresh.sum())])
    return cached, fresh, order[at:pool - free_short], table, T, parents, pool, width


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("B,page,longest", [(1, 16, 40), (7, 16, 300), (33, 32, 90), (257, 64, 500), (1024, 128, 200)])
def test_plan_parity(B, page, longest, tree):
    cached, fresh, free, table, T, parents, pool, width = plan_case(B + page, B, page, longest, tree)
    attn = moe.Attention(1, 1, 64, page, pool, width)
    lists = [x.tolist() for x in (cached, fresh, free, table)]
    got = run_plan(attn, *lists, T, None if parents is None else parents.astype(int).tolist())
    compare_plan(got, ref.plan(cached, fresh, free, table, page, pool, T, parents))
    used = got[5][1]
    s = got[2][got[2] >= 0]
    assert len(set(s.tolist())) == len(s) == int(fresh.sum()), "slots are distinct"
    assert used == int((-(-(cached + fresh) // page) - -(-cached // page)).sum())


def test_plan_deep_chain():
    """A chain of 64 drafted rows: the longest walk."""
    attn = moe.Attention(1, 1, 64, 16, 64, 16)
    args = ([3, 0], [64, 64], list(range(20)), [[50] + [-1] * 15, [-1] * 16], 130, list(range(-1, 63)) * 2 + [5, -1])
    compare_plan(run_plan(attn, *args), ref.plan(*args[:3], np.array(args[3]), 16, 64, 130, args[5]))


@pytest.mark.parametrize("what,flag", [("free", 4), ("page", 4), ("table", 2), ("rows", 1), ("negative", 1), ("parent", 8), ("wide", 8),
                                       ("held", 4)])
def test_plan_flags(what, flag):
    cached, fresh, free, T, parents = [20, 40, 0], [5, 30, 17], [9, 8, 7, 6, 5], 60, None
    table = [[0, 1, -1, -1, -1], [2, 3, 4, -1, -1], [-1] * 5]
    if what == "free":
        free = free[:2]
    elif what == "page":
        free[1] = 10
    elif what == "table":
        fresh[1] = 45
        free = list(range(5, 10)) + [0]
        T = 70
    elif what == "rows":
        T = 40
    elif what == "negative":
        cached[0] = -3
        fresh[2] = -1
    elif what == "parent":
        parents = [-1] * T
        parents[7], parents[10], parents[20] = 2, 5, -9
    elif what == "wide":
        fresh, T = [5, 3, 70], 80
        parents = [-1] * T
        free = [9, 8, 7, 6, 5, 5]
    elif what == "held":
        table[1][2] = 77
    attn = moe.Attention(1, 1, 64, 16, 10, 5)
    info = torch.zeros(4, dtype=torch.int32, device=DEV)
    got = run_plan(attn, cached, fresh, free, table, T, parents, info)
    want = ref.plan(cached, fresh, free, np.array(table), 16, 10, T, parents)
    compare_plan(got, want)
    assert got[5][3] == flag
    again = run_plan(attn, [1], [1], [], [[0] + [-1] * 4], 1, None, info)     # the bits stay
    assert again[5][3] == flag


def test_plan_without_requests_or_rows():
    attn = moe.Attention(1, 1, 64, 16, 10, 5)
    i32 = torch.int32
    e = torch.empty(0, dtype=i32, device=DEV)
    cu, info = torch.full((1,), -7, dtype=i32, device=DEV), torch.zeros(4, dtype=i32, device=DEV)
    slots, pos = torch.full((9,), -7, dtype=i32, device=DEV), torch.full((9,), -7, dtype=i32, device=DEV)
    moe.moe_kv_plan(attn, e, e, e, torch.empty((0, 5), dtype=i32, device=DEV), cu, slots, pos, info)
    assert cu.tolist() == [0] and (slots == -1).all() and (pos == -1).all() and info.tolist() == [0, 0, 0, 0]
    moe.moe_kv_plan(attn, ints([17]), ints([0]), ints([3]), ints([[1, 2, -1, -1, -1]]), torch.empty(2, dtype=i32, device=DEV),
                    e, e, info)
    assert info.tolist() == [0, 0, 17, 0]


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("rows,hk,d,page,order", [(1, 1, 64, 16, "plain"), (57, 8, 128, 16, "fused"), (300, 3, 64, 128, "heads"),
                                                  (5000, 2, 128, 32, "fused"), (17, 5, 128, 64, "gaps")])
def test_append_parity(dt, rows, hk, d, page, order):
    dt = TYPES[dt]
    pool = -(-rows // page) + 3
    attn = moe.Attention(hk, hk, d, page, pool, 1, dt)
    if order == "fused":
        x = randn((rows, 3 * hk * d), dt, 1)
        k, v = x[:, hk * d:2 * hk * d].view(rows, hk, d), x[:, 2 * hk * d:].view(rows, hk, d)
    elif order == "heads":
        k, v = (randn((hk, rows, d), dt, i).transpose(0, 1) for i in (1, 2))
    elif order == "gaps":
        k, v = (randn((3 * rows, hk + 1, d + 8), dt, i)[::3, 1:, 8:] for i in (1, 2))
    else:
        k, v = (randn((rows, hk, d), dt, i) for i in (1, 2))
    g = gen(3)
    slots = torch.randperm(pool * page, generator=g, device=DEV)[:rows].int()
    slots[::7] = -1
    if rows > 3:
        slots[2], slots[3] = pool * page, 2 ** 31 - 1            # out of range: skipped
    kc, vc = (torch.full((pool, hk, page, d), 5.0, dtype=dt, device=DEV) for _ in range(2))
    want = [c.clone() for c in (kc, vc)]
    for i, s in enumerate(slots.tolist()):
        if 0 <= s < pool * page:
            want[0][s // page, :, s % page] = k[i]
            want[1][s // page, :, s % page] = v[i]
    moe.moe_kv_append(attn, k, v, slots, kc, vc)
    torch.cuda.synchronize()
    assert torch.equal(kc, want[0]) and torch.equal(vc, want[1])


# ---------------------------------------------------------------- together

def test_prompt_then_trees_equal_the_whole_sequence():
    """Prompts are admitted, then three verify steps with trees: the rows of
    every step equal attention over the accepted sequence and the path."""
    hq, hk, d, page, dt, B = 8, 2, 128, 16, torch.bfloat16, 3
    pool, width = 40, 12
    attn = moe.Attention(hq, hk, d, page, pool, width, dt)
    kc, vc = (torch.full((pool, hk, page, d), math.nan, dtype=dt, device=DEV) for _ in range(2))
    table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    rng = np.random.default_rng(1)
    free = ints(rng.permutation(pool).tolist())
    cached, fresh = [0] * B, [37, 64, 5]
    seq = [[torch.empty((0, hk, d), dtype=dt, device=DEV)] * 2 for _ in range(B)]
    for step in range(4):
        T = sum(fresh) + 3
        parents = None
        if step:
            parents = np.concatenate([[int(rng.integers(-1, i)) if i else -1 for i in range(f)] for f in fresh] + [[-1] * 3]).astype(int).tolist()
        cu, info = torch.empty(B + 1, dtype=torch.int32, device=DEV), torch.zeros(4, dtype=torch.int32, device=DEV)
        slots, pos = (torch.empty(T, dtype=torch.int32, device=DEV) for _ in range(2))
        words = torch.empty(T, dtype=torch.int64, device=DEV) if step else None
        moe.moe_kv_plan(attn, ints(cached), ints(fresh), free, table, cu, slots, pos, info,
                        parents=ints(parents) if step else None, tree_mask=words)
        q, k, v = (randn((T, h, d), dt, 100 * step + i) for i, h in enumerate((hq, hk, hk)))
        moe.moe_kv_append(attn, k, v, slots, kc, vc)
        out = torch.empty_like(q)
        ws = moe.alloc_attn_workspace(attn, B, T)
        if step == 0:
            moe.moe_attn_prompt(attn, q, k, v, cu, out, ws)
        else:
            moe.moe_attn_tree(attn, q, cu, ints(cached), table, kc, vc, out, ws, tree_mask=words)
        torch.cuda.synchronize()
        assert info.tolist()[3] == 0
        free = free[int(info[1]):]
        keep = torch.full((T,), -1, dtype=torch.int32, device=DEV)
        lo = 0
        for b, f in enumerate(fresh):
            paths = []
            for i in range(f):
                path, j = [i], (parents[lo + i] if step else i - 1)
                while j >= 0:
                    path.append(j)
                    j = parents[lo + j] if step else j - 1
                path = path[::-1]
                paths.append(path)
                if not step and i != f - 1:
                    continue
                rows = torch.tensor(path, device=DEV) + lo
                kk, vv = torch.cat([seq[b][0], k[rows]]), torch.cat([seq[b][1], v[rows]])
                vis = torch.ones((1, kk.shape[0]), dtype=torch.bool, device=DEV)
                ref.check(out[lo + i:lo + i + 1], None, ref.attend(q[lo + i:lo + i + 1], kk, vv, vis, d ** -0.5), f"step {step} row {i}")
            best = max(paths, key=len)                             # the accepted path; its rows move to their final slots
            rows = torch.tensor(best, device=DEV) + lo
            for n, r in enumerate(best):
                keep[lo + r] = slots[lo + n]
            seq[b] = [torch.cat([seq[b][0], k[rows]]), torch.cat([seq[b][1], v[rows]])]
            lo += f
            cached[b] += len(best)
        if step:
            moe.moe_kv_append(attn, k, v, keep, kc, vc)
        # pages of rejected rows stay in the table and go back to the free list's front
        for b in range(B):
            have, held = -(-cached[b] // page), int((table[b] >= 0).sum())
            if held > have:
                free = torch.cat([table[b, have:held], free])
                table[b, have:held] = -1
        fresh = [int(x) for x in rng.integers(1, 9, B)]


# ---------------------------------------------------------------- refusals

def test_refusals():
    dt = torch.bfloat16
    attn = moe.Attention(4, 2, 64, 16, 8, 4, dt)
    q, k = randn((6, 4, 64), dt, 1), randn((6, 2, 64), dt, 2)
    out, ws, cu = torch.empty_like(q), moe.alloc_attn_workspace(attn, 1, 6), ints([0, 6])
    cache, table, slots = torch.zeros((8, 2, 16, 64), dtype=dt, device=DEV), ints([[0, 1, 2, 3]]), ints([0, 1, 2, 3, 4, 5])

    def status(fn, *a, **kw):
        with pytest.raises(moe.MoEError) as e:
            fn(*a, **kw)
        return e.value.status
    with pytest.raises(TypeError):
        moe.moe_attn_prompt(attn, q.half(), k, k, cu, out, ws)
    with pytest.raises(ValueError):
        moe.moe_attn_prompt(attn, q, k[:5], k, cu, out, ws)
    with pytest.raises(ValueError):
        moe.moe_attn_prompt(attn, q.transpose(1, 2).contiguous().transpose(1, 2), k, k, cu, out, ws)
    with pytest.raises(ValueError):
        moe.moe_attn_tree(attn, q, cu, ints([1, 2]), table, cache, cache, out, ws)
    with pytest.raises(ValueError):
        moe.moe_attn_tree(attn, q, cu, ints([1]), table, cache[:7], cache, out, ws)
    with pytest.raises(TypeError):
        moe.moe_kv_append(attn, k, k, slots.long(), cache, cache)
    with pytest.raises(ValueError):
        moe.moe_kv_append(attn, k.cpu(), k, slots, cache, cache)
    odd = torch.zeros(6 * 4 * 64 + 8, dtype=dt, device=DEV)
    assert status(moe.moe_attn_prompt, attn, odd[1:6 * 4 * 64 + 1].view(6, 4, 64), k, k, cu, out, ws) == 1       # misaligned
    assert status(moe.moe_attn_prompt, attn, q, k[:, :1].expand(6, 2, 64), k, cu, out, ws) == 1                  # stride 0
    narrow = torch.zeros((6, 2, 68), dtype=dt, device=DEV)[:, :, :64]
    assert status(moe.moe_kv_append, attn, narrow, k, slots, cache, cache) == 1                                  # stride of 68
    assert status(moe.moe_attn_prompt, attn, q, k, k, cu, out, ws[:128]) == 4
    assert status(moe.moe_attn_tree, attn, q, cu, ints([1]), table, cache, cache, out, ws[:128]) == 4
    big = torch.zeros(1026, dtype=torch.int32, device=DEV)
    assert status(moe.moe_attn_prompt, attn, q, k, k, big, out, ws) == 2                                         # 1025 requests
    i = torch.zeros(6, dtype=torch.int32, device=DEV)
    word = torch.zeros(6, dtype=torch.int64, device=DEV)
    info = torch.zeros(4, dtype=torch.int32, device=DEV)
    assert status(moe.moe_kv_plan, attn, ints([1]), ints([1]), slots, table, cu.clone(), i, i.clone(), info, tree_mask=word) == 1
    moe.moe_attn_prompt(attn, q[:0], k[:0], k[:0], cu[:1].contiguous(), out[:0], ws)                             # nothing to do
    moe.moe_attn_tree(attn, q[:0], ints([0, 0]), ints([7]), table, cache, cache, out[:0], ws)
    moe.moe_kv_append(attn, k[:0], k[:0], slots[:0], cache, cache)
    torch.cuda.synchronize()
    assert (cache == 0).all()


def test_example_runs_the_operators_together():
    """The serving loop around the MoE layer: stepwise, paged attention equals the whole sequences'.  Both sides round
    P and the result to bf16: 2 (u A + u |o|) on each, with A at most max |v| and v of unit variance."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "paged_step.py")
    spec = importlib.util.spec_from_file_location("paged_step", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    off, largest = example.main(4)
    assert largest > 0.1
    assert off <= 4 * 2 * 2.0 ** -8 * 5.0
