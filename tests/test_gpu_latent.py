"""Latent attention over the paged cache on the GPU against its definition in 64
bits (``latent_ref``)."""
import math

import numpy as np
import pytest
import torch

import attn_ref
import latent_ref as ref
from quantized_moe_expert_router_gb300 import moe
from test_gpu_attn import ints, offsets, randn, random_words

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
SCALE = 192 ** -0.5


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_moe_expert_router_gb300 import build
    build.build()
    moe.load_library()


class Latent:
    """Requests of `cached` tokens and `fresh` rows over a shuffled pool whose unused places hold NaN."""

    def __init__(self, heads, page, dt, cached, fresh, seed, extra_pages=3):
        self.lat, self.dt, self.page, self.heads = None, dt, page, heads
        B = len(cached)
        need = [-(-(c + f) // page) for c, f in zip(cached, fresh)]
        pool, width = sum(need) + extra_pages, max(max(need), 1) + 1
        order = np.random.default_rng(seed).permutation(pool)
        table = np.full((B, width), -1, np.int32)
        self.cache = torch.full((pool, page, 576), math.nan, dtype=dt, device=DEV)
        self.tokens, at = [], 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            at += n
            x = randn((cached[b] + fresh[b], 576), dt, seed + 7 * b + 1)
            self.tokens.append(x)
            p = torch.arange(x.shape[0], device=DEV)
            pages = torch.from_numpy(table[b].astype(np.int64)).to(DEV)[p // page]
            self.cache[pages, p % page] = x
        self.table, self.cached, self.cu = torch.from_numpy(table).to(DEV), ints(cached), offsets(fresh)
        self.fresh, T = fresh, sum(fresh)
        self.q = randn((T, heads, 576), dt, seed + 1000)
        self.lat = moe.LatentAttention(heads, page, pool, width, dt)

    def run(self, mask=None, ws=None, out=None, lse=True):
        T = self.q.shape[0]
        out = torch.empty((T, self.heads, 512), dtype=self.dt, device=DEV) if out is None else out
        lse = torch.empty((T, self.heads), dtype=torch.float32, device=DEV) if lse else None
        ws = moe.alloc_latent_workspace(self.lat, len(self.fresh), T) if ws is None else ws
        moe.moe_latent_tree(self.lat, self.q[:, :, :512], self.q[:, :, 512:], self.cu, self.cached, self.table, self.cache, out, ws,
                            tree_mask=mask, lse=lse)
        assert moe.moe_latent_get_device_status(self.lat, ws) == 0
        return out, lse

    def visible(self, b, mask, lo):
        f, c = self.fresh[b], int(self.cached[b])
        vis = torch.ones((f, c + f), dtype=torch.bool, device=DEV)
        vis[:, c:] = torch.ones((f, f), dtype=torch.bool, device=DEV).tril() if mask is None else attn_ref.words_to_visible(mask[lo:lo + f], f)
        return vis

    def want(self, mask=None, unseen=None):
        parts, lo = [], 0
        for b, f in enumerate(self.fresh):
            vis = self.visible(b, mask, lo)
            if unseen is not None:
                vis &= ~unseen[b][None]
            x = self.tokens[b][:, None]
            parts.append(ref.attend(self.q[lo:lo + f], x, x[:, :, :512], vis, SCALE))
            lo += f
        return [torch.cat([p[i] for p in parts]) for i in range(4)]


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("heads,page,cached,fresh", [
    (1, 16, [0], [1]), (16, 16, [5], [1]), (16, 16, [127, 128, 129, 0], [1, 1, 1, 1]), (32, 64, [1000, 63, 64, 65], [1, 1, 1, 1]),
    (64, 32, [300], [1]), (64, 64, [1000, 2000], [1, 1]), (128, 64, [1500, 3], [1, 1]), (128, 128, [129], [3]), (5, 16, [500, 12], [8, 3]),
    (16, 128, [900, 17, 0], [64, 33, 64]), (97, 32, [70, 200], [2, 5]), (40, 64, [4096, 1], [7, 30]), (3, 128, [255, 256, 257], [64, 2, 30]),
    (12, 16, [77, 300], [0, 11]), (20, 32, [20000], [1]), (64, 16, [9000], [4]),
])
def test_tree_parity(dt, heads, page, cached, fresh):
    c = Latent(heads, page, TYPES[dt], cached, fresh, seed=heads + page)
    attn_ref.check(*c.run(), c.want(), "causal")
    for empty in (False, True):
        mask = random_words(fresh, 3, empty)
        attn_ref.check(*c.run(mask), c.want(mask), f"masked, empty {empty}")


@pytest.mark.parametrize("heads,page", [(8, 16), (64, 128), (128, 64)])
def test_tree_continues_a_prompt(heads, page):
    """More than 64 fresh rows without a mask: the next part of a prompt."""
    c = Latent(heads, page, torch.bfloat16, [300, 0, 41], [200, 129, 1], seed=5)
    attn_ref.check(*c.run(), c.want())


def test_tree_many_requests():
    """Requests of every kind by the hundred: items of a CTA follow one another, some requests are empty."""
    cached, fresh = [(37 * i) % 411 for i in range(700)], [(5 * i) % 3 for i in range(700)]
    c = Latent(16, 32, torch.bfloat16, cached, fresh, seed=21)
    attn_ref.check(*c.run(), c.want())


def test_tree_long_and_short():
    c = Latent(64, 64, torch.bfloat16, [30000, 10, 700, 128, 5000], [1, 2, 1, 3, 1], seed=22)
    attn_ref.check(*c.run(), c.want())


def test_tree_rows_past_the_64th_are_seen_by_none():
    c = Latent(4, 16, torch.bfloat16, [20], [70], seed=6)
    mask = random_words([70], 4)
    mask[64:] = -1
    attn_ref.check(*c.run(mask), c.want(mask))


def test_tree_nothing_cached_and_empty_words():
    c = Latent(8, 16, torch.bfloat16, [0, 0], [4, 9], seed=7)
    out, lse = c.run(torch.zeros(13, dtype=torch.int64, device=DEV))
    assert (out == 0).all() and (lse == -math.inf).all()


@pytest.mark.parametrize("entry", [-1, 10 ** 6])
@pytest.mark.parametrize("fresh", [[1, 3], [40, 64]])
def test_tree_table_entries_out_of_range_are_not_seen(entry, fresh):
    page, cached = 16, [70, 200]
    c = Latent(8, page, torch.bfloat16, cached, fresh, seed=8)
    c.table[0, 1] = entry
    c.table[1, 0] = entry
    c.table[1, 9] = entry
    unseen = []
    for b in range(2):
        p = torch.arange(cached[b] + fresh[b], device=DEV) // page
        unseen.append(p == 1 if b == 0 else (p == 0) | (p == 9))
    attn_ref.check(*c.run(), c.want(unseen=unseen))


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_tree_unseen_drafted_rows_have_no_effect(dt, bad):
    """Row 2 of the tree is poisoned: rows that do not descend from it stay exact."""
    fresh = [7, 40]
    c = Latent(16, 64, TYPES[dt], [130, 50], fresh, seed=9)
    words = random_words(fresh, 5)
    words &= ~4
    lo = 0
    for b, f in enumerate(fresh):
        p = int(c.cached[b]) + 2
        c.cache[int(c.table[b, p // 64]), p % 64] = bad
        words[lo + 5] |= 4
        lo += f
    out, _ = c.run(words)
    want = c.want(words)
    sees = ((words >> 2) & 1).bool()
    attn_ref.check(out[~sees], None, [w[~sees] for w in want])
    assert torch.isnan(out[sees].float()).all()


@pytest.mark.parametrize("fresh", [[3], [1]])
def test_tree_a_bad_element_of_a_hidden_key(fresh):
    """One element of a latent is infinite, and the scores of the rows that see it -infinite: it has no weight, and
    this element of their output alone is NaN."""
    c = Latent(16, 16, torch.bfloat16, [20], fresh, seed=23)
    place = 20 if fresh[0] > 1 else 5
    c.q[:, :, 300] = -1.0
    c.cache[int(c.table[0, place // 16]), place % 16, 300] = math.inf
    c.tokens[0][place, 300] = 0.0
    mask = random_words(fresh, 5) if fresh[0] > 1 else None
    if mask is not None:
        mask[0], mask[1], mask[2] = 1, 2, 7            # rows 0 and 2 see the first fresh token
    out, _ = c.run(mask)
    rows = [0, 2] if mask is not None else [0]
    assert torch.isnan(out[rows][:, :, 300].float()).all()
    others = torch.arange(512, device=DEV) != 300
    blind = torch.zeros(20 + fresh[0], dtype=torch.bool, device=DEV)
    blind[place] = True
    want, seen = c.want(mask, unseen=[blind]), c.want(mask)
    for r in range(fresh[0]):
        w = want if r in rows else seen
        got = out[r][:, others] if r in rows else out[r]
        attn_ref.check(got, None, [w[0][r][:, others] if r in rows else w[0][r], None, w[2][r][:, others] if r in rows else w[2][r], None])


def test_tree_strides_and_untouched_rows():
    c = Latent(6, 32, torch.bfloat16, [33, 500], [2, 8], seed=10)
    T = 10
    wide = torch.full((6, T + 5, 1024), 9.0, dtype=c.dt, device=DEV)
    q = torch.full((T + 5, 12, 512), math.nan, dtype=c.dt, device=DEV)
    r = torch.full((6, T + 5, 192), math.nan, dtype=c.dt, device=DEV)
    q[:T, ::2], r[:, :T, 128:] = c.q[:, :, :512], c.q[:, :, 512:].transpose(0, 1)
    o = wide[:, :, 512:].transpose(0, 1)
    moe.moe_latent_tree(c.lat, q[:, ::2], r[:, :, 128:].transpose(0, 1), c.cu, c.cached, c.table, c.cache, o,
                        moe.alloc_latent_workspace(c.lat, 2, T + 5))
    torch.cuda.synchronize()
    attn_ref.check(o[:T], None, c.want())
    assert (o[T:] == 9.0).all() and (wide[:, :, :512] == 9.0).all()


def test_tree_offsets_past_32_bits():
    """Pages at the end of a cache of 2^32 + elements."""
    page, dt = 128, torch.bfloat16
    pool = 2 ** 32 // (576 * page) + 8
    lat = moe.LatentAttention(16, page, pool, 4, dt)
    cache = torch.empty(lat.cache_shape, dtype=dt, device=DEV)
    n, c = 300, 296
    table = ints([pool - 1, 2, pool - 5, -1]).view(1, 4)
    x = randn((n, 576), dt, 40)
    p = torch.arange(n, device=DEV)
    slots = (table[0, p // page].long() * page + p % page).int()
    rope = moe.Rope(64)
    moe.moe_latent_append(lat, rope, x[:, :512], x[:, 512:], torch.zeros_like(slots), slots, cache)
    q = randn((n - c, 16, 576), dt, 42)
    out = torch.empty((n - c, 16, 512), dtype=dt, device=DEV)
    moe.moe_latent_tree(lat, q[:, :, :512], q[:, :, 512:], ints([0, n - c]), ints([c]), table, cache, out,
                        moe.alloc_latent_workspace(lat, 1, n - c))
    vis = torch.ones((n, n), dtype=torch.bool, device=DEV).tril()[c:]
    attn_ref.check(out, None, ref.attend(q, x[:, None], x[:, None, :512], vis, SCALE))


@pytest.mark.parametrize("n", [40, 20000])
def test_tree_scores_of_minus_infinity(n):
    """Tokens whose infinite element gives a score of -infinity, whole parts of a context among them: no weight, and a NaN there."""
    c = Latent(16, 16, torch.bfloat16, [n], [1], seed=35)
    c.q[:, :, 7] = 1.0
    unseen = torch.arange(n + 1, device=DEV) < n // 2
    p = torch.arange(n // 2, device=DEV)
    c.cache[c.table[0].long()[p // 16], p % 16, 7] = -math.inf
    want = c.want(unseen=[unseen])
    out, lse = c.run()
    assert out[:, :, 7].isnan().all()
    out[:, :, 7] = want[0][:, :, 7].to(out.dtype)
    attn_ref.check(out, lse, want)
    c.cache[..., 7] = -math.inf                                     # no token is left
    out, lse = c.run()
    assert out[:, :, 7].isnan().all() and (out.nan_to_num() == 0).all() and (lse == -math.inf).all()


def test_tree_large_scores():
    """Scores of hundreds: the maximum moves many times, and weights underflow."""
    c = Latent(16, 16, torch.bfloat16, [2000], [2], seed=24)
    c.q *= 30.0
    attn_ref.check(*c.run(), c.want())


def test_tree_scores_far_below_zero():
    """Scores of -10^33, thousands of roundings apart: the largest has all the weight."""
    c = Latent(16, 16, torch.bfloat16, [300], [1], seed=34)
    x = (1.0 + torch.rand((301, 576), device=DEV)).mul(1e15).bfloat16()
    x[:, 512:] = 0.0
    p = torch.arange(301, device=DEV)
    c.cache[c.table[0].long()[p // 16], p % 16] = x
    c.q[:] = -1e17
    out, lse = c.run()
    best = x[:, :512].double().sum(1).argmin()
    assert torch.equal(out[0], x[best, :512].expand(16, 512)) and (lse < -1e32).all()


def test_tree_rising_scores():
    """Every tile's maximum passes the last one's: the rescaling runs at each of them, in every row."""
    c = Latent(33, 128, torch.float16, [1500], [1], seed=25)
    n = 1501
    x = c.tokens[0]
    x[:, 512] = torch.linspace(0, 60, n, device=DEV).half()
    p = torch.arange(n, device=DEV)
    c.cache[c.table[0].long()[p // 128], p % 128] = x
    c.q[:, :, 512] = 40.0
    attn_ref.check(*c.run(), c.want())


def test_tree_repeats_bitwise_with_one_workspace():
    c = Latent(64, 32, torch.bfloat16, [5000, 30, 1200], [8, 64, 1], seed=11)
    ws = moe.alloc_latent_workspace(c.lat, 3, 73)
    a = c.run(ws=ws)
    d = Latent(64, 32, torch.bfloat16, [3], [1], seed=12)
    d.run(ws=ws)
    b = c.run(ws=ws)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_tree_in_a_graph_follows_its_lengths():
    """A captured step, replayed after the lengths on the device have changed (and on another stream)."""
    c = Latent(16, 16, torch.bfloat16, [700, 90], [1, 1], seed=12)
    ws = moe.alloc_latent_workspace(c.lat, 2, 2)
    out = torch.empty((2, 16, 512), dtype=c.dt, device=DEV)
    call = lambda: moe.moe_latent_tree(c.lat, c.q[:, :, :512], c.q[:, :, 512:], c.cu, c.cached, c.table, c.cache, out, ws)  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            call()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            call()
        g.replay()
    side.synchronize()
    attn_ref.check(out, None, c.want())
    c.cached.copy_(ints([10, 33]))
    c.tokens = [x[:n] for x, n in zip(c.tokens, (11, 34))]
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    attn_ref.check(out, None, c.want())


def test_lengths_past_the_block_table_are_cut():
    """The context ends with the table: the rest of its third page, which holds NaN, is part of it."""
    c = Latent(4, 16, torch.bfloat16, [40], [1], seed=26)
    c.cached.fill_(2 ** 31 - 1)
    out, _ = c.run()
    assert torch.isnan(out.float()).all()
    c.cache[int(c.table[0, 2]), 9:] = c.cache[int(c.table[0, 2]), 8]
    c.tokens[0] = torch.cat([c.tokens[0], c.tokens[0][40:].expand(7, 576)])
    c.fresh, vis = [1], torch.ones((1, 48), dtype=torch.bool, device=DEV)
    x = c.tokens[0][:, None]
    attn_ref.check(*c.run(), ref.attend(c.q, x, x[:, :, :512], vis, SCALE))


@pytest.mark.parametrize("heads,cached,fresh", [
    (16, [(31 * i) % 250 for i in range(17)], [1] * 17), (64, [(53 * i) % 500 for i in range(70)], [1] * 70),
    (64, [200, 90, 30, 7], [8, 3, 8, 1]), (128, [(17 * i) % 130 for i in range(90)], [1 + i % 3 for i in range(90)]), (5, [70], [20]),
])
def test_items_whole_and_cut(heads, cached, fresh):
    """The table's width decides whether items are cut: the same requests in a table as wide as they need and in a wide one."""
    c = Latent(heads, 16, torch.bfloat16, cached, fresh, seed=30)
    mask = random_words(fresh, 7)
    want = c.want(mask)
    attn_ref.check(*c.run(mask), want, "narrow")
    more = torch.full((len(fresh), 3000), -1, dtype=torch.int32, device=DEV)
    c.table = torch.cat([c.table, more], 1)
    c.lat = moe.LatentAttention(heads, 16, c.cache.shape[0], c.table.shape[1], c.dt)
    attn_ref.check(*c.run(mask), want, "wide")


def test_two_calls_at_once():
    """Two streams, a workspace each: the same bits as one after the other."""
    cs = [Latent(64, 32, torch.bfloat16, [9000, 700], [2, 1], seed=31), Latent(16, 16, torch.bfloat16, [3000] * 20, [1] * 20, seed=32)]
    alone = [c.run() for c in cs]
    streams, outs = [torch.cuda.Stream() for _ in cs], [torch.empty_like(a[0]) for a in alone]
    spaces = [moe.alloc_latent_workspace(c.lat, 20, 20) for c in cs]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, s, o, w in zip(cs, streams, outs, spaces):
            moe.moe_latent_tree(c.lat, c.q[:, :, :512], c.q[:, :, 512:], c.cu, c.cached, c.table, c.cache, o, w, stream=s)
    torch.cuda.synchronize()
    for c, o, a, w in zip(cs, outs, alone, spaces):
        assert torch.equal(o, a[0]) and moe.moe_latent_get_device_status(c.lat, w) == 0


def test_results_follow_the_kernel_before():
    """The call's kernels may start before the kernel ahead of them in the stream ends: they read its results all the same."""
    c = Latent(16, 16, torch.bfloat16, [400, 30], [1, 2], seed=33)
    want, q = c.run()[0], c.q.clone()
    ws, out = moe.alloc_latent_workspace(c.lat, 2, 3), torch.empty((3, 16, 512), dtype=c.dt, device=DEV)
    big = torch.randn((1 << 24,), device=DEV)
    for _ in range(10):
        c.q.zero_()
        big.mul_(1.0)
        c.q.copy_(q)
        moe.moe_latent_tree(c.lat, c.q[:, :, :512], c.q[:, :, 512:], c.cu, c.cached, c.table, c.cache, out, ws)
        got = out.clone()
        assert torch.equal(got, want)


def test_latent_plan_is_the_plan_of_its_pages():
    cached, fresh, parents = [40, 0, 17], [5, 3, 64], [-1, 0, 0, 1, 3, -1, -1, 1] + [i - 1 for i in range(64)]
    lat, attn = moe.LatentAttention(8, 16, 40, 8), moe.Attention(8, 2, 64, 16, 40, 8)
    table = np.full((3, 8), -1, np.int32)
    table[0, :3], table[2, :2] = [3, 1, 2], [9, 4]
    got = []
    for call, handle in ((moe.moe_latent_plan, lat), (moe.moe_kv_plan, attn)):
        t, cu, slots, positions = ints(table.tolist()), ints([0] * 4), ints([-7] * 80), ints([-7] * 80)
        words, info = torch.full((80,), -7, dtype=torch.int64, device=DEV), ints([0] * 4)
        call(handle, ints(cached), ints(fresh), ints(list(range(10, 40))), t, cu, slots, positions, info, parents=ints(parents + [-1] * 8), tree_mask=words)
        got.append([x.cpu().numpy() for x in (t, cu, slots, positions, words, info)])
    want = attn_ref.plan(cached, fresh, list(range(10, 40)), table, 16, 40, 80, parents + [-1] * 8)
    for a, b, w in zip(*got, want):
        np.testing.assert_array_equal(a, w)
        np.testing.assert_array_equal(b, w)


def test_a_wait_that_runs_out_is_reported():
    """Copies that never complete (the handle's test hook): the call ends, the flag is raised once, and the
    workspace works again."""
    c = Latent(16, 16, torch.bfloat16, [300, 20], [2, 1], seed=27)
    ws = moe.alloc_latent_workspace(c.lat, 2, 3)
    stalled = moe.LatentAttention(16, 16, c.cache.shape[0], c.table.shape[1], c.dt, flags=moe.ATTN_TEST_STALL)
    out = torch.empty((3, 16, 512), dtype=c.dt, device=DEV)
    moe.moe_latent_tree(stalled, c.q[:, :, :512], c.q[:, :, 512:], c.cu, c.cached, c.table, c.cache, out, ws)
    assert moe.moe_latent_get_device_status(stalled, ws) == moe.FLAG_TIMEOUT
    assert moe.moe_latent_get_device_status(stalled, ws) == 0
    attn_ref.check(*c.run(ws=ws), c.want())


def test_refusals():
    c = Latent(4, 16, torch.bfloat16, [20], [2], seed=28)
    ws = moe.alloc_latent_workspace(c.lat, 1, 2)
    out = torch.empty((2, 4, 512), dtype=c.dt, device=DEV)
    good = dict(q=c.q[:, :, :512], q_rope=c.q[:, :, 512:], cu=c.cu, cached=c.cached, block_table=c.table, cache=c.cache, out=out, ws=ws)
    moe.moe_latent_tree(c.lat, **good)
    for kind, kw, match in [
            (TypeError, dict(q=good["q"].half()), "q is"), (ValueError, dict(q_rope=c.q[:, :, 500:]), "q_rope of shape"),
            (ValueError, dict(out=out[:1]), "out of shape"), (TypeError, dict(cu=c.cu.long()), "cu is"),
            (ValueError, dict(cached=ints([1, 2])), "cached of shape"), (ValueError, dict(block_table=c.table[:, :1]), "block_table"),
            (TypeError, dict(cache=c.cache.half()), "cache is"), (ValueError, dict(cache=c.cache[:1]), "cache of shape"),
            (ValueError, dict(ws=ws[::2]), "ws with strides"), (TypeError, dict(tree_mask=ints([1, 1])), "tree_mask is"),
            (ValueError, dict(lse=torch.empty((2, 3), device=DEV)), "lse of shape"), (ValueError, dict(q=good["q"].cpu()), "q of shape"),
            (ValueError, dict(ws=ws.cpu()), "ws is on")]:
        with pytest.raises(kind, match=match):
            moe.moe_latent_tree(c.lat, **{**good, **kw})
    with pytest.raises(moe.MoEError) as e:
        moe.moe_latent_tree(c.lat, **{**good, "ws": ws[:1024]})
    assert e.value.status == 4
    with pytest.raises(ValueError, match="not a workspace"):
        moe.moe_latent_get_device_status(c.lat, ws[:1024])
    attn, rope, i32 = moe.Attention(4, 4, 64, 16, 2, 2), moe.Rope(64), torch.zeros(4, dtype=torch.int32, device=DEV)
    for call in (lambda: moe.moe_kv_plan(c.lat, *[i32] * 8), lambda: moe.moe_latent_plan(attn, *[i32] * 8),
                 lambda: moe.moe_attn_get_device_status(c.lat, ws), lambda: moe.moe_latent_get_device_status(attn, ws),
                 lambda: moe.moe_attn_workspace_bytes(c.lat, 1, 1), lambda: moe.moe_latent_workspace_bytes(attn, 1, 1),
                 lambda: moe.moe_rope_apply(attn, i32[:2], out, out), lambda: moe.moe_latent_tree(attn, **good),
                 lambda: moe.moe_latent_append(c.lat, attn, c.q[:, 0, :512], c.q[:, 0, 512:], i32[:2], i32[:2], c.cache),
                 lambda: moe.moe_rope_append(c.lat, rope, out, out, out, i32, i32, out, out, out)):
        with pytest.raises(TypeError, match="not a"):              # another kind of handle
            call()
    none = c.q[:0]
    moe.moe_latent_tree(c.lat, none[:, :, :512], none[:, :, 512:], ints([0, 0]), c.cached, c.table, c.cache, out[:0], ws)
    moe.moe_latent_tree(c.lat, good["q"], good["q_rope"], ints([0]), ints([]), c.table[:0], c.cache, out, ws)
    torch.cuda.synchronize()
