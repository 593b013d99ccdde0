"""The attention calls on the shapes that choose among their kernels (prompts of
many and few row tiles; trees of few items, many items, many rows per request),
against the definition in 64 bits with the
bounds of ``attn_ref``."""
import math

import numpy as np
import pytest
import torch

import attn_ref as ref
from quantized_moe_expert_router_gb300 import moe
from test_gpu_attn import Cache, built, gen, ints, offsets, prompt_ref, randn, random_words, run_prompt  # noqa: F401  (built: the module's build fixture)

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def ragged(n, longest, seed, zeros=0.1):
    rng = np.random.default_rng(seed)
    c = rng.integers(1, longest + 1, n)
    c[rng.random(n) < zeros] = 0
    return c.tolist()


def poison(c, words, row, bad):
    """Makes the drafted row `row` of every request that has it infinite or NaN; only the request's row after it sees it."""
    words, lo, sees = words & ~(1 << row), 0, torch.zeros(c.T, dtype=torch.bool, device=DEV)
    for b, f in enumerate(c.fresh):
        if f > row:
            p = int(c.cached[b]) + row
            pg, at = int(c.table[b, p // c.page]), p % c.page
            c.k[pg, :, at] = bad
            c.v[pg, :, at] = bad
            if f > row + 1:
                words[lo + row + 1] |= 1 << row
                sees[lo + row + 1] = True
        lo += f
    return words, sees


# ---------------------------------------------------------------- prompts of more row tiles than SMs, and of fewer

PROMPTS = [   # kv heads, group, D, lengths
    (40, 1, 64, [129, 1, 0, 513, 300, 64]), (24, 2, 128, [129, 1, 0, 513, 300]), (8, 12, 128, [10, 11, 21, 250]),
    (4, 32, 64, [200, 3, 57]), (2, 128, 128, [33, 90]), (32, 3, 64, [42, 43, 84, 85, 400]),                       # pairs of row tiles
    (1, 1, 64, [128, 129, 256, 257, 900]), (4, 4, 128, [640]), (1, 8, 128, [2000]), (2, 7, 64, [1, 18, 19, 400]),  # single ones
]


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("case", range(len(PROMPTS)))
def test_prompt_items_parity(dt, case):
    hk, g, d, lengths = PROMPTS[case]
    T, dt = sum(lengths), TYPES[dt]
    attn = moe.Attention(hk * g, hk, d, 16, 1, 1, dt)
    for rep in range(2):
        q, k, v = (randn((T, h, d), dt, 300 + 10 * rep + i, 1.5 if i == 0 else 1.0) for i, h in enumerate((hk * g, hk, hk)))
        out, lse = run_prompt(attn, q, k, v, lengths)
        ref.check(out, lse, prompt_ref(q, k, v, lengths, d ** -0.5))
    a = run_prompt(attn, q, k, v, lengths)
    assert torch.equal(a[0], out) and torch.equal(a[1], lse)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("hk,d", [(40, 64), (24, 128), (2, 64), (2, 128)])
def test_prompt_items_unseen_rows(hk, d, bad):
    """Everything from a row of each request on is poisoned: the rows before stay exact."""
    lengths, last, dt = [300, 129, 700], [170, 128, 515], torch.bfloat16
    attn = moe.Attention(2 * hk, hk, d, 16, 1, 1, dt)
    T, cu = sum(lengths), offsets(lengths).tolist()
    q, k, v = (randn((T, h, d), dt, 340 + i) for i, h in enumerate((2 * hk, hk, hk)))
    want = prompt_ref(q, k, v, lengths, d ** -0.5)
    for lo, n, at in zip(cu, lengths, last):
        for x in (q, k, v):
            x[lo + at:lo + n] = bad
    out, _ = run_prompt(attn, q, k, v, lengths)
    for lo, n, at in zip(cu, lengths, last):
        ref.check(out[lo:lo + at], None, [w[lo:lo + at] for w in want])
        assert torch.isnan(out[lo + at:lo + n].float()).all()


@pytest.mark.parametrize("hk,d", [(40, 64), (24, 128), (2, 64), (2, 128)])
@pytest.mark.parametrize("at", [0, 127, 128, 300])
def test_prompt_items_infinite_value_reaches_the_rows_that_see_it(hk, d, at):
    n, dt = 600, torch.float16
    attn = moe.Attention(2 * hk, hk, d, 16, 1, 1, dt)
    q, k, v = (randn((n, h, d), dt, 350 + i) for i, h in enumerate((2 * hk, hk, hk)))
    want = prompt_ref(q, k, v, [n], d ** -0.5)
    v[at, :, 5] = math.inf
    out, _ = run_prompt(attn, q, k, v, [n])
    ref.check(out[:at], None, [w[:at] for w in want])
    assert (out[at:, :, 5] == math.inf).all()
    keep = [e for e in range(d) if e != 5]
    ref.check(out[:, :, keep], None, [want[0][:, :, keep], want[1], want[2][:, :, keep], want[3]])


# ---------------------------------------------------------------- many items: requests x kv heads x row tiles above the SMs

MANY = [   # kv heads, group, D, page, cached, rows of a request
    (8, 1, 64, 16, ragged(24, 500, 1), [1] * 24),
    (8, 4, 128, 16, ragged(24, 500, 2), [1] * 24),
    (8, 8, 128, 64, ragged(21, 300, 3) + [9000], [2] * 22),
    (4, 8, 64, 32, ragged(30, 400, 4), [4] * 30),                        # two row tiles each
    (1, 16, 128, 128, ragged(60, 200, 5), [3] * 60),                     # three
    (16, 1, 64, 16, [0] * 12 + [7000], [1] * 13),                        # nearly everything in one request
    (2, 5, 128, 16, ragged(50, 90, 6), ([7, 0, 3, 1, 12] * 10)),         # requests without rows
]


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("case", range(len(MANY)))
def test_many_items_parity(dt, case):
    hk, g, d, page, cached, fresh = MANY[case]
    c = Cache(hk * g, hk, d, page, TYPES[dt], cached, fresh, seed=70 + case)
    ref.check(*c.run(), c.want(), "causal")
    mask = random_words(fresh, case, True)
    ref.check(*c.run(mask), c.want(mask), "masked, empty rows")


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("d,page,fresh", [(128, 64, [7] * 30), (64, 16, [20, 3] * 20)])
def test_many_items_unseen_drafted_rows(bad, d, page, fresh):
    c = Cache(8, 8 if d == 128 else 4, d, page, torch.float16, ragged(len(fresh), 300, 9), fresh, seed=90)
    words, sees = poison(c, random_words(fresh, 9), 2, bad)
    out, _ = c.run(words)
    want = c.want(words)
    ref.check(out[~sees], None, [w[~sees] for w in want])
    assert sees.any() and torch.isnan(out[sees].float()).all()


@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_many_items_infinite_values_reach_the_rows_that_see_them(bad):
    """Only v is infinite or NaN: a row that sees it has that element in its output, the others do not."""
    fresh = [5] * 40
    c = Cache(8, 4, 128, 32, torch.bfloat16, ragged(40, 100, 10), fresh, seed=91)
    words = random_words(fresh, 10)
    words &= ~2
    words[3::5] |= 2
    for b in range(40):
        p = int(c.cached[b]) + 1
        c.v[int(c.table[b, p // 32]), :, p % 32, 3] = bad
    out, _ = c.run(words)
    sees = ((words >> 1) & 1).bool()
    ref.check(out[~sees], None, [w[~sees] for w in c.want(words)])
    assert torch.isfinite(out[sees][:, :, 4:]).all()
    assert (out[sees][:, :, 3] == math.inf).all() if bad == math.inf else torch.isnan(out[sees][:, :, 3].float()).all()


def test_many_items_table_entries_out_of_range():
    page, cached, fresh = 16, [90] * 24, [1] * 24
    c = Cache(8, 8, 64, page, torch.bfloat16, cached, fresh, seed=92)
    c.table[3, 0], c.table[7, 2], c.table[7, 5] = -1, 10 ** 6, -(2 ** 31)
    p = torch.arange(91, device=DEV) // page
    unseen = [torch.zeros(91, dtype=torch.bool, device=DEV) for _ in cached]
    unseen[3], unseen[7] = p == 0, (p == 2) | (p == 5)                   # request 7's own row is among them
    ref.check(*c.run(), c.want(unseen=unseen))


def test_many_items_repeat_bitwise_and_follow_their_lengths():
    c = Cache(16, 8, 128, 32, torch.float16, ragged(40, 900, 11, 0.0), [1] * 40, seed=93)
    ws, out = moe.alloc_attn_workspace(c.attn, 40, 40), torch.empty_like(c.q)
    a, b = c.run(), c.run()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        moe.moe_attn_tree(c.attn, c.q, c.cu, c.cached, c.table, c.k, c.v, out, ws)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            moe.moe_attn_tree(c.attn, c.q, c.cu, c.cached, c.table, c.k, c.v, out, ws)
        g.replay()
    side.synchronize()
    assert torch.equal(out, a[0])
    shorter = [int(x) // 3 for x in c.cached.tolist()]
    c.cached.copy_(ints(shorter))
    c.rows = [[x[:n + 1] for x in kv] for kv, n in zip(c.rows, shorter)]
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    ref.check(out, None, c.want())


# ---------------------------------------------------------------- few items, equal shares of the line

@pytest.mark.parametrize("d", [64, 128])
def test_few_items_one_long_among_many_short(d):
    """More parts than CTAs at any even length: the line is cut where the CTAs' shares end."""
    cached, fresh = [40000] + [3] * 140, [2] + [1] * 140
    c = Cache(4, 1, d, 16, torch.bfloat16, cached, fresh, seed=94)
    ref.check(*c.run(), c.want())
    mask = random_words(fresh, 12, True)
    ref.check(*c.run(mask), c.want(mask))


# ---------------------------------------------------------------- many rows per request

WIDE = [   # kv heads, group, D, page, cached, rows; block tables for contexts past what L2 keeps
    (2, 2, 128, 128, [5000, 40], [33, 60], 300),                         # at most 128 rows: row tiles over alternate key tiles
    (2, 1, 64, 64, [3000, 0, 700], [64, 64, 50], 1100),
    (1, 8, 128, 16, [1000, 129, 127], [16, 5, 8], 2800),
    (1, 12, 128, 32, [2000, 31], [10, 4], 2100),                         # 12 does not divide 128
    (1, 1, 128, 16, [30000], [64], 8200),                                # one item over all CTAs
    (2, 4, 64, 16, [1500], [200], 2),                                    # no mask above 64 rows: a prompt's next part
    (2, 4, 64, 16, [1500], [200], 600),                                  # the same with a long block table
    (1, 3, 128, 128, [5, 700], [300, 65], 300),
    (4, 16, 128, 16, ragged(40, 300, 20), [9] * 40, 2),                  # more items than CTAs, whole and shared ones
    (8, 8, 64, 32, ragged(24, 700, 21), [33] * 24, 2),
]


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("case", range(len(WIDE)))
def test_many_rows_parity(dt, case):
    hk, g, d, page, cached, fresh, cols = WIDE[case]
    c = Cache(hk * g, hk, d, page, TYPES[dt], cached, fresh, seed=110 + case, extra_cols=cols)
    ref.check(*c.run(), c.want(), "causal")
    mask = random_words(fresh, case, True)
    ref.check(*c.run(mask), c.want(mask), "masked, empty rows")
    a, b = c.run(mask), c.run(mask)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("hk,g,d,page,cached,fresh,cols", [
    (2, 2, 128, 128, [5000, 40], [33, 60], 300), (2, 1, 64, 64, [3000, 0, 700], [64, 64, 50], 1100),
    (4, 16, 128, 16, ragged(40, 300, 22), [9] * 40, 2),
])
def test_many_rows_unseen_drafted_rows(bad, hk, g, d, page, cached, fresh, cols):
    c = Cache(hk * g, hk, d, page, torch.float16, cached, fresh, seed=130, extra_cols=cols)
    words, sees = poison(c, random_words(fresh, 13), 2, bad)
    out, _ = c.run(words)
    ref.check(out[~sees], None, [w[~sees] for w in c.want(words)])
    assert sees.any() and torch.isnan(out[sees].float()).all()


def test_many_rows_fresh_data_every_call():
    """Other values in every call on one workspace, wide and narrow calls in turn."""
    for rep in range(4):
        c = Cache(16, 1, 128, 16, torch.bfloat16, [900 + 200 * rep, 77], [9, 20], seed=140 + rep, extra_cols=4200)
        ref.check(*c.run(), c.want(), f"call {rep}")
        c = Cache(8, 8, 64, 16, torch.bfloat16, [300 + rep] * 24, [1] * 24, seed=150 + rep)
        ref.check(*c.run(), c.want(), f"call {rep}")


def test_one_workspace_for_all_kernels():
    """Calls of each form in turn on one workspace: each leaves it fit for the next, and the status word stays 0."""
    forms = [([2000], [1], 2), ([300] * 24, [1] * 24, 2), ([1200, 60], [33, 20], 2100), ([50], [200], 2)]
    for rep in range(2):
        for i, (cached, fresh, cols) in enumerate(forms):
            c = Cache(16, 8, 128, 16, torch.bfloat16, cached, fresh, seed=160 + i, extra_cols=cols)
            if rep == 0 and i == 0:
                ws = moe.alloc_attn_workspace(c.attn, 24, 512)
            out = torch.empty_like(c.q)
            moe.moe_attn_tree(c.attn, c.q, c.cu, c.cached, c.table, c.k, c.v, out, ws)
            ref.check(out, None, c.want(), f"form {i}")
            k = torch.randn((300, 8, 128), generator=gen(i), device=DEV).bfloat16()
            q = k.repeat(1, 2, 1)
            moe.moe_attn_prompt(c.attn, q, k, k, ints([0, 300]), torch.empty_like(q), ws)
            assert moe.moe_attn_get_device_status(c.attn, ws) == 0


@pytest.mark.parametrize("fresh,extra", [([1], 0), ([1] * 24, 0), ([40], 0), ([9], 4200)])
@pytest.mark.parametrize("cached", [1 << 20, 2 ** 31 - 1])
def test_lengths_past_the_block_table(fresh, extra, cached):
    """A request that claims more tokens than its row of the block table has: its rows see the table's tokens, whose
    missing pages count for nothing."""
    n = 200
    c = Cache(8, 8, 128, 16, torch.bfloat16, [n] * len(fresh), [0] * len(fresh), seed=170, extra_cols=extra)
    T = sum(fresh)
    cu = ints([0] + np.cumsum(fresh).tolist())
    q = torch.randn((T, 8, 128), generator=gen(171), device=DEV).bfloat16()
    out, lse = torch.empty_like(q), torch.empty((T, 8), dtype=torch.float32, device=DEV)
    # the page that holds the context's last tokens holds NaN behind them: fill it up with zero rows
    for b in range(len(fresh)):
        pg = int(c.table[b, n // 16])
        c.k[pg, :, n % 16:] = 0
        c.v[pg, :, n % 16:] = 0
        c.rows[b] = [torch.cat([x, torch.zeros((16 - n % 16, 8, 128), dtype=x.dtype, device=DEV)]) for x in c.rows[b]]
    ws = moe.alloc_attn_workspace(c.attn, len(fresh), T)
    moe.moe_attn_tree(c.attn, q, cu, ints([cached] * len(fresh)), c.table, c.k, c.v, out, ws, lse=lse)
    torch.cuda.synchronize()
    vis = [torch.ones((f, 208), dtype=torch.bool, device=DEV) for f in fresh]
    parts = [ref.attend(x, *c.rows[b], vis[b], 128 ** -0.5) for b, x in enumerate(q.split(fresh))]
    ref.check(out, lse, [torch.cat([p[i] for p in parts]) for i in range(4)])
    assert moe.moe_attn_get_device_status(c.attn, ws) == 0


def test_workspace_elsewhere_is_refused():
    c = Cache(4, 2, 64, 16, torch.bfloat16, [20], [1], seed=180)
    out, ws = torch.empty_like(c.q), moe.alloc_attn_workspace(c.attn, 1, 1).cpu()
    with pytest.raises(ValueError, match="ws is on cpu"):
        moe.moe_attn_tree(c.attn, c.q, c.cu, c.cached, c.table, c.k, c.v, out, ws)
    with pytest.raises(ValueError, match="ws is on cpu"):
        moe.moe_attn_prompt(c.attn, c.q, c.q[:, :2], c.q[:, :2], c.cu, out, ws)
