"""attn_wide_kernel with many short items a CTA: items of one key tile, with and
without a masked one, in every order, against the definition in 64 bits.  A few
requests are repeated many times, so that the reference is that of the few."""
import numpy as np
import pytest
import torch

import attn_ref as ref
from quantized_moe_expert_router_gb300 import moe
from test_gpu_attn import TYPES, Cache, built, gen, ints, offsets, prompt_ref, randn, random_words  # noqa: F401  (built: the module's build fixture)

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def check_repeated(out, lse, want, reps, label):
    out, lse = out.view(reps, -1, *out.shape[1:]), lse.view(reps, -1, lse.shape[-1])
    for r in range(reps):
        ref.check(out[r], lse[r], want, f"{label}, repetition {r}")


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("hk,g,d,lengths,reps", [
    (8, 1, 64, [1, 128, 2, 127, 64, 3, 90, 128], 60), (8, 1, 128, [128, 1, 33, 127], 90),       # one key tile each
    (4, 3, 64, [84, 1, 42, 130, 85], 80), (2, 8, 128, [129, 1, 16, 255, 31], 80),               # one to three
])
def test_prompts_of_one_key_tile(dt, hk, g, d, lengths, reps):
    dt, n = TYPES[dt], sum(lengths)
    attn = moe.Attention(hk * g, hk, d, 16, 1, 1, dt)
    ws = moe.alloc_attn_workspace(attn, reps * len(lengths), reps * n)
    for call in range(4):
        q, k, v = (randn((n, h, d), dt, 400 + 10 * call + i, 1.5 if i == 0 else 1.0) for i, h in enumerate((hk * g, hk, hk)))
        want = prompt_ref(q, k, v, lengths, d ** -0.5)
        q, k, v = (x.repeat(reps, 1, 1) for x in (q, k, v))
        out, lse = torch.empty_like(q), torch.empty(q.shape[:2], dtype=torch.float32, device=DEV)
        moe.moe_attn_prompt(attn, q, k, v, offsets(lengths * reps), out, ws, lse=lse)
        check_repeated(out, lse, want, reps, f"call {call}")
    assert moe.moe_attn_get_device_status(attn, ws) == 0


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("g,d,page,cached,fresh,reps", [
    (64, 64, 16, [123], [5], 300),                                   # an item with a masked tile, one without, in turn
    (64, 128, 16, [123, 251, 40], [5, 5, 3], 100),                   # the same over one and two key tiles
    (32, 64, 128, [127, 0, 119, 300, 1], [9, 9, 9, 4, 17], 50),
    (8, 64, 32, [90, 700, 31, 260], [33, 33, 33, 33], 30),
])
def test_cache_items_of_one_key_tile(dt, g, d, page, cached, fresh, reps):
    c = Cache(2 * g, 2, d, page, TYPES[dt], cached, fresh, seed=200 + d + g, extra_cols=256 // page)
    B, T = len(fresh) * reps, c.T * reps
    q, cu = c.q.repeat(reps, 1, 1), offsets(fresh * reps)
    table, lengths = c.table.repeat(reps, 1), c.cached.repeat(reps)
    ws = moe.alloc_attn_workspace(c.attn, B, T)
    for empty in (None, False, True):
        mask = None if empty is None else random_words(fresh, 21, empty)
        out, lse = torch.empty_like(q), torch.empty(q.shape[:2], dtype=torch.float32, device=DEV)
        moe.moe_attn_tree(c.attn, q, cu, lengths, table, c.k, c.v, out, ws, tree_mask=None if mask is None else mask.repeat(reps), lse=lse)
        check_repeated(out, lse, c.want(mask), reps, f"masked {mask is not None}, empty {empty}")
    assert moe.moe_attn_get_device_status(c.attn, ws) == 0


@pytest.mark.parametrize("d", [64, 128])
def test_bad_values_stay_with_their_item(d):
    """Items whose masked tile holds infinite values between items that hold none: the note of bad tokens is the item's own."""
    g, cached, fresh, reps = 64, [123, 123], [5, 5], 150
    c = Cache(g, 1, d, 16, torch.bfloat16, cached, fresh, seed=230 + d, extra_cols=16)
    p = 124                                              # the second fresh row of request 0, which its word below lets no row see but row 2
    c.v[int(c.table[0, p // 16]), :, p % 16, 3] = float("inf")
    words = random_words(fresh, 23)
    words[:5] &= ~2
    words[2] |= 2
    want = c.want(words)
    out = torch.empty((c.T * reps, g, d), dtype=torch.bfloat16, device=DEV)
    ws = moe.alloc_attn_workspace(c.attn, 2 * reps, c.T * reps)
    moe.moe_attn_tree(c.attn, c.q.repeat(reps, 1, 1), offsets(fresh * reps), c.cached.repeat(reps), c.table.repeat(reps, 1), c.k, c.v, out, ws,
                      tree_mask=words.repeat(reps))
    keep = [i for i in range(c.T) if i != 2]
    for r, o in enumerate(out.view(reps, c.T, g, d)):
        ref.check(o[keep], None, [w[keep] for w in want], f"repetition {r}")
        assert (o[2, :, 3] == float("inf")).all() and torch.isfinite(o[2, :, 4:]).all()
    assert moe.moe_attn_get_device_status(c.attn, ws) == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("cached,fresh,cols", [([0, 9], [4, 5], 2), ([0] * 20 + [50], [2] * 21, 2), ([0, 300], [40, 64], 2100),
                                               ([0] * 30, [33] * 30, 600)])
def test_rows_that_see_nothing(d, cached, fresh, cols):
    """Outputs of 0 and a logarithm of minus infinity, in each kernel; the rows between them as they are."""
    c = Cache(16, 8, d, 16, torch.bfloat16, cached, fresh, seed=280, extra_cols=cols)
    words = random_words(fresh, 31)
    words[::3] = 0
    want = c.want(words)
    out, lse = c.run(words)
    ref.check(out, lse, want)
    none = torch.isinf(want[1])
    assert none.any() and (want[1][none] == -float("inf")).all()
    assert (lse[none] == -float("inf")).all() and (out[none] == 0).all()
