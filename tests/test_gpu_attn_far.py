"""Attention on scores that are large against their differences, where c m (the scaled maximum) rounded by itself
would move a weight by more than the result's rounding: prompts and trees in each of their kernels, and both
latent forms, against the definition in 64 bits.

Scores are integers of at most 24 bits times a power of two, sums of three products of powers of two and small
integers, so every one of them is exact in fp32 and the bound has no part that grows with them:
    |error| <= (2 u + 2^-13) A + u |value| + n LOST,   A = sum_j w_j |v_j|,
u for the weights and u for the result; the exponentials' arguments c (s - m) are below 2^5 where a weight counts, so their
roundings, the factor's and the SFU's are 2^-18, and c m as such is taken only up to 2^10: 2^-15 ln 2 for each of
two maxima; twice that for a quotient."""
import math

import numpy as np
import pytest
import torch

from attn_ref import LOST, U
from quantized_moe_expert_router_gb300 import moe
from test_gpu_attn import Cache, built, ints, offsets  # noqa: F401  (built: the module's build fixture)

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def definition(q, k, v, visible, scale):
    """q [n][H][d], k, v [m][Hk][d], visible [n][m] -> out, lse, bound (float64)."""
    (n, h, _), g = q.shape, q.shape[1] // k.shape[1]
    out, bound = torch.empty((2, n, h, v.shape[2]), dtype=torch.float64, device=DEV)
    lse = torch.empty((n, h), dtype=torch.float64, device=DEV)
    for i in range(h):
        s = torch.where(visible, scale * (q[:, i].double() @ k[:, i // g].double().T), -math.inf)
        w, vi = torch.softmax(s, 1), v[:, i // g].double()
        out[:, i], lse[:, i] = w @ vi, torch.logsumexp(s, 1)
        bound[:, i] = (2 * U[q.dtype] + 2.0 ** -13) * (w @ vi.abs()) + U[q.dtype] * out[:, i].abs() \
            + visible.sum(1)[:, None] * LOST[q.dtype] * vi.abs().max()
    return out, lse, bound


def check(out, lse, want):
    assert torch.isfinite(out).all()
    off = (out.double() - want[0]).abs() / want[2]
    assert (off <= 1).all(), f"off by {float(off.max()):.2f} times the bound"
    assert ((lse.double() - want[1]).abs() <= 2.0 ** -22 * want[1].abs() + 2.0 ** -12).all()


class Far:
    """Rows and tokens with scores sign * 2^power + step * (level of the token + a number of the head), step the least that
    sums of this size resolve.  kind: "spread", levels that compete, by groups of tokens; "rise", one token of a group
    is some 2^8.2 above the others of the group before; "ties", all weight to tokens of one score."""

    def __init__(self, power, sign, kind, scale, group, seed):
        self.power, self.sign, self.kind, self.scale, self.group = power, sign, kind, float(np.float32(scale)), group
        self.rng = np.random.default_rng(seed)
        self.step = 2.0 ** (power - 23)
        self.unit = self.scale * 1.4427 * self.step          # of a level, in the exponent

    def keys(self, shape, dt):
        """[tokens][heads][d], of which the first three elements count."""
        n = shape[0]
        token = np.arange(n)
        if self.kind == "spread":
            top = int(min(96, max(1, 6 / self.unit)))
            level = self.rng.integers(0, top + 1, -(-n // self.group))[token // self.group] + self.rng.integers(0, 3, n)
        elif self.kind == "rise":
            level = np.where(token % self.group == self.group // 2, math.ceil(8.2 / self.unit), 0) * (token >= self.group)
        else:
            level = self.rng.integers(0, 2, n)
        assert level.max() < 128
        k = torch.zeros(shape, dtype=dt, device=DEV)
        k[..., 0] = self.sign * 2.0 ** (self.power - self.power // 2)
        k[..., 1] = torch.tensor(level, device=DEV, dtype=dt)[:, None]
        k[..., 2] = 1.0
        return k

    def queries(self, shape, dt):
        q = torch.zeros(shape, dtype=dt, device=DEV)
        q[..., 0] = 2.0 ** (self.power // 2)
        q[..., 1] = self.step
        q[..., 2] = self.step * (torch.arange(shape[1], device=DEV) * 29 % 128)
        return q

    def values(self, shape, dt):
        """Groups of tokens differ in sign, so that a group's weight shows."""
        v = 1.0 + torch.tensor(self.rng.random(shape), device=DEV)
        return (v * (1 - 2 * (torch.arange(shape[0], device=DEV) // self.group % 2))[:, None, None]).to(dt)


SCORES = [(20, 1, "spread", 1.0), (24, 1, "spread", None), (24, -1, "spread", None), (26, 1, "spread", None), (26, -1, "rise", None),
          (25, 1, "rise", None), (40, 1, "spread", 2.0 ** -18), (36, 1, "ties", None), (60, -1, "ties", None)]


FORMS = pytest.mark.parametrize("dt,power,sign,kind,scale", [(dt, *s) for dt in TYPES for s in SCORES if dt == "bf16" or s[0] <= 26])   # f16 ends at 2^16


def causal(n):
    return torch.ones((n, n), dtype=torch.bool, device=DEV).tril()


@FORMS
@pytest.mark.parametrize("heads,n", [(4, 700), (90, 500)])             # single row tiles over alternate key tiles, pairs
def test_latent_prompt(heads, n, dt, power, sign, kind, scale):
    f, t = Far(power, sign, kind, 192 ** -0.5 if scale is None else scale, 128, 1), TYPES[dt]
    q, k, v = f.queries((n, heads, 192), t), f.keys((n, heads, 128), t), f.values((n, heads, 128), t)
    lat = moe.LatentAttention(heads, 16, 1, 1, t, softmax_scale=f.scale)
    ws, out = moe.alloc_latent_workspace(lat, 1, n), torch.empty((n, heads, 128), dtype=t, device=DEV)
    lse = torch.empty((n, heads), dtype=torch.float32, device=DEV)
    r = torch.zeros((n, 64), dtype=t, device=DEV)
    moe.moe_latent_prompt(lat, q, k, r, v, offsets([n]), out, ws, lse=lse)
    assert moe.moe_latent_get_device_status(lat, ws) == 0
    check(out, lse, definition(q[..., :128], k, v, causal(n), f.scale))


@FORMS
@pytest.mark.parametrize("hk,g,d,n", [(1, 4, 64, 700), (2, 2, 128, 700), (45, 2, 64, 500), (24, 4, 128, 500)])
def test_prompt(hk, g, d, n, dt, power, sign, kind, scale):
    f, t = Far(power, sign, kind, d ** -0.5 if scale is None else scale, 128, 2), TYPES[dt]
    q, k, v = f.queries((n, hk * g, d), t), f.keys((n, hk, d), t), f.values((n, hk, d), t)
    attn = moe.Attention(hk * g, hk, d, 16, 1, 1, t, softmax_scale=f.scale)
    ws, out = moe.alloc_attn_workspace(attn, 1, n), torch.empty((n, hk * g, d), dtype=t, device=DEV)
    lse = torch.empty((n, hk * g), dtype=torch.float32, device=DEV)
    moe.moe_attn_prompt(attn, q, k, v, offsets([n]), out, ws, lse=lse)
    assert moe.moe_attn_get_device_status(attn, ws) == 0
    check(out, lse, definition(q, k, v, causal(n), f.scale))


@FORMS
@pytest.mark.parametrize("hk,g,d,page,cached,fresh,cols,group", [
    (2, 4, 128, 16, [1500, 90], [1, 3], 2, 16), (1, 8, 64, 32, [2000], [2], 2, 32),                   # few items
    (8, 4, 128, 16, [300 + 7 * i for i in range(24)], [1] * 24, 2, 16), (8, 4, 64, 64, [500] * 24, [1] * 24, 2, 32),   # many
    (2, 2, 128, 128, [3000, 40], [33, 60], 300, 128), (2, 1, 64, 64, [3000, 0, 700], [64, 64, 50], 1100, 128),      # many rows
    (4, 16, 128, 16, [150 + 9 * i for i in range(40)], [9] * 40, 300, 128),
])
def test_tree(hk, g, d, page, cached, fresh, cols, group, dt, power, sign, kind, scale):
    f, t = Far(power, sign, kind, d ** -0.5 if scale is None else scale, group, 3), TYPES[dt]
    c = Cache(hk * g, hk, d, page, t, cached, fresh, seed=7, extra_cols=cols)
    q, lo, parts = f.queries((c.T, hk * g, d), t), 0, []
    for b, (a, n) in enumerate(zip(cached, fresh)):
        k, v = f.keys((a + n, hk, d), t), f.values((a + n, hk, d), t)
        p = torch.arange(a + n, device=DEV)
        pg = c.table[b, p // page].long()
        c.k[pg, :, p % page], c.v[pg, :, p % page] = k, v
        parts.append(definition(q[lo:lo + n], k, v, causal(a + n)[a:], f.scale))
        lo += n
    attn = moe.Attention(hk * g, hk, d, page, c.k.shape[0], c.table.shape[1], t, softmax_scale=f.scale)
    ws, out = moe.alloc_attn_workspace(attn, len(fresh), c.T), torch.empty_like(q)
    lse = torch.empty((c.T, hk * g), dtype=torch.float32, device=DEV)
    moe.moe_attn_tree(attn, q, c.cu, c.cached, c.table, c.k, c.v, out, ws, lse=lse)
    assert moe.moe_attn_get_device_status(attn, ws) == 0
    check(out, lse, [torch.cat([p[i] for p in parts]) for i in range(3)])


@FORMS
@pytest.mark.parametrize("heads,page,cached,fresh,wide", [
    (16, 16, [1500], [1], False), (64, 64, [1700, 90], [3, 1], False), (128, 32, [700, 1200, 3], [2, 5, 1], False),    # cut
    (16, 64, [150 + 3 * i for i in range(60)], [1] * 60, False), (16, 64, [150 + 3 * i for i in range(60)], [1] * 60, True),   # whole, and cut
])
def test_latent_tree(heads, page, cached, fresh, wide, dt, power, sign, kind, scale):
    """The scores come from the key part alone, so that the values are the latents of the other forms' values."""
    f, t = Far(power, sign, kind, 192 ** -0.5 if scale is None else scale, 64, 4), TYPES[dt]
    need = [-(-(a + n) // page) for a, n in zip(cached, fresh)]
    table = torch.full((len(need), max(need) + (2000 if wide else 0)), -1, dtype=torch.int32, device=DEV)
    order = torch.randperm(sum(need), generator=torch.Generator().manual_seed(5)).int().to(DEV)
    cache = torch.full((sum(need), page, 576), math.nan, dtype=t, device=DEV)
    T, lo, at, parts = sum(fresh), 0, 0, []
    q = f.queries((T, heads, 64), t)
    for b, (a, n) in enumerate(zip(cached, fresh)):
        table[b, :need[b]] = order[at:at + need[b]]
        k, v = f.keys((a + n, 1, 64), t), f.values((a + n, 1, 512), t)
        p = torch.arange(a + n, device=DEV)
        cache[table[b, p // page].long(), p % page] = torch.cat([v, k], 2)[:, 0]
        parts.append(definition(q[lo:lo + n], k, v, causal(a + n)[a:], f.scale))
        lo, at = lo + n, at + need[b]
    lat = moe.LatentAttention(heads, page, sum(need), table.shape[1], t, softmax_scale=f.scale)
    ws, out = moe.alloc_latent_workspace(lat, len(fresh), T), torch.empty((T, heads, 512), dtype=t, device=DEV)
    lse = torch.empty((T, heads), dtype=torch.float32, device=DEV)
    moe.moe_latent_tree(lat, torch.zeros_like(out), q, offsets(fresh), ints(cached), table, cache, out, ws, lse=lse)
    assert moe.moe_latent_get_device_status(lat, ws) == 0
    check(out, lse, [torch.cat([p[i] for p in parts]) for i in range(3)])
