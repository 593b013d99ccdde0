"""The attention operators in 64 bits, one row and one token at a time where
it matters, and the error that their kernels may have.

Bound of an output element.  Let w be the row's softmax weights and
A = sum_j w_j |v_j|.  The kernels form scores from exact products of 2-byte
elements summed in fp32, round each weight to the element type before it
multiplies v (unit roundoff u: half of the type's epsilon), sum in fp32 and round
the result (u again).  A score is off by at most (D + 4) 2^-24 S, with S the
largest sum over the head of |scale q k| of the row's visible tokens (the
scale and the base-2 exponent's argument are among the 4), and a weight, a
quotient of two exponentials, by twice that relatively; the SFU exponential
and the reciprocal add 2^-21.  Together
    |error| <= (2 u + 2 (D + 4) 2^-24 S + 2^-20) A  + tiny,
with tiny for weights that f16 cannot hold: a weight under 2^-24 of the row's
largest may be lost, 2^-25 of max |v| per visible token (f16), and 2^-133 for
bf16, taken as 2^-60.  The second-order terms and the fp32 sums over n tokens
(n 2^-24 A) are covered by doubling 2^-20 and adding n 2^-24."""
import math

import numpy as np
import torch

U = {t: torch.finfo(t).eps / 2 for t in (torch.bfloat16, torch.float16)}      # 8 and 11 significant bits
LOST = {torch.bfloat16: 2.0 ** -60, torch.float16: 2.0 ** -25}


def attend(q, k, v, visible, scale):
    """q [n][Hq][D], k, v [m][Hk][D], visible [n][m] bool -> out, lse, bound, lse_bound (float64).
    Keys and values that no row sees may hold anything."""
    n, hq, d = q.shape
    hk = k.shape[1]
    dt = q.dtype
    seen = visible.any(0)
    q, k, v = q.double(), torch.where(seen[:, None, None], k.double(), 0.0), torch.where(seen[:, None, None], v.double(), 0.0)
    out, bound = torch.zeros((2, n, hq, d), dtype=torch.float64, device=q.device)
    lse = torch.full((n, hq), -math.inf, dtype=torch.float64, device=q.device)
    lse_bound = torch.zeros((n, hq), dtype=torch.float64, device=q.device)
    for h in range(hq):
        kh, vh = k[:, h // (hq // hk)], v[:, h // (hq // hk)]
        s = torch.where(visible, scale * (q[:, h] @ kh.T), -math.inf)
        mag = torch.where(visible, scale * (q[:, h].abs() @ kh.abs().T), 0.0)
        big = mag.amax(1) if mag.shape[1] else torch.zeros(n, dtype=torch.float64, device=q.device)
        row = visible.any(1)
        w = torch.softmax(torch.where(row[:, None], s, 0.0), 1) * row[:, None] if s.shape[1] else s
        out[:, h] = w @ vh
        a = w @ vh.abs()
        eps = 2 * U[dt] + 2 * (d + 4) * 2.0 ** -24 * big + 2.0 ** -19 + visible.sum(1) * 2.0 ** -24
        vmax = vh.abs().max() if vh.numel() else 0.0
        bound[:, h] = eps[:, None] * a + (visible.sum(1) * LOST[dt])[:, None] * vmax
        if s.shape[1]:
            lse[:, h] = torch.where(row, torch.logsumexp(s, 1), -math.inf)
        lse_bound[:, h] = (d + 4) * 2.0 ** -24 * big + 2.0 ** -19 * (1 + lse[:, h].abs().nan_to_num(posinf=0.0))
    return out, lse, bound, lse_bound


def check(out, lse, ref, label=""):
    ro, rl, bo, bl = ref
    assert torch.isfinite(out).all(), f"{label}: non-finite output"
    d = (out.double() - ro).abs()
    assert (d <= bo).all(), f"{label}: off by {float((d / bo.clamp(min=1e-300)).max()):.2f} times the bound"
    if lse is not None:
        assert (torch.isinf(lse) == torch.isinf(rl)).all(), f"{label}: rows that see nothing"
        e = torch.where(torch.isinf(rl), 0.0, (lse.double() - rl).abs())
        assert (e <= bl).all(), f"{label}: lse off by {float((e / bl.clamp(min=1e-300)).max()):.2f} times the bound"


def words_to_visible(words, n):
    """int64 mask words of n rows -> [n][n] bool (bit j of row i; rows from the 65th on are seen by none)."""
    vis = torch.zeros((n, n), dtype=torch.bool, device=words.device)
    m = min(n, 64)
    if m:
        vis[:, :m] = ((words[:, None] >> torch.arange(m, device=words.device)) & 1).bool()
    return vis


def plan(cached, fresh, free, table, page, num_pages, T, parents=None):
    """moe_kv_plan, one row and one page at a time (numpy)."""
    table = np.array(table, np.int32)
    B, width = table.shape
    flags, used, cu = 0, 0, [0]
    slots, positions, words = np.full(T, -1, np.int32), np.full(T, -1, np.int32), np.zeros(T, np.uint64)
    top, places = 0, []
    for b in range(B):
        c, f = max(int(cached[b]), 0), max(int(fresh[b]), 0)
        flags |= 1 if cached[b] < 0 or fresh[b] < 0 else 0
        f = min(f, T)
        need, have = -(-(c + f) // page), -(-c // page)
        flags |= 2 if need > width else 0
        flags |= 8 if parents is not None and f > 64 else 0
        top = max(top, c + f)
        for col in range(have, min(need, width)):
            pg = int(free[used]) if used < len(free) else -1
            if not 0 <= pg < num_pages:
                pg = -1
                flags |= 4
            table[b, col] = pg
            used += 1
        for i in range(f):
            places.append((b, c, i))
        cu.append(cu[-1] + f)
    flags |= 1 if cu[-1] > T else 0
    for t, (b, c, i) in enumerate(places[:T]):
        p = c + i
        positions[t] = p
        if p // page < width:
            pg = int(table[b, p // page])
            if 0 <= pg < num_pages:
                slots[t] = pg * page + p % page
            else:
                flags |= 4
        if parents is not None:
            path = [i]
            while i < 64:
                up = int(parents[cu[b] + path[-1]])
                if up == -1:
                    break
                if not 0 <= up < path[-1]:
                    flags |= 8
                    break
                path.append(up)
            if i < 64:
                words[t] = np.uint64(sum(1 << j for j in path))
            positions[t] = c + len(path) - 1
    info = [cu[-1], min(used, len(free)), top, flags]
    return table, np.array(cu, np.int32), slots, positions, words.view(np.int64), np.array(info, np.int32)
