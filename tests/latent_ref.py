"""Latent attention in 64 bits, and the error that its kernels may have: the
bound of ``attn_ref`` with keys of 576 (absorbed) or 192 elements (expanded)."""
import math

import torch

from attn_ref import LOST, U


def attend(q, k, v, visible, scale):
    """q [n][H][dk], k [m][H or 1][dk], v [m][H or 1][dv], visible [n][m] bool -> out, lse, bound, lse_bound (float64).
    Keys and values that no row sees may hold anything."""
    n, h, d = q.shape
    dt, dev = q.dtype, q.device
    seen = visible.any(0)[:, None, None]
    k, v = torch.where(seen, k.double(), 0.0), torch.where(seen, v.double(), 0.0)
    out, bound = torch.zeros((2, n, h, v.shape[2]), dtype=torch.float64, device=dev)
    lse = torch.full((n, h), -math.inf, dtype=torch.float64, device=dev)
    lse_bound = torch.zeros((n, h), dtype=torch.float64, device=dev)
    row, count = visible.any(1), visible.sum(1)
    if k.shape[0] == 0:
        return out, lse, bound, lse_bound
    for i in range(h):
        ki, vi, qi = k[:, i % k.shape[1]], v[:, i % v.shape[1]], q[:, i].double()
        s = torch.where(visible, scale * (qi @ ki.T), -math.inf)
        big = torch.where(visible, scale * (qi.abs() @ ki.abs().T), 0.0).amax(1)
        w = torch.softmax(torch.where(row[:, None], s, 0.0), 1) * row[:, None]
        out[:, i] = w @ vi
        eps = 2 * U[dt] + 2 * (d + 4) * 2.0 ** -24 * big + 2.0 ** -19 + count * 2.0 ** -24
        bound[:, i] = eps[:, None] * (w @ vi.abs()) + (count * LOST[dt])[:, None] * vi.abs().max()
        lse[:, i] = torch.where(row, torch.logsumexp(s, 1), -math.inf)
        lse_bound[:, i] = (d + 4) * 2.0 ** -24 * big + 2.0 ** -19 * (1 + lse[:, i].abs().nan_to_num(posinf=0.0))
    return out, lse, bound, lse_bound
