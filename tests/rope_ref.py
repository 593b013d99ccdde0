"""Rotary positions in 64 bits, and the error that their kernel may have.

A coefficient, s cos a or s sin a, is off by s (2^-20.9 + 2^-21.3 + 2^-23): the SFU's sine
and cosine on [-pi, pi], an angle rounded to fp32 twice (pi 2^-23), and the factor's
product; and by s p f 2^-50 for frequencies of 53 bits out of a power and a quotient.
An element sums two products in fp32 (2^-23 of their sizes) and is rounded
once (u of its value, or half the smallest step of its type).  With m = s (|x| + |y|):
    |error| <= m (2^-19 + p f 2^-50) + u |value| + tiny."""
import math

import torch

U = {t: torch.finfo(t).eps / 2 for t in (torch.bfloat16, torch.float16)}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}


def frequencies(dims, theta, scaling="plain", factor=1.0, original=0, low=1.0, high=32.0):
    out = []
    for i in range(dims // 2):
        w = theta ** (-2.0 * i / dims)
        if scaling == "linear":
            w /= factor
        elif scaling == "base":
            w = (theta * factor ** (dims / (dims - 2))) ** (-2.0 * i / dims)
        elif scaling == "yarn":
            at = [dims / 2 * math.log(original / (2 * math.pi * t)) / math.log(theta) for t in (high, low)]
            lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), dims - 1)
            r = min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0)
            w = r * w / factor + (1 - r) * w
        elif scaling == "bands":
            s = min(max((original * w / (2 * math.pi) - low) / (high - low), 0.0), 1.0)
            w = s * w + (1 - s) * w / factor
        out.append(w)
    return torch.tensor(out, dtype=torch.float64)


def turn(x, positions, freq, interleaved, factor=1.0):
    """x [rows][heads][d] -> (float64 result, bound); rows at negative positions keep their values."""
    freq, n = freq.to(x.device), 2 * freq.numel()
    v = x.double()
    a = positions.double()[:, None] * freq
    cos, sin = (factor * a.cos())[:, None], (factor * a.sin())[:, None]
    p, q = (v[..., 0:n:2], v[..., 1:n:2]) if interleaved else (v[..., :n // 2], v[..., n // 2:n])
    join = (lambda f, g: torch.stack([f, g], -1).flatten(-2)) if interleaved else (lambda f, g: torch.cat([f, g], -1))
    out = torch.cat([join(p * cos - q * sin, p * sin + q * cos), v[..., n:]], -1)
    size = factor * (p.abs() + q.abs()) * (2.0 ** -19 + (a.abs() * 2.0 ** -50)[:, None])
    bound = torch.cat([join(size, size) + U[x.dtype] * out[..., :n].abs() + TINY[x.dtype], torch.zeros_like(v[..., n:])], -1)
    live = (positions >= 0)[:, None, None]
    return torch.where(live, out, v), torch.where(live, bound, 0.0)


def check(got, want, label=""):
    out, bound = want
    d = (got.double() - out).abs()
    assert (d <= bound).all(), f"{label}: off by {float((d / bound.clamp(min=1e-300)).max()):.2f} times the bound"
