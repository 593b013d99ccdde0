"""Rows whose context is cut into parts (or over the warps of a CTA) against what they would be in one piece, where a part of the
context has no weight."""
import math

import pytest
import torch

import attn_ref as ref
from test_gpu_attn import DEV, Cache, built  # noqa: F401  (built: the module's build fixture)

pytestmark = pytest.mark.gpu
FORMS = [   # kv heads, group, D, page, cached, rows, further block-table entries
    (2, 4, 128, 16, [3000, 90], [1, 3], 2), (1, 8, 64, 32, [4000], [2], 2),                                       # few items
    (8, 4, 128, 16, [300 + 7 * i for i in range(24)], [1] * 24, 2), (8, 4, 64, 64, [500] * 24, [1] * 24, 2),       # many
    (2, 2, 128, 128, [5000, 40], [33, 60], 300), (2, 1, 64, 64, [3000, 0, 700], [64, 64, 50], 1100),               # many rows
]


@pytest.mark.parametrize("hk,g,d,page,cached,fresh,cols", FORMS)
@pytest.mark.parametrize("all_of_it", [False, True])
def test_scores_of_minus_infinity_before_infinite_values(hk, g, d, page, cached, fresh, cols, all_of_it):
    """Zero times infinity is NaN wherever the context is cut: tokens of no weight with an infinite element of v, whole parts of
    the context among them, and in the end all cached ones."""
    c = Cache(hk * g, hk, d, page, torch.bfloat16, cached, fresh, seed=31, extra_cols=cols)
    c.q[:, :, 7] = 1.0
    unseen, hit, lo = [], torch.zeros(c.T, dtype=torch.bool, device=DEV), 0
    for b, (a, n) in enumerate(zip(cached, fresh)):
        m = a if all_of_it else a // 2
        p = torch.arange(m, device=DEV)
        pg = c.table[b, p // page].long()
        c.k[pg, :, p % page, 7] = -math.inf
        c.v[pg, :, p % page, 5] = math.inf
        unseen.append(torch.arange(a + n, device=DEV) < m)
        hit[lo:lo + n] = m > 0
        lo += n
    out, lse = c.run()
    want = c.want(unseen=unseen)
    assert out[hit, :, 5].isnan().all(), "a value of no weight was lost with its part"
    out[hit, :, 5] = want[0][hit, :, 5].to(out.dtype)
    ref.check(out, lse, want)
