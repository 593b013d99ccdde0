"""A device wait of the attention kernels that runs out: the call returns, the status
word says so, and the workspace serves the next call.  The wait is made to run
out by a test hook of the handle (20 ms instead of 2 s, for bytes that no copy brings)."""
import time

import pytest
import torch

import attn_ref as ref
from quantized_moe_expert_router_gb300 import moe
from test_gpu_attn import Cache, built, offsets, prompt_ref, randn  # noqa: F401  (built: the module's build fixture)

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def stalled(attn):
    c = attn.cfg
    return moe.Attention(c.q_heads, c.kv_heads, c.head_dim, c.page_size, c.num_pages, c.max_pages, attn.dtype, flags=moe.ATTN_TEST_STALL)


def expect_timeout(attn, ws, call):
    """The waits that may run out one after another: some ten of 20 ms each."""
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    call(stalled(attn))
    torch.cuda.synchronize()
    assert time.perf_counter() - t0 < 1.0
    assert moe.moe_attn_get_device_status(attn, ws) == moe.FLAG_TIMEOUT
    assert moe.moe_attn_get_device_status(attn, ws) == 0


@pytest.mark.parametrize("hk,g,d,lengths", [
    (40, 1, 64, [129, 1, 0, 513, 300, 64]), (24, 2, 128, [700, 129, 513]),          # pairs of row tiles, several items a CTA
    (2, 4, 64, [500, 33]), (1, 8, 128, [400]), (1, 1, 128, [1]),                    # single ones
])
def test_prompt_wait_that_runs_out(hk, g, d, lengths):
    T, dt = sum(lengths), torch.bfloat16
    attn = moe.Attention(hk * g, hk, d, 16, 1, 1, dt)
    q, k, v = (randn((T, h, d), dt, 500 + i) for i, h in enumerate((hk * g, hk, hk)))
    out, ws = torch.empty_like(q), moe.alloc_attn_workspace(attn, len(lengths), T)
    for _ in range(2):
        expect_timeout(attn, ws, lambda a: moe.moe_attn_prompt(a, q, k, v, offsets(lengths), out, ws))
        moe.moe_attn_prompt(attn, q, k, v, offsets(lengths), out, ws)
        torch.cuda.synchronize()
        ref.check(out, None, prompt_ref(q, k, v, lengths, d ** -0.5))
        assert moe.moe_attn_get_device_status(attn, ws) == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("cached,fresh,cols", [
    ([2000, 3], [1, 5], 2), ([40000] + [3] * 140, [1] * 141, 2),                    # few items: parts, and the line
    ([300] * 24, [1] * 24, 2),                                                      # many items
    ([1200, 60], [33, 20], 2100), ([90, 300, 700] * 12, [33] * 36, 600),            # many rows: parts, and the line
])
def test_tree_wait_that_runs_out(d, cached, fresh, cols):
    c = Cache(16, 8, d, 16, torch.float16, cached, fresh, seed=260, extra_cols=cols)
    out, ws = torch.empty_like(c.q), moe.alloc_attn_workspace(c.attn, len(fresh), c.T)
    for _ in range(2):
        expect_timeout(c.attn, ws, lambda a: moe.moe_attn_tree(a, c.q, c.cu, c.cached, c.table, c.k, c.v, out, ws))
        moe.moe_attn_tree(c.attn, c.q, c.cu, c.cached, c.table, c.k, c.v, out, ws)
        torch.cuda.synchronize()
        ref.check(out, None, c.want())
        assert moe.moe_attn_get_device_status(c.attn, ws) == 0


@pytest.mark.parametrize("cached,fresh,cols", [([2000, 3], [1, 5], 2), ([300] * 24, [1] * 24, 2), ([1200, 60], [33, 20], 2100)])
def test_status_leaves_the_workspace_as_new(cached, fresh, cols):
    """Whatever a call that did not end left in it: every word that a call has to find at zero is zero."""
    c = Cache(16, 8, 128, 16, torch.bfloat16, cached, fresh, seed=270, extra_cols=cols)
    out, ws = torch.empty_like(c.q), moe.alloc_attn_workspace(c.attn, len(fresh), c.T)
    ws.fill_(255)
    moe.moe_attn_get_device_status(c.attn, ws)
    moe.moe_attn_tree(c.attn, c.q, c.cu, c.cached, c.table, c.k, c.v, out, ws)
    torch.cuda.synchronize()
    ref.check(out, None, c.want())
    assert moe.moe_attn_get_device_status(c.attn, ws) == 0


def test_status_refuses_what_is_not_a_workspace():
    attn = moe.Attention(4, 2, 64, 16, 8, 4)
    ws = moe.alloc_attn_workspace(attn, 1, 1)
    for bad in (ws[:1024], ws[:16], ws.cpu(), torch.zeros(1, dtype=torch.uint8, device=DEV).expand(ws.numel())):
        with pytest.raises(ValueError, match="is not a workspace"):
            moe.moe_attn_get_device_status(attn, bad)
