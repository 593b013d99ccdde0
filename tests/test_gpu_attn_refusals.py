"""Arguments of the attention calls at the edge of what they take."""
import pytest
import torch

from quantized_moe_expert_router_gb300 import moe
from test_gpu_attn import Cache, built  # noqa: F401  (built: the module's build fixture)

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def test_workspace_with_strides_is_refused():
    """Bytes that only a stride makes up are not there to be written."""
    c = Cache(4, 2, 64, 16, torch.bfloat16, [20], [1], seed=181)
    out, n = torch.empty_like(c.q), moe.moe_attn_workspace_bytes(c.attn, 1, 1)
    for ws in (torch.zeros(1, dtype=torch.uint8, device=DEV).expand(n), torch.zeros(2 * n, dtype=torch.uint8, device=DEV)[::2]):
        with pytest.raises(ValueError, match="ws with strides"):
            moe.moe_attn_tree(c.attn, c.q, c.cu, c.cached, c.table, c.k, c.v, out, ws)
        with pytest.raises(ValueError, match="ws with strides"):
            moe.moe_attn_prompt(c.attn, c.q, c.q[:, :2], c.q[:, :2], c.cu, out, ws)


def test_one_row_with_heads_far_apart():
    """The strides of an axis of length one are not looked at, whatever the other's: heads 2^35 + 8 elements apart."""
    apart, d = 2 ** 35 + 8, 64
    attn = moe.Attention(2, 2, d, 16, 1, 1)
    x = torch.empty(apart + 3 * d, dtype=torch.bfloat16, device=DEV)
    views = [x[i * d:].as_strided((1, 2, d), (1, apart, 1), x.storage_offset() + i * d) for i in range(3)]
    for i, t in enumerate(views):
        t.copy_(torch.randn((1, 2, d), device=DEV) + i)
    q, k, v = views
    out, cu = torch.empty((1, 2, d), dtype=torch.bfloat16, device=DEV), torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    moe.moe_attn_prompt(attn, q, k, v, cu, out, moe.alloc_attn_workspace(attn, 1, 1))
    assert torch.equal(out, v)                                     # one token sees itself alone
    kc, vc = (torch.zeros(attn.cache_shape, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    moe.moe_kv_append(attn, k, v, torch.tensor([5], dtype=torch.int32, device=DEV), kc, vc)
    assert torch.equal(kc[0, :, 5], k[0]) and torch.equal(vc[0, :, 5], v[0]) and (kc[0, :, :5] == 0).all()
    table, cached = torch.zeros((1, 1), dtype=torch.int32, device=DEV), torch.tensor([5], dtype=torch.int32, device=DEV)
    moe.moe_attn_tree(attn, q, cu, cached, table, kc, vc, out, moe.alloc_attn_workspace(attn, 1, 1),
                      tree_mask=torch.zeros(1, dtype=torch.int64, device=DEV))
    assert torch.isfinite(out).all()
    del x, views, q, k, v, t
    torch.cuda.empty_cache()                                       # 64 GB
