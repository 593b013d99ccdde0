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
