"""Host-side checks of the attention entry points, and the plain plan of
``attn_ref`` against hand-made values: no GPU needed."""
import ctypes
import math
import shutil

import numpy as np
import pytest
import torch

import attn_ref as ref
from quantized_moe_expert_router_gb300 import build, moe


@pytest.fixture(scope="module")
def lib():
    if shutil.which(build.NVCC) is None:
        pytest.skip("nvcc not found")
    build.build()
    return ctypes.CDLL(build.MOE_LIB)


@pytest.mark.parametrize("kw,status", [
    (dict(q_heads=0), 2), (dict(kv_heads=0), 2), (dict(q_heads=7), 2), (dict(q_heads=258, kv_heads=2), 2), (dict(head_dim=96), 2),
    (dict(head_dim=256), 2), (dict(page_size=8), 2), (dict(page_size=48), 2), (dict(page_size=256), 2), (dict(num_pages=0), 2),
    (dict(max_pages=0), 2), (dict(num_pages=2 ** 27), 2), (dict(max_pages=2 ** 27), 2), (dict(dtype=2), 1), (dict(softmax_scale=0.0), 1),
    (dict(softmax_scale=math.nan), 1), (dict(softmax_scale=math.inf), 1), (dict(softmax_scale=-1.0), 1), (dict(flags=1), 1),
])
def test_create_rejects_bad_configs_on_the_host(lib, kw, status):
    cfg = moe.moe_attn_config(**{**dict(q_heads=8, kv_heads=2, head_dim=128, page_size=16, num_pages=64, max_pages=8, dtype=0,
                                        softmax_scale=0.1, flags=0), **kw})
    out = ctypes.c_void_p()
    lib.moe_attn_create.argtypes = [ctypes.POINTER(moe.moe_attn_config), ctypes.c_int, ctypes.POINTER(ctypes.c_void_p)]
    assert lib.moe_attn_create(ctypes.byref(cfg), 0, ctypes.byref(out)) == status and not out.value
    assert lib.moe_attn_create(None, 0, ctypes.byref(out)) == 1


def test_null_handles_are_rejected(lib):
    n = ctypes.c_size_t()
    assert lib.moe_attn_workspace_bytes(None, 1, 1, ctypes.byref(n)) == 1
    assert lib.moe_kv_append(None, 0, None, None, None, None, None, None) == 1
    assert lib.moe_attn_prompt(None, 0, 0, None, None, None, None, None, None, None, ctypes.c_size_t(0), None) == 1
    assert lib.moe_attn_tree(None, 0, 0, None, None, None, None, None, None, None, None, None, None, ctypes.c_size_t(0), None) == 1
    assert lib.moe_attn_destroy(None) == 0


def test_reference_plan_by_hand():
    table, cu, slots, pos, words, info = ref.plan([3, 0], [2, 3], [7, 5, 4], [[2, -1], [-1, -1]], 4, 8, 6, [-1, -1, -1, 0, 0, 9])
    assert table.tolist() == [[2, 7], [5, -1]] and cu.tolist() == [0, 2, 5]
    assert slots.tolist() == [11, 28, 20, 21, 22, -1]
    assert pos.tolist() == [3, 3, 0, 1, 1, -1]
    assert words.tolist() == [1, 2, 1, 3, 5, 0] and info.tolist() == [5, 2, 5, 0]


def test_reference_attention_by_hand():
    q = torch.zeros((2, 2, 64), dtype=torch.float16)
    k = torch.zeros((3, 1, 64), dtype=torch.float16)
    v = torch.arange(3, dtype=torch.float16)[:, None, None].expand(3, 1, 64)
    vis = torch.tensor([[True, False, True], [False, False, False]])
    out, lse, bound, _ = ref.attend(q, k, v, vis, 1.0)
    assert (out[0] == 1.0).all() and (out[1] == 0.0).all()
    np.testing.assert_allclose(lse[0].numpy(), math.log(2.0))
    assert torch.isinf(lse[1]).all() and (bound[0] < 0.01).all()


def test_reference_visibility_of_words():
    vis = ref.words_to_visible(torch.tensor([1, 3, -1], dtype=torch.int64), 3)
    assert vis.tolist() == [[True, False, False], [True, True, False], [True, True, True]]
    wide = ref.words_to_visible(torch.full((70,), -1, dtype=torch.int64), 70)
    assert wide[:, :64].all() and not wide[:, 64:].any()


def test_reference_roundoff_is_that_of_the_types():
    """The largest relative error of rounding 1 + x, x in [0, 1], is u / (1 + u)."""
    x = 1 + torch.arange(2 ** 16, dtype=torch.float64) / 2 ** 16
    for dt, u in ref.U.items():
        err = ((x.to(dt).double() - x) / x).abs().max()
        assert abs(float(err) - u / (1 + u)) < 1e-4 * u


@pytest.mark.parametrize("flags", [0x80000001, 0x40000000])
def test_create_knows_one_flag(lib, flags):
    cfg = moe.moe_attn_config(8, 2, 128, 16, 64, 8, 0, 0.1, flags)
    out = ctypes.c_void_p()
    lib.moe_attn_create.argtypes = [ctypes.POINTER(moe.moe_attn_config), ctypes.c_int, ctypes.POINTER(ctypes.c_void_p)]
    assert lib.moe_attn_create(ctypes.byref(cfg), 0, ctypes.byref(out)) == 1 and not out.value
