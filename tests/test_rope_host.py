"""Rotary positions without a GPU: the handle's frequencies and what it refuses."""
import ctypes
import math
import shutil

import pytest
import torch

import rope_ref as ref
from quantized_moe_expert_router_gb300 import build, moe

SCALINGS = {"plain": {}, "linear": dict(factor=4.0), "base": dict(factor=8.0),
            "yarn": dict(factor=32.0, original=4096, low=1.0, high=32.0), "bands": dict(factor=8.0, original=8192, low=1.0, high=4.0)}
KIND = {"plain": 0, "linear": 1, "base": 2, "yarn": 3, "bands": 4}


@pytest.fixture(scope="module", autouse=True)
def built():
    if shutil.which(build.NVCC) is None:
        pytest.skip("nvcc not found")
    build.build()


@pytest.mark.parametrize("scaling", sorted(SCALINGS))
@pytest.mark.parametrize("dims,theta", [(16, 10000.0), (64, 50000.0), (128, 500000.0), (256, 1e6), (48, 2.0)])
def test_frequencies(scaling, dims, theta):
    r = moe.Rope(dims, theta, scaling=KIND[scaling], **SCALINGS[scaling])
    want = ref.frequencies(dims, theta, scaling, **SCALINGS[scaling])
    got = torch.tensor(moe.moe_rope_frequencies(r), dtype=torch.float64)
    # a power, a logarithm's ramp and a quotient, each of some 2^-52
    assert got.shape == want.shape and ((got - want).abs() <= 2.0 ** -48 * want).all()


def test_frequencies_by_hand():
    f = moe.moe_rope_frequencies(moe.Rope(16, 256.0))
    assert f == pytest.approx([1.0, 0.5, 0.25, 0.125, 0.0625, 0.03125, 0.015625, 0.0078125], rel=1e-14)
    f = moe.moe_rope_frequencies(moe.Rope(16, 256.0, scaling=moe.ROPE_BANDS, factor=2.0, original=16, low=1.0, high=2.0))
    s = 16 * 0.5 / (2 * math.pi) - 1                  # pair 1 makes 1.27 turns over the original context
    assert f[0] == pytest.approx(1.0) and f[7] == pytest.approx(0.0078125 / 2)
    assert f[1] == pytest.approx(0.5 * (s + (1 - s) / 2))


def test_yarn_ends_by_hand():
    """original = 2 pi 256 and theta = 256 over 16 elements: d(t) = 8 (1 - ln t / ln 256), so 16 turns at pair 4 and 1 at pair 8."""
    r = moe.Rope(16, 256.0, scaling=moe.ROPE_YARN, factor=4.0, original=1608, low=1.0, high=16.0)
    plain = moe.moe_rope_frequencies(moe.Rope(16, 256.0))
    got = [a / b for a, b in zip(moe.moe_rope_frequencies(r), plain)]
    assert got[:4] == pytest.approx([1.0] * 4)         # d(16) is just under 4: the ramp starts at pair 3
    assert got[4] == pytest.approx(1 - 0.75 / 5) and got[7] == pytest.approx(1 - 0.75 * 4 / 5)


@pytest.mark.parametrize("kw,status", [
    (dict(dims=8), 2), (dict(dims=24), 2), (dict(dims=272), 2), (dict(layout=2), 1), (dict(scaling=5), 1), (dict(scaling=-1), 1),
    (dict(theta=1.0), 1), (dict(theta=math.nan), 1), (dict(theta=math.inf), 1), (dict(attn_factor=0.0), 1), (dict(attn_factor=math.nan), 1),
    (dict(scaling=1, factor=0.5), 1), (dict(scaling=2, factor=math.inf), 1), (dict(scaling=3, factor=2.0, original=0), 1),
    (dict(scaling=3, factor=2.0, original=64, low=4.0, high=4.0), 1), (dict(scaling=4, factor=2.0, original=64, low=0.0, high=4.0), 1),
    (dict(scaling=4, factor=math.nan, original=64, low=1.0, high=4.0), 1),
])
def test_create_refuses(kw, status):
    with pytest.raises(moe.MoEError) as e:
        moe.Rope(**{**dict(dims=64), **kw})
    assert e.value.status == status


def test_create_refuses_other_types_and_flags():
    with pytest.raises(TypeError):
        moe.Rope(64, dtype=torch.float32)
    lib, out = moe.load_library(), ctypes.c_void_p()
    cfg = moe.moe_rope_config(64, 0, 0, 2, 10000.0, 1.0, 1.0, 32.0, 0, 1.0, 0)
    assert lib.moe_rope_create(ctypes.byref(cfg), 0, ctypes.byref(out)) == 1
    cfg.dtype, cfg.flags = 0, 1
    assert lib.moe_rope_create(ctypes.byref(cfg), 0, ctypes.byref(out)) == 1
    cfg.flags = 0
    assert lib.moe_rope_create(ctypes.byref(cfg), -1, ctypes.byref(out)) == 1 and lib.moe_rope_create(None, 0, ctypes.byref(out)) == 1
    assert not out.value and lib.moe_rope_destroy(None) == 0 and lib.moe_rope_frequencies(None, None) == 1


def test_null_and_negative_arguments_are_refused():
    lib, r = moe.load_library(), moe.Rope(64)
    rows = moe._pack_rows(16, 64, 64)
    assert lib.moe_rope_apply(None, 1, 64, 16, 1, rows, rows, 0, None, None, None) == 1
    assert lib.moe_rope_apply(r.handle, -1, 64, 16, 1, rows, rows, 0, None, None, None) == 1
    assert lib.moe_rope_apply(r.handle, 1, 64, None, 1, rows, rows, 0, None, None, None) == 1
    assert lib.moe_rope_apply(r.handle, 1, 48, 16, 1, rows, rows, 0, None, None, None) == 2
    assert lib.moe_rope_apply(r.handle, 1, 72, 16, 1, rows, rows, 0, None, None, None) == 2
    assert lib.moe_rope_apply(r.handle, 1, 1040, 16, 1, rows, rows, 0, None, None, None) == 2
    assert lib.moe_rope_apply(r.handle, 1, 64, 16, 1025, rows, rows, 0, None, None, None) == 2
    assert lib.moe_rope_apply(r.handle, 2 ** 20 + 1, 64, 16, 1, rows, rows, 0, None, None, None) == 2
    assert lib.moe_rope_apply(r.handle, 1, 64, 16, 1, rows, None, 0, None, None, None) == 1
    assert lib.moe_rope_apply(r.handle, 1, 64, 16, 1, rows, rows, 1, rows, None, None) == 1
    assert lib.moe_rope_apply(r.handle, 2, 64, 16, 1, moe._pack_rows(16, 60, 64), rows, 0, None, None, None) == 1
    assert lib.moe_rope_apply(r.handle, 1, 64, 16, 1, moe._pack_rows(24, 64, 64), rows, 0, None, None, None) == 1
    assert lib.moe_rope_apply(r.handle, 0, 64, None, 1, None, None, 0, None, None, None) == 0
    assert lib.moe_rope_append(None, r.handle, 1, 16, 16, rows, rows, rows, rows, 16, 16, None) == 1
    assert lib.moe_latent_append(None, r.handle, 1, 16, 16, rows, rows, None, None, None, 16, None) == 1


@pytest.mark.parametrize("kw,status", [
    (dict(heads=0), 2), (dict(heads=129), 2), (dict(latent_dim=256), 2), (dict(rope_dim=32), 2), (dict(head_dim=64), 2),
    (dict(page_size=8), 2), (dict(page_size=48), 2), (dict(page_size=256), 2), (dict(num_pages=0), 2), (dict(max_pages=0), 2),
    (dict(num_pages=2 ** 27), 2), (dict(max_pages=2 ** 27), 2), (dict(dtype=2), 1), (dict(softmax_scale=0.0), 1),
    (dict(softmax_scale=math.nan), 1), (dict(softmax_scale=-1.0), 1), (dict(softmax_scale=1e-31), 1), (dict(softmax_scale=1e31), 1),
    (dict(flags=1), 1), (dict(flags=0x80000001), 1),
])
def test_latent_create_refuses(kw, status):
    cfg = moe.moe_latent_config(**{**dict(heads=16, latent_dim=512, rope_dim=64, head_dim=128, page_size=16, num_pages=64, max_pages=8,
                                          dtype=0, softmax_scale=0.1, flags=0), **kw})
    lib, out = moe.load_library(), ctypes.c_void_p()
    assert lib.moe_latent_create(ctypes.byref(cfg), 0, ctypes.byref(out)) == status and not out.value
    assert lib.moe_latent_create(None, 0, ctypes.byref(out)) == 1 and lib.moe_latent_destroy(None) == 0
