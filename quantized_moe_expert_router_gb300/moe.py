"""Thin ctypes binding of the C ABI in include/moe.h (argument marshalling only).

Every function here has the name of the C entry point it calls.  Tensors are
torch tensors on the layer's CUDA device (PyTorch is used for device memory
and streams only); the computation runs in the library's kernels.  The module
raises if ``_lib/libmoe.so`` is missing: there is no CPU or PyTorch fallback.
"""
from __future__ import annotations

import ctypes
import math
import os
import struct
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_lib", "libmoe.so")

MOE_OK = 0
STATUS_NAMES = {
    0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED_SHAPE",
    3: "MOE_ERR_INVALID_VALUE", 4: "MOE_ERR_WORKSPACE_TOO_SMALL",
    5: "MOE_ERR_OUT_OF_MEMORY", 6: "MOE_ERR_CUDA", 7: "MOE_ERR_DEVICE_TIMEOUT",
    8: "MOE_ERR_BAD_EXPERT_ID",
}
FLAG_BAD_EXPERT_ID = 0x1
FLAG_DUPLICATE_ID = 0x2
FLAG_TIMEOUT = 0x4
CONFIG_TEST_ROUTER_STALL = 0x80000000   # test hook: the router's bounded wait runs out
CONFIG_MXFP4 = 0x1                      # MXFP4 weights (e8m0 scale per 32 elements)
CONFIG_GROUPED_ABOVE_8 = 0x2            # the grouped tcgen05 path for every call of more than 8 tokens
CONFIG_W4A4 = 0x4                       # activations quantized to NVFP4 with each matrix's input scale
ACT_BF16, ACT_F32 = 0, 1                # source types of moe_quantize_nvfp4
ATTN_BF16, ATTN_F16 = 0, 1              # element types of an Attention
ATTN_TEST_STALL = 0x80000000            # test hook: the attention's bounded waits run out
KV_FLAG_LENGTH = 0x1                    # moe_kv_plan's info[3]: a negative length, or more rows than given
KV_FLAG_TABLE = 0x2                     # a context longer than a block-table row
KV_FLAG_PAGES = 0x4                     # free pages ran out, or a page id is out of range
KV_FLAG_TREE = 0x8                      # a bad parent, or a tree of more than 64 rows

EXPORTED = (
    "moe_layer_create", "moe_layer_destroy", "moe_packed_bytes", "moe_workspace_bytes",
    "moe_pack_weights", "moe_route", "moe_forward", "moe_get_device_status",
    "moe_set_stage_events", "moe_route_noalloc", "moe_route_forward",
    "moe_ffn_create", "moe_ffn_destroy", "moe_ffn_packed_bytes", "moe_ffn_workspace_bytes",
    "moe_ffn_pack_weights", "moe_ffn_partial", "moe_ffn_finish", "moe_ffn_forward", "moe_quantize_nvfp4",
    "moe_attn_create", "moe_attn_destroy", "moe_attn_workspace_bytes", "moe_kv_plan", "moe_kv_append",
    "moe_attn_prompt", "moe_attn_tree", "moe_attn_get_device_status",
    "moe_status_string",
)


class MoEError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} failed: {STATUS_NAMES.get(status, status)}")


class moe_config(ctypes.Structure):
    _fields_ = [("num_experts", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("hidden", ctypes.c_int32), ("intermediate", ctypes.c_int32),
                ("max_tokens", ctypes.c_int32), ("flags", ctypes.c_uint32)]


class moe_fp4_tensor(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("global_scale", ctypes.c_void_p), ("input_scale", ctypes.c_void_p)]


class moe_canonical_weights(ctypes.Structure):
    _fields_ = [("gate", moe_fp4_tensor), ("up", moe_fp4_tensor), ("down", moe_fp4_tensor)]


class moe_ffn_config(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("shared_experts", ctypes.c_int32),
                ("shared_intermediate", ctypes.c_int32), ("eps", ctypes.c_float), ("flags", ctypes.c_uint32)]


class moe_ffn_weights(ctypes.Structure):
    _fields_ = [("routed_down", moe_fp4_tensor), ("routed_up", moe_fp4_tensor),
                ("shared", moe_canonical_weights), ("norm_gamma", ctypes.c_void_p)]


class moe_attn_config(ctypes.Structure):
    _fields_ = [("q_heads", ctypes.c_int32), ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("num_pages", ctypes.c_int32), ("max_pages", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("softmax_scale", ctypes.c_float), ("flags", ctypes.c_uint32)]


_lock = threading.Lock()
_lib = None


def load_library(path: str = LIB_PATH):
    """Load libmoe.so (built by ``build.build()``); raise if it is absent."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(path):
                raise RuntimeError(f"{path} is missing: run quantized_moe_expert_router_gb300.build.build() "
                                   "(there is no CPU fallback)")
            lib = ctypes.CDLL(path)
            P, I32, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
            lib.moe_layer_create.argtypes = [ctypes.POINTER(moe_config), I32, ctypes.POINTER(P)]
            lib.moe_layer_destroy.argtypes = [P]
            lib.moe_packed_bytes.argtypes = [P, ctypes.POINTER(SZ)]
            lib.moe_workspace_bytes.argtypes = [P, I32, ctypes.POINTER(SZ)]
            lib.moe_pack_weights.argtypes = [P, ctypes.POINTER(moe_canonical_weights), P, P]
            lib.moe_route.argtypes = [P, P, I32, P, P, P, P, P, SZ, P]
            lib.moe_forward.argtypes = [P, P, I32, P, P, P, P, P, SZ, P]
            lib.moe_get_device_status.argtypes = [P, P, P, ctypes.POINTER(ctypes.c_int32)]
            lib.moe_set_stage_events.argtypes = [P, P, I32]
            lib.moe_route_noalloc.argtypes = [P, P, I32, P, P, P, P, P]
            lib.moe_route_forward.argtypes = [P, P, I32, P, P, P, P, P, P, P, SZ, P]
            lib.moe_ffn_create.argtypes = [ctypes.POINTER(moe_ffn_config), P, ctypes.POINTER(P)]
            lib.moe_ffn_destroy.argtypes = [P]
            lib.moe_ffn_packed_bytes.argtypes = [P, ctypes.POINTER(SZ)]
            lib.moe_ffn_workspace_bytes.argtypes = [P, I32, ctypes.POINTER(SZ)]
            lib.moe_ffn_pack_weights.argtypes = [P, ctypes.POINTER(moe_ffn_weights), P, P]
            lib.moe_ffn_partial.argtypes = [P, P, I32, P, P, P, P, P, P, P, P, SZ, P]
            lib.moe_ffn_finish.argtypes = [P, P, I32, P, P, P, P, SZ, P]
            lib.moe_ffn_forward.argtypes = [P, P, I32, P, P, P, P, P, P, P, P, SZ, P]
            lib.moe_quantize_nvfp4.argtypes = [P, I32, ctypes.c_int64, I32, ctypes.c_float, P, P, P]
            R = P                                    # a moe_attn_rows, as bytes
            lib.moe_attn_create.argtypes = [ctypes.POINTER(moe_attn_config), I32, ctypes.POINTER(P)]
            lib.moe_attn_destroy.argtypes = [P]
            lib.moe_attn_workspace_bytes.argtypes = [P, I32, I32, ctypes.POINTER(SZ)]
            lib.moe_kv_plan.argtypes = [P, I32, I32, P, P, P, I32, P, P, P, P, P, P, P, P]
            lib.moe_kv_append.argtypes = [P, I32, R, R, P, P, P, P]
            lib.moe_attn_prompt.argtypes = [P, I32, I32, R, R, R, P, R, P, P, SZ, P]
            lib.moe_attn_tree.argtypes = [P, I32, I32, R, P, P, P, P, P, P, R, P, P, SZ, P]
            lib.moe_attn_get_device_status.argtypes = [P, P, P, ctypes.POINTER(ctypes.c_int32)]
            lib.moe_status_string.argtypes = [I32]
            lib.moe_status_string.restype = ctypes.c_char_p
            for name in EXPORTED[:-1]:
                getattr(lib, name).restype = I32
            _lib = lib
    return _lib


def _check(fn, status):
    if status != MOE_OK:
        raise MoEError(fn, status)


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


class Layer:
    """Owns one ``moe_layer_t`` handle (host memory only)."""

    def __init__(self, num_experts, top_k, hidden, intermediate, max_tokens, device=0, flags=0):
        lib = load_library()
        self.cfg = moe_config(num_experts, top_k, hidden, intermediate, max_tokens, flags)
        self.device = device
        h = ctypes.c_void_p()
        _check("moe_layer_create", lib.moe_layer_create(ctypes.byref(self.cfg), device, ctypes.byref(h)))
        self.handle = h

    def close(self):
        if getattr(self, "handle", None) is not None and _lib is not None:
            _lib.moe_layer_destroy(self.handle)
            self.handle = None

    def __del__(self):
        self.close()


def moe_layer_create(num_experts, top_k, hidden, intermediate, max_tokens, device=0) -> Layer:
    return Layer(num_experts, top_k, hidden, intermediate, max_tokens, device)


def moe_layer_destroy(layer: Layer) -> None:
    layer.close()


def moe_packed_bytes(layer: Layer) -> int:
    n = ctypes.c_size_t()
    _check("moe_packed_bytes", load_library().moe_packed_bytes(layer.handle, ctypes.byref(n)))
    return n.value


def moe_workspace_bytes(layer: Layer, num_tokens: int) -> int:
    n = ctypes.c_size_t()
    _check("moe_workspace_bytes", load_library().moe_workspace_bytes(layer.handle, num_tokens, ctypes.byref(n)))
    return n.value


def _fp4(m):
    return moe_fp4_tensor(_ptr(m["codes"]), _ptr(m["scales"]), _ptr(m["g"]), _ptr(m["a"]))


def moe_pack_weights(layer: Layer, canon: dict, packed: torch.Tensor, stream=None) -> None:
    """canon: {'gate'|'up'|'down': {'codes','scales','g','a'}} device tensors."""
    cw = moe_canonical_weights(_fp4(canon["gate"]), _fp4(canon["up"]), _fp4(canon["down"]))
    _check("moe_pack_weights", load_library().moe_pack_weights(
        layer.handle, ctypes.byref(cw), _ptr(packed), _stream(stream)))


def moe_route(layer, x, num_tokens, w_router, bias, ids, weights, ws, stream=None) -> None:
    _check("moe_route", load_library().moe_route(
        layer.handle, _ptr(x), num_tokens, _ptr(w_router), _ptr(bias), _ptr(ids), _ptr(weights),
        _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def moe_forward(layer, x, num_tokens, ids, weights, packed, y, ws, stream=None) -> None:
    _check("moe_forward", load_library().moe_forward(
        layer.handle, _ptr(x), num_tokens, _ptr(ids), _ptr(weights), _ptr(packed), _ptr(y),
        _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def moe_route_forward(layer, x, num_tokens, w_router, bias, packed, ids, weights, y, ws, stream=None) -> None:
    """The whole layer: routing then the routed experts (ids/weights written)."""
    _check("moe_route_forward", load_library().moe_route_forward(
        layer.handle, _ptr(x), num_tokens, _ptr(w_router), _ptr(bias), _ptr(packed), _ptr(ids),
        _ptr(weights), _ptr(y), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def moe_route_noalloc(layer, x, num_tokens, w_router, bias, ids, weights, stream=None) -> None:
    """moe_route for callers that cannot allocate a workspace: the router's
    scratch lives in a fixed array inside the library (C <= 8 tokens).  Calls
    that overlap on the GPU share that array and race; the first call on a
    device must happen outside stream capture."""
    _check("moe_route_noalloc", load_library().moe_route_noalloc(
        layer.handle, _ptr(x), num_tokens, _ptr(w_router), _ptr(bias), _ptr(ids), _ptr(weights),
        _stream(stream)))


def moe_get_device_status(layer, ws, stream=None) -> int:
    f = ctypes.c_int32()
    _check("moe_get_device_status", load_library().moe_get_device_status(
        layer.handle, _ptr(ws), _stream(stream), ctypes.byref(f)))
    return f.value


def moe_set_stage_events(layer, events) -> None:
    lib = load_library()
    if events is None:
        _check("moe_set_stage_events", lib.moe_set_stage_events(layer.handle, None, 0))
        return
    arr = (ctypes.c_void_p * len(events))(*[e.cuda_event for e in events])
    layer._stage_events = (events, arr)      # keep alive
    _check("moe_set_stage_events", lib.moe_set_stage_events(layer.handle, arr, len(events)))


def moe_quantize_nvfp4(src: torch.Tensor, a: float, codes: torch.Tensor, scales: torch.Tensor, stream=None) -> None:
    """NVFP4 quantization of src [rows][n] (torch.bfloat16, or uint16 bf16
    bits, or torch.float32) with input scale a into codes uint8 [rows][n/2]
    and scales uint8 [rows][n/16] (device tensors)."""
    dtype = ACT_F32 if src.dtype == torch.float32 else ACT_BF16
    if src.dtype not in (torch.float32, torch.bfloat16, torch.uint16, torch.int16):
        raise TypeError(f"moe_quantize_nvfp4: unsupported source dtype {src.dtype}")
    n = src.shape[-1]
    rows = src.numel() // n if n else 0
    _check("moe_quantize_nvfp4", load_library().moe_quantize_nvfp4(
        _ptr(src), dtype, rows, n, float(a), _ptr(codes), _ptr(scales), _stream(stream)))


def moe_status_string(status: int) -> str:
    return load_library().moe_status_string(status).decode()


# ------------------------------------------------------------ conveniences

def alloc_workspace(layer: Layer, num_tokens: int, device=None) -> torch.Tensor:
    """Zero-filled workspace (uint8) of moe_workspace_bytes(num_tokens)."""
    n = moe_workspace_bytes(layer, num_tokens)
    return torch.zeros(n, dtype=torch.uint8, device=device or f"cuda:{layer.device}")


def alloc_packed(layer: Layer, device=None) -> torch.Tensor:
    return torch.empty(moe_packed_bytes(layer), dtype=torch.uint8, device=device or f"cuda:{layer.device}")


# ------------------------------------------------ the FFN around the routed sum

class Ffn:
    """Owns one ``moe_ffn_t`` handle tied to a routed ``Layer`` (host memory only)."""

    def __init__(self, routed: Layer, hidden, shared_experts, shared_intermediate, eps=1e-6):
        lib = load_library()
        self.routed = routed
        self.cfg = moe_ffn_config(hidden, shared_experts, shared_intermediate, eps, 0)
        h = ctypes.c_void_p()
        _check("moe_ffn_create", lib.moe_ffn_create(ctypes.byref(self.cfg), routed.handle, ctypes.byref(h)))
        self.handle = h

    def close(self):
        if getattr(self, "handle", None) is not None and _lib is not None:
            _lib.moe_ffn_destroy(self.handle)
            self.handle = None

    def __del__(self):
        self.close()


def moe_ffn_packed_bytes(ffn: Ffn) -> int:
    n = ctypes.c_size_t()
    _check("moe_ffn_packed_bytes", load_library().moe_ffn_packed_bytes(ffn.handle, ctypes.byref(n)))
    return n.value


def moe_ffn_workspace_bytes(ffn: Ffn, num_tokens: int) -> int:
    n = ctypes.c_size_t()
    _check("moe_ffn_workspace_bytes", load_library().moe_ffn_workspace_bytes(ffn.handle, num_tokens, ctypes.byref(n)))
    return n.value


def _fp4_1(m):
    return moe_fp4_tensor(_ptr(m["codes"]), _ptr(m["scales"]), _ptr(m["g"]), _ptr(m["a"]))


def moe_ffn_pack_weights(ffn: Ffn, w: dict, packed: torch.Tensor, stream=None) -> None:
    """w: {'routed_down', 'routed_up': {'codes','scales','g','a'} (g, a: one-element tensors),
    'shared': {'gate'|'up'|'down': ...}, 'gamma'} device tensors."""
    sh = w["shared"]
    cw = moe_ffn_weights(_fp4_1(w["routed_down"]), _fp4_1(w["routed_up"]),
                         moe_canonical_weights(_fp4(sh["gate"]), _fp4(sh["up"]), _fp4(sh["down"])),
                         _ptr(w["gamma"]))
    _check("moe_ffn_pack_weights", load_library().moe_ffn_pack_weights(
        ffn.handle, ctypes.byref(cw), _ptr(packed), _stream(stream)))


def moe_ffn_partial(ffn, u, num_tokens, w_router, bias, routed_packed, ffn_packed, ids, weights, y_routed, ws,
                    stream=None) -> None:
    _check("moe_ffn_partial", load_library().moe_ffn_partial(
        ffn.handle, _ptr(u), num_tokens, _ptr(w_router), _ptr(bias), _ptr(routed_packed), _ptr(ffn_packed),
        _ptr(ids), _ptr(weights), _ptr(y_routed), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def moe_ffn_finish(ffn, u, num_tokens, y_routed, ffn_packed, out, ws, stream=None) -> None:
    _check("moe_ffn_finish", load_library().moe_ffn_finish(
        ffn.handle, _ptr(u), num_tokens, _ptr(y_routed), _ptr(ffn_packed), _ptr(out), _ptr(ws),
        ws.numel() * ws.element_size(), _stream(stream)))


def moe_ffn_forward(ffn, u, num_tokens, w_router, bias, routed_packed, ffn_packed, ids, weights, out, ws,
                    stream=None) -> None:
    _check("moe_ffn_forward", load_library().moe_ffn_forward(
        ffn.handle, _ptr(u), num_tokens, _ptr(w_router), _ptr(bias), _ptr(routed_packed), _ptr(ffn_packed),
        _ptr(ids), _ptr(weights), _ptr(out), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def alloc_ffn_workspace(ffn: Ffn, num_tokens: int, device=None) -> torch.Tensor:
    n = moe_ffn_workspace_bytes(ffn, num_tokens)
    return torch.zeros(n, dtype=torch.uint8, device=device or f"cuda:{ffn.routed.device}")


def alloc_ffn_packed(ffn: Ffn, device=None) -> torch.Tensor:
    return torch.empty(moe_ffn_packed_bytes(ffn), dtype=torch.uint8, device=device or f"cuda:{ffn.routed.device}")


# ------------------------------------------------ the attention beside the FFN

class Attention:
    """Owns one ``moe_attn_t`` handle (host memory only): the geometry of the
    heads and of the paged cache, [num_pages][kv_heads][page_size][head_dim]
    each for keys and values.  ``softmax_scale`` is 1 / sqrt(head_dim) unless
    given."""

    def __init__(self, q_heads, kv_heads, head_dim, page_size, num_pages, max_pages, dtype=torch.bfloat16,
                 softmax_scale=None, device=0, flags=0):
        if dtype not in (torch.bfloat16, torch.float16):
            raise TypeError(f"Attention: unsupported dtype {dtype}")
        lib = load_library()
        scale = head_dim ** -0.5 if softmax_scale is None else softmax_scale
        self.cfg = moe_attn_config(q_heads, kv_heads, head_dim, page_size, num_pages, max_pages,
                                   ATTN_F16 if dtype == torch.float16 else ATTN_BF16, scale, flags)
        self.dtype, self.device = dtype, device
        self.q_heads, self.kv_heads, self.head_dim, self.max_pages = q_heads, kv_heads, head_dim, max_pages
        self.cache_shape = (num_pages, kv_heads, page_size, head_dim)
        h = ctypes.c_void_p()
        _check("moe_attn_create", lib.moe_attn_create(ctypes.byref(self.cfg), device, ctypes.byref(h)))
        self.handle = h

    def close(self):
        if getattr(self, "handle", None) is not None and _lib is not None:
            _lib.moe_attn_destroy(self.handle)
            self.handle = None

    def __del__(self):
        self.close()


def moe_attn_workspace_bytes(attn: Attention, num_requests: int, num_rows: int) -> int:
    n = ctypes.c_size_t()
    _check("moe_attn_workspace_bytes", load_library().moe_attn_workspace_bytes(
        attn.handle, num_requests, num_rows, ctypes.byref(n)))
    return n.value


def alloc_attn_workspace(attn: Attention, num_requests: int, num_rows: int, device=None) -> torch.Tensor:
    """Zero-filled workspace (uint8) of moe_attn_workspace_bytes."""
    n = moe_attn_workspace_bytes(attn, num_requests, num_rows)
    return torch.zeros(n, dtype=torch.uint8, device=device or f"cuda:{attn.device}")


def moe_attn_get_device_status(attn: Attention, ws: torch.Tensor, stream=None) -> int:
    fn, f = "moe_attn_get_device_status", ctypes.c_int32()
    if ws.get_device() != attn.device or not ws.is_contiguous() or ws.nbytes < moe_attn_workspace_bytes(attn, 0, 0):
        raise ValueError(f"{fn}: ws of {ws.nbytes} bytes on {ws.device} is not a workspace on cuda:{attn.device}")
    _check(fn, load_library().moe_attn_get_device_status(
        attn.handle, ws.data_ptr(), _stream(torch.cuda.current_stream(attn.device) if stream is None else stream), ctypes.byref(f)))
    return f.value


# The calls below run once or more per step and layer, so what they look at is
# written out: dtype, number of elements, contiguity and device of each array, in
# one condition.  What went wrong is found out only then (_attn_refuse).

_pack_rows = struct.Struct("@Pqq").pack         # a moe_attn_rows


def _attn_refuse(fn, dev, *arrays):
    """Raise for the first of (name, tensor, dtype, shape) that is not a contiguous tensor like that on cuda:dev."""
    for name, t, dtype, shape in arrays:
        if t is None:
            continue
        if t.dtype is not dtype:
            raise TypeError(f"{fn}: {name} is {t.dtype}, not {dtype}")
        if t.numel() != math.prod(shape) or not t.is_contiguous() or t.get_device() != dev:
            raise ValueError(f"{fn}: {name} of shape {tuple(t.shape)} on {t.device} is not a contiguous {shape} on cuda:{dev}")


def _attn_ws(fn, dev, ws):
    if ws.get_device() != dev:
        raise ValueError(f"{fn}: ws is on {ws.device}, not on cuda:{dev}")
    if not ws.is_contiguous():
        raise ValueError(f"{fn}: ws with strides {ws.stride()} is not contiguous")


def _attn_rows(fn, name, attn, t, shape):
    """The moe_attn_rows of [rows][heads][head_dim] with a contiguous last axis and any strides of the others."""
    s = t.stride()
    if t.dtype is attn.dtype and t.shape == shape and s[2] == 1 and t.get_device() == attn.device:
        return _pack_rows(t.data_ptr(), s[0], s[1])
    if t.dtype is not attn.dtype:
        raise TypeError(f"{fn}: {name} is {t.dtype}, not {attn.dtype}")
    raise ValueError(f"{fn}: {name} of shape {tuple(t.shape)}, strides {s}, on {t.device} is not {shape} with a contiguous "
                     f"last axis on cuda:{attn.device}")


def _attn_caches(fn, attn, k_cache, v_cache):
    dt, shape, dev = attn.dtype, attn.cache_shape, attn.device
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        if t.dtype is not dt:
            raise TypeError(f"{fn}: {name} is {t.dtype}, not {dt}")
        if t.shape != shape or not t.is_contiguous() or t.get_device() != dev:
            raise ValueError(f"{fn}: {name} of shape {tuple(t.shape)} on {t.device} is not a contiguous {shape} on cuda:{dev}")


def moe_kv_plan(attn, cached, fresh, free_pages, block_table, cu, slots, positions, info, parents=None, tree_mask=None,
                stream=None) -> None:
    """Block table entries, row offsets, slots, positions and (from parents)
    tree masks of one step; int32 tensors, tree_mask int64."""
    dev, i32, B, T, F = attn.device, torch.int32, cached.numel(), slots.numel(), free_pages.numel()
    if (cached.dtype is not i32 or not cached.is_contiguous() or cached.get_device() != dev
            or fresh.dtype is not i32 or fresh.numel() != B or not fresh.is_contiguous() or fresh.get_device() != dev
            or free_pages.dtype is not i32 or not free_pages.is_contiguous() or free_pages.get_device() != dev
            or block_table.dtype is not i32 or block_table.shape != (B, attn.max_pages) or not block_table.is_contiguous()
            or block_table.get_device() != dev
            or cu.dtype is not i32 or cu.numel() != B + 1 or not cu.is_contiguous() or cu.get_device() != dev
            or slots.dtype is not i32 or not slots.is_contiguous() or slots.get_device() != dev
            or positions.dtype is not i32 or positions.numel() != T or not positions.is_contiguous() or positions.get_device() != dev
            or info.dtype is not i32 or info.numel() != 4 or not info.is_contiguous() or info.get_device() != dev
            or parents is not None and (parents.dtype is not i32 or parents.numel() != T or not parents.is_contiguous()
                                        or parents.get_device() != dev)
            or tree_mask is not None and (tree_mask.dtype is not torch.int64 or tree_mask.numel() != T
                                          or not tree_mask.is_contiguous() or tree_mask.get_device() != dev)):
        _attn_refuse("moe_kv_plan", dev, ("cached", cached, i32, (B,)), ("fresh", fresh, i32, (B,)), ("free_pages", free_pages, i32, (F,)),
                     ("block_table", block_table, i32, (B, attn.max_pages)), ("cu", cu, i32, (B + 1,)), ("slots", slots, i32, (T,)),
                     ("positions", positions, i32, (T,)), ("info", info, i32, (4,)), ("parents", parents, i32, (T,)),
                     ("tree_mask", tree_mask, torch.int64, (T,)))
        raise ValueError(f"moe_kv_plan: block_table has shape {tuple(block_table.shape)}, not {(B, attn.max_pages)}")
    status = _lib.moe_kv_plan(
        attn.handle, B, T, cached.data_ptr(), fresh.data_ptr(), free_pages.data_ptr(), F,
        None if parents is None else parents.data_ptr(), block_table.data_ptr(), cu.data_ptr(), slots.data_ptr(),
        positions.data_ptr(), None if tree_mask is None else tree_mask.data_ptr(), info.data_ptr(),
        torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream)
    if status:
        _check("moe_kv_plan", status)


def moe_kv_append(attn, k, v, slots, k_cache, v_cache, stream=None) -> None:
    """Write k and v rows [rows][kv_heads][head_dim] to their slots (negative: skipped)."""
    fn, dev, dt, T = "moe_kv_append", attn.device, attn.dtype, slots.numel()
    shape, cs = (T, attn.kv_heads, attn.head_dim), attn.cache_shape
    if slots.dtype is not torch.int32 or not slots.is_contiguous() or slots.get_device() != dev:
        _attn_refuse(fn, dev, ("slots", slots, torch.int32, (T,)))
    if (k_cache.dtype is not dt or k_cache.shape != cs or not k_cache.is_contiguous() or k_cache.get_device() != dev
            or v_cache.dtype is not dt or v_cache.shape != cs or not v_cache.is_contiguous() or v_cache.get_device() != dev):
        _attn_caches(fn, attn, k_cache, v_cache)
    status = _lib.moe_kv_append(
        attn.handle, T, _attn_rows(fn, "k", attn, k, shape), _attn_rows(fn, "v", attn, v, shape), slots.data_ptr(),
        k_cache.data_ptr(), v_cache.data_ptr(),
        torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream)
    if status:
        _check(fn, status)


def moe_attn_prompt(attn, q, k, v, cu, out, ws, lse=None, stream=None) -> None:
    """Causal attention over packed prompts: q, out [rows][q_heads][head_dim],
    k, v [rows][kv_heads][head_dim], cu int32 [requests + 1], lse fp32
    [rows][q_heads]."""
    fn, dev, T, n = "moe_attn_prompt", attn.device, q.shape[0], cu.numel()
    hq = attn.q_heads
    qs, ks = (T, hq, attn.head_dim), (T, attn.kv_heads, attn.head_dim)
    if (cu.dtype is not torch.int32 or not cu.is_contiguous() or cu.get_device() != dev
            or ws.get_device() != dev or not ws.is_contiguous()
            or lse is not None and (lse.dtype is not torch.float32 or lse.numel() != T * hq or not lse.is_contiguous()
                                    or lse.get_device() != dev)):
        _attn_refuse(fn, dev, ("cu", cu, torch.int32, (n,)), ("lse", lse, torch.float32, (T, hq)))
        _attn_ws(fn, dev, ws)
    status = _lib.moe_attn_prompt(
        attn.handle, n - 1, T, _attn_rows(fn, "q", attn, q, qs), _attn_rows(fn, "k", attn, k, ks),
        _attn_rows(fn, "v", attn, v, ks), cu.data_ptr(), _attn_rows(fn, "out", attn, out, qs),
        None if lse is None else lse.data_ptr(), ws.data_ptr(), ws.nbytes,
        torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream)
    if status:
        _check(fn, status)


def moe_attn_tree(attn, q, cu, cached, block_table, k_cache, v_cache, out, ws, tree_mask=None, lse=None,
                  stream=None) -> None:
    """Attention of the step's rows over the cache: all cached tokens of the
    row's request, and its fresh rows as the row's word of tree_mask (int64)
    says, or up to the row itself without one."""
    fn, dev, i32, dt, T, n = "moe_attn_tree", attn.device, torch.int32, attn.dtype, q.shape[0], cu.numel()
    hq, cs = attn.q_heads, attn.cache_shape
    qs = (T, hq, attn.head_dim)
    if (cu.dtype is not i32 or not cu.is_contiguous() or cu.get_device() != dev
            or ws.get_device() != dev or not ws.is_contiguous()
            or cached.dtype is not i32 or cached.numel() != n - 1 or not cached.is_contiguous() or cached.get_device() != dev
            or block_table.dtype is not i32 or block_table.shape != (n - 1, attn.max_pages) or not block_table.is_contiguous()
            or block_table.get_device() != dev
            or tree_mask is not None and (tree_mask.dtype is not torch.int64 or tree_mask.numel() != T
                                          or not tree_mask.is_contiguous() or tree_mask.get_device() != dev)
            or lse is not None and (lse.dtype is not torch.float32 or lse.numel() != T * hq or not lse.is_contiguous()
                                    or lse.get_device() != dev)):
        _attn_refuse(fn, dev, ("cu", cu, i32, (n,)), ("cached", cached, i32, (n - 1,)),
                     ("block_table", block_table, i32, (n - 1, attn.max_pages)), ("tree_mask", tree_mask, torch.int64, (T,)),
                     ("lse", lse, torch.float32, (T, hq)))
        _attn_ws(fn, dev, ws)
        raise ValueError(f"{fn}: block_table has shape {tuple(block_table.shape)}, not {(n - 1, attn.max_pages)}")
    if (k_cache.dtype is not dt or k_cache.shape != cs or not k_cache.is_contiguous() or k_cache.get_device() != dev
            or v_cache.dtype is not dt or v_cache.shape != cs or not v_cache.is_contiguous() or v_cache.get_device() != dev):
        _attn_caches(fn, attn, k_cache, v_cache)
    status = _lib.moe_attn_tree(
        attn.handle, n - 1, T, _attn_rows(fn, "q", attn, q, qs), cu.data_ptr(), cached.data_ptr(), block_table.data_ptr(),
        None if tree_mask is None else tree_mask.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
        _attn_rows(fn, "out", attn, out, qs), None if lse is None else lse.data_ptr(), ws.data_ptr(), ws.nbytes,
        torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream)
    if status:
        _check(fn, status)
