"""Expanded latent attention over packed prompts on the GPU against its definition
in 64 bits (``latent_ref``)."""
import math

import pytest
import torch

import attn_ref
import latent_ref as ref
from quantized_moe_expert_router_gb300 import moe
from test_gpu_attn import offsets, randn

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
SCALE = 192 ** -0.5


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_moe_expert_router_gb300 import build
    build.build()
    moe.load_library()


def rows(T, heads, dt, seed):
    """q, and k, v, k_rope as parts of what a projection gives."""
    x = randn((T, heads, 256), dt, seed + 1)
    return randn((T, heads, 192), dt, seed, 1.5), x[:, :, :128], x[:, :, 128:], randn((T, 576), dt, seed + 2)[:, 512:]


def want(q, k, v, r, lengths, lo=0):
    parts = []
    for n in lengths:
        at = slice(lo, lo + n)
        vis = torch.ones((n, n), dtype=torch.bool, device=DEV).tril()
        keys = torch.cat([k[at], r[at, None].expand(n, k.shape[1], 64)], -1)
        parts.append(ref.attend(q[at], keys, v[at], vis, SCALE))
        lo += n
    return [torch.cat([p[i] for p in parts]) for i in range(4)]


def run(q, k, v, r, lengths, cu=None, out=None, lat=None, ws=None):
    T, heads = q.shape[:2]
    lat = moe.LatentAttention(heads, 16, 1, 1, q.dtype) if lat is None else lat
    ws = moe.alloc_latent_workspace(lat, len(lengths), T) if ws is None else ws
    out = torch.empty((T, heads, 128), dtype=q.dtype, device=DEV) if out is None else out
    lse = torch.empty((T, heads), dtype=torch.float32, device=DEV)
    moe.moe_latent_prompt(lat, q, k, r, v, offsets(lengths) if cu is None else cu, out, ws, lse=lse)
    assert moe.moe_latent_get_device_status(lat, ws) == 0
    return out, lse


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("heads,lengths", [
    (1, [1]), (2, [2, 1, 3]), (7, [0, 5, 0, 17, 0]), (1, [127, 128, 129]), (16, [512]), (3, [255, 256, 257, 1]), (64, [300]), (128, [130, 7]),
    (5, [511, 33]), (1, [1500]), (4, [2000, 1025, 90]), (33, [1000, 640, 385]), (16, [4096]), (9, [700] * 11),
])
def test_parity(dt, heads, lengths):
    x = rows(sum(lengths), heads, TYPES[dt], 1)
    attn_ref.check(*run(*x, lengths), want(*x, lengths))


def test_many_requests():
    lengths = [(7 * i) % 23 for i in range(1024)]
    x = rows(sum(lengths), 4, torch.bfloat16, 3)
    attn_ref.check(*run(*x, lengths), want(*x, lengths))


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("heads,dt", [(2, "bf16"), (90, "f16")])
def test_unseen_rows_have_no_effect(heads, dt, bad):
    """Rows after a row, other requests' rows and rows of no request hold anything."""
    lengths, pad0, pad1 = [130, 75, 300], 5, 40
    T = pad0 + sum(lengths) + pad1
    x = rows(T, heads, TYPES[dt], 10)
    clean = [t.clone() for t in x]
    cu = offsets(lengths) + pad0
    poisoned = []
    for b, last in enumerate([129, 60, 170]):            # from this row on, the request is poisoned
        lo = int(cu[b])
        for t in x:
            t[lo + last:lo + lengths[b]] = bad
        poisoned.append((lo, lo + last))
    for t in x:
        t[:pad0] = bad
        t[T - pad1:] = bad
    out = torch.full((T, heads, 128), 3.0, dtype=TYPES[dt], device=DEV)
    run(*x, lengths, cu=cu, out=out)
    w = want(*clean, lengths, pad0)
    for b, (lo, hi) in enumerate(poisoned):
        at = slice(lo - pad0, hi - pad0)
        attn_ref.check(out[lo:hi], None, [t[at] for t in w], f"request {b}")
        assert torch.isnan(out[hi:int(cu[b + 1])].float()).all(), "rows that see a poisoned row"
    assert (out[:pad0] == 3.0).all() and (out[T - pad1:] == 3.0).all()


def test_one_infinite_value_reaches_the_rows_that_see_it():
    heads, n, at, dt = 3, 300, 140, torch.bfloat16
    q, k, v, r = rows(n, heads, dt, 20)
    clean = v.clone()
    v[at, 1, 77] = math.inf
    out, _ = run(q, k, v, r, [n])
    w = want(q, k, clean, r, [n])
    hit = torch.zeros((n, heads, 128), dtype=torch.bool, device=DEV)
    hit[at:, 1, 77] = True
    assert (out[hit] == math.inf).all()
    attn_ref.check(torch.where(hit, 0, out), None, [torch.where(hit, 0.0, w[0]), None, w[2], None])


@pytest.mark.parametrize("n", [300, 1200])
@pytest.mark.parametrize("sign", [-1, 1])
def test_scores_thousands_of_roundings_apart(n, sign):
    """Scores of 10^33 on either side of zero: the largest that a row sees has all its weight.
    Token of rank 128 a + b: 64 keys of 2^50 (1 + a / 128) and 64 of 2^50 (1 + b / 128) by queries of
    2^56 and 2^49, integers below 2^22 times 2^92, so all sums are exact and no two alike."""
    q, k, v, r = rows(n, 2, torch.bfloat16, 60)
    rank = torch.randperm(n, generator=torch.Generator().manual_seed(61)).to(DEV)
    k = torch.cat([rank.div(128, rounding_mode="floor")[:, None].expand(n, 64), (rank % 128)[:, None].expand(n, 64)], 1)
    k = (2.0 ** 50 * (1 + k / 128.0))[:, None].expand(n, 2, 128).bfloat16().contiguous()
    q[:, :, :64], q[:, :, 64:], r = sign * 2.0 ** 56, sign * 2.0 ** 49, torch.zeros_like(r)
    out, lse = run(q, k, v, r, [n])
    at = (sign * rank).cummax(0).indices[:, None, None].expand(n, 2, 128)
    assert torch.equal(out, v.gather(0, at)) and (lse * sign > 1e32).all()


@pytest.mark.parametrize("order", ["heads_first", "gaps"])
def test_strides(order):
    heads, lengths, dt = 6, [150, 45], torch.bfloat16
    T = sum(lengths)
    if order == "heads_first":
        q, k, v = (randn((heads, T, d), dt, 5 + d).transpose(0, 1) for d in (192, 128, 120 + 8))
        o = torch.empty((heads, T, 128), dtype=dt, device=DEV).transpose(0, 1)
    else:
        q, k, v = (randn((2 * T, heads + 1, d + 8), dt, 5 + d)[::2, 1:, :d] for d in (192, 128, 128))
        o = torch.empty((T, heads, 152), dtype=dt, device=DEV)[:, :, 8:136]
    r = randn((2 * T, 72), dt, 9)[::2, 8:]
    run(q, k, v, r, lengths, out=o)
    attn_ref.check(o, None, want(q, k, v, r, lengths))


def test_repeats_bitwise_with_a_workspace_of_both_forms():
    x = rows(900, 8, torch.bfloat16, 30)
    lat = moe.LatentAttention(8, 16, 4, 4)
    ws = moe.alloc_latent_workspace(lat, 2, 900)
    a = run(*x, [700, 200], lat=lat, ws=ws)
    cache = torch.zeros(lat.cache_shape, dtype=torch.bfloat16, device=DEV)
    q = randn((2, 8, 576), torch.bfloat16, 31)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    moe.moe_latent_tree(lat, q[:, :, :512], q[:, :, 512:], ints([0, 2]), ints([30]), ints([[0, 1, 2, 3]]), cache,
                        torch.empty((2, 8, 512), dtype=torch.bfloat16, device=DEV), ws)
    b = run(*x, [700, 200], lat=lat, ws=ws)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_captured():
    x = rows(700, 16, torch.bfloat16, 32)
    lat = moe.LatentAttention(16, 16, 1, 1)
    ws, cu, out = moe.alloc_latent_workspace(lat, 2, 700), offsets([500, 200]), torch.empty((700, 16, 128), dtype=torch.bfloat16, device=DEV)
    call = lambda: moe.moe_latent_prompt(lat, x[0], x[1], x[3], x[2], cu, out, ws)  # noqa: E731
    call()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    out.zero_()
    cu.copy_(offsets([130, 333]))
    g.replay()
    torch.cuda.synchronize()
    w = want(*x, [130, 333])
    attn_ref.check(out[:463], None, w)
    assert (out[463:] == 0).all()


def test_the_two_forms_agree():
    """One layer both ways: keys and values expanded from the latents by random weights, and the weights taken into
    the query and the output.  The expanded rows are rounded to bf16, the absorbed queries too."""
    heads, n, dt = 8, 200, torch.bfloat16
    lat = moe.LatentAttention(heads, 16, 16, 16)
    c, r = randn((n, 512), dt, 40), randn((n, 64), dt, 41)
    wk, wv = (randn((heads, 128, 512), dt, 42 + i, 512 ** -0.5) for i in range(2))
    q = randn((n, heads, 192), dt, 44)
    k, v = (torch.einsum("nc,hdc->nhd", c.float(), w.float()).to(dt) for w in (wk, wv))
    ws = moe.alloc_latent_workspace(lat, 1, n)
    out = torch.empty((n, heads, 128), dtype=dt, device=DEV)
    cu = offsets([n])
    moe.moe_latent_prompt(lat, q, k, r, v, cu, out, ws)
    table = torch.arange(16, dtype=torch.int32, device=DEV).view(1, 16)
    slots = torch.arange(n, dtype=torch.int32, device=DEV)
    cache = torch.empty(lat.cache_shape, dtype=dt, device=DEV)
    moe.moe_latent_append(lat, moe.Rope(64), c, r, torch.zeros_like(slots), slots, cache)
    qa = torch.einsum("nhd,hdc->nhc", q[:, :, :128].float(), wk.float()).to(dt)
    oa = torch.empty((n, heads, 512), dtype=dt, device=DEV)
    moe.moe_latent_tree(lat, qa, q[:, :, 128:], cu, torch.zeros(1, dtype=torch.int32, device=DEV), table, cache, oa, ws)
    both = torch.einsum("nhc,hdc->nhd", oa.float(), wv.float())
    # Scores: 128 roundings of k and 512 of q K, each with a standard deviation of 2^-9 / sqrt(3) of values of about 1 and
    # 0.5, are off by 0.001 each after the scale, 0.012 together at eight of these; weights by 1.2 %, outputs by
    # twice that of the largest value.  Values and both outputs are rounded by 2^-9 each: 3.1 % in all.
    assert float((both - out.float()).abs().max()) < 0.031 * float(out.float().abs().max())


def test_a_wait_that_runs_out_is_reported():
    x = rows(300, 4, torch.bfloat16, 50)
    stalled = moe.LatentAttention(4, 16, 1, 1, flags=moe.ATTN_TEST_STALL)
    ws = moe.alloc_latent_workspace(stalled, 1, 300)
    out = torch.empty((300, 4, 128), dtype=torch.bfloat16, device=DEV)
    moe.moe_latent_prompt(stalled, x[0], x[1], x[3], x[2], offsets([300]), out, ws)
    assert moe.moe_latent_get_device_status(stalled, ws) == moe.FLAG_TIMEOUT
    attn_ref.check(*run(*x, [300], ws=ws), want(*x, [300]))


def test_refusals():
    q, k, v, r = rows(4, 2, torch.bfloat16, 60)
    lat = moe.LatentAttention(2, 16, 1, 1)
    ws, out = moe.alloc_latent_workspace(lat, 1, 4), torch.empty((4, 2, 128), dtype=torch.bfloat16, device=DEV)
    good = dict(q=q, k=k, k_rope=r, v=v, cu=offsets([4]), out=out, ws=ws)
    moe.moe_latent_prompt(lat, **good)
    for kind, kw, match in [
            (ValueError, dict(q=q[:, :, :128]), "q of shape"), (ValueError, dict(k=k[:, :, :64]), "k of shape"), (TypeError, dict(v=v.half()), "v is"),
            (ValueError, dict(k_rope=r[:3]), "k_rope of shape"), (TypeError, dict(k_rope=r.half()), "k_rope is"),
            (TypeError, dict(cu=good["cu"].long()), "cu is"), (ValueError, dict(ws=ws[::2]), "ws with strides"),
            (ValueError, dict(lse=torch.empty((4, 1), device=DEV)), "lse of shape"), (ValueError, dict(out=out.cpu()), "out of shape")]:
        with pytest.raises(kind, match=match):
            moe.moe_latent_prompt(lat, **{**good, **kw})
    with pytest.raises(moe.MoEError) as e:
        moe.moe_latent_prompt(lat, **{**good, "ws": ws[:512]})
    assert e.value.status == 4
    with pytest.raises(moe.MoEError) as e:                         # rows that overlap themselves
        moe.moe_latent_prompt(lat, **{**good, "k_rope": r[:1].expand(4, 64)})
    assert e.value.status == 1
    moe.moe_latent_prompt(lat, q[:0], k[:0], r[:0], v[:0], offsets([0]), out[:0], ws)
    torch.cuda.synchronize()
