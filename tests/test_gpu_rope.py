"""Rotary positions on the GPU against their definition in 64 bits (``rope_ref``):
in place, into other arrays, and into the paged caches."""
import pytest
import torch

import rope_ref as ref
from quantized_moe_expert_router_gb300 import moe
from test_rope_host import KIND, SCALINGS

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
LAYOUT = {False: moe.ROPE_HALF, True: moe.ROPE_INTERLEAVED}


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_moe_expert_router_gb300 import build
    build.build()
    moe.load_library()


def randn(shape, dt, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device=DEV).to(dt)


def some_positions(rows, far, seed, gaps=False):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    p = torch.randint(0, far + 1, (rows,), generator=g, device=DEV, dtype=torch.int32)
    p[0] = far
    if gaps:
        p[1::5] = -1
    return p


def handle(dims, dt, interleaved, scaling="plain", theta=10000.0, attn_factor=1.0):
    return (moe.Rope(dims, theta, LAYOUT[interleaved], KIND[scaling], attn_factor=attn_factor, dtype=dt, **SCALINGS[scaling]),
            ref.frequencies(dims, theta, scaling, **SCALINGS[scaling]))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("rows,hq,hk,d,dims,far,scaling", [
    (1, 1, 1, 64, 64, 0, "plain"), (1, 32, 8, 128, 128, 1000, "plain"), (3, 5, 0, 128, 64, 77, "linear"), (7, 3, 1, 128, 16, 100000, "base"),
    (67, 7, 2, 192, 128, 1000000, "yarn"), (500, 33, 3, 64, 32, 4000, "bands"), (4099, 9, 1, 256, 256, 2 ** 24, "plain"),
    (2, 1024, 1, 16, 16, 9, "plain"), (130, 6, 2, 1024, 48, 50, "plain"), (3000, 40, 8, 128, 128, 30000, "yarn"),
])
def test_apply_parity(interleaved, dt, rows, hq, hk, d, dims, far, scaling):
    dt = TYPES[dt]
    rope, f = handle(dims, dt, interleaved, scaling, attn_factor=1.25 if scaling == "yarn" else 1.0)
    factor = 1.25 if scaling == "yarn" else 1.0
    pos = some_positions(rows, far, 1)
    q, k = randn((rows, hq, d), dt, 2), (randn((rows, hk, d), dt, 3) if hk else None)
    want = [ref.turn(x, pos, f, interleaved, factor) for x in (q, k) if x is not None]
    q0, k0 = q.clone(), (k.clone() if hk else None)
    qo, ko = torch.full_like(q, 9.0), (torch.full_like(k, 9.0) if hk else None)
    moe.moe_rope_apply(rope, pos, q, qo, k, ko)
    assert torch.equal(q, q0) and (not hk or torch.equal(k, k0))
    ref.check(qo, want[0], "q")
    if hk:
        ref.check(ko, want[1], "k")
    moe.moe_rope_apply(rope, pos, q, q, k, k)                      # in place: the same bits
    assert torch.equal(q, qo) and (not hk or torch.equal(k, ko))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("far", [2 ** 24 + 1, 2 ** 31 - 1])
def test_far_positions(interleaved, far):
    """The angle is an integer product: int32's last position is as good as the first."""
    rope, f = handle(64, torch.bfloat16, interleaved)
    pos = torch.arange(far - 99, far + 1, dtype=torch.int64, device=DEV).int()
    q = randn((100, 3, 64), torch.bfloat16, 5)
    out = torch.empty_like(q)
    moe.moe_rope_apply(rope, pos, q, out)
    ref.check(out, ref.turn(q, pos, f, interleaved))


@pytest.mark.parametrize("rows", [9, 3001])
def test_views_gaps_and_what_is_left_alone(rows):
    """Parts of a fused projection, heads first, a part of each head; rows at negative positions and everything
    around the views stay as they were."""
    dt = torch.bfloat16
    rope, f = handle(64, dt, True)
    pos = some_positions(rows, 5000, 6, gaps=True)
    x = randn((rows, 6, 192 + 8), dt, 7)
    q = x[:, :, 128:192]                                           # the last 64 of the first 192
    k = randn((2, rows, 64), dt, 8).transpose(0, 1)
    before, want, kwant = x.clone(), ref.turn(q, pos, f, True), ref.turn(k, pos, f, True)
    ko = torch.full((rows, 2, 72), 5.0, dtype=dt, device=DEV)
    moe.moe_rope_apply(rope, pos, q, q, k, ko[:, :, :64])
    ref.check(q, want)
    assert torch.equal(x[:, :, :128], before[:, :, :128]) and torch.equal(x[:, :, 192:], before[:, :, 192:])
    dead = pos < 0
    assert (ko[dead] == 5.0).all() and (ko[:, :, 64:] == 5.0).all() and torch.equal(x[dead], before[dead])
    ref.check(ko[~dead][:, :, :64], [w[~dead] for w in kwant])


@pytest.mark.parametrize("value", [float("nan"), float("inf"), 60000.0])
def test_values_out_of_range_stay_in_their_pair(value):
    rope, f = handle(64, torch.float16, False)
    q = randn((4, 2, 64), torch.float16, 9)
    clean = ref.turn(q, (pos := some_positions(4, 100, 10)), f, False)
    q[1, 1, 5] = value
    out = torch.empty_like(q)
    moe.moe_rope_apply(rope, pos, q, out)
    keep = torch.ones_like(q, dtype=torch.bool)
    keep[1, 1, 5] = keep[1, 1, 37] = False
    ref.check(torch.where(keep, out, 0), [torch.where(keep, w, 0.0) for w in clean])
    if value == 60000.0:
        ref.check(out, ref.turn(q, pos, f, False))
    else:
        assert not torch.isfinite(out[1, 1, 5]) and not torch.isfinite(out[1, 1, 37])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rows,hk,g,d,dims,page", [(1, 1, 1, 64, 64, 16), (56, 8, 4, 128, 128, 16), (333, 3, 2, 64, 32, 32), (2049, 2, 5, 128, 64, 128)])
def test_append_parity(interleaved, rows, hk, g, d, dims, page):
    dt = torch.float16 if page == 32 else torch.bfloat16
    rope, f = handle(dims, dt, interleaved, "bands")
    pool = -(-rows // page) + 3
    attn = moe.Attention(hk * g, hk, d, page, pool, 4, dt)
    pos = some_positions(rows, 9000, 11, gaps=rows > 9)
    slots = torch.randperm(pool * page, device=DEV)[:rows].int()
    if rows > 9:
        slots[2], slots[3], slots[4] = -1, pool * page, -2 ** 31
    x = randn((rows, (hk * g + 2 * hk) * d), dt, 12)
    q, k, v = (x[:, a * d:b * d].unflatten(1, (-1, d)) for a, b in ((0, hk * g), (hk * g, hk * (g + 1)), (hk * (g + 1), hk * (g + 2))))
    kc, vc = (torch.full(attn.cache_shape, 7.0, dtype=dt, device=DEV) for _ in range(2))
    qo = torch.full((rows, hk * g, d), 7.0, dtype=dt, device=DEV)
    moe.moe_rope_append(attn, rope, q, k, v, pos, slots, qo, kc, vc)
    live = pos >= 0
    ref.check(qo[live], [w[live] for w in ref.turn(q, pos, f, interleaved)], "q")
    assert (qo[~live] == 7.0).all()
    there = live & (slots >= 0) & (slots < pool * page)
    at = slots[there].long()
    by_token = [c.transpose(1, 2).reshape(pool * page, hk, d) for c in (kc, vc)]
    ref.check(by_token[0][at], [w[there] for w in ref.turn(k, pos, f, interleaved)], "k")
    assert torch.equal(by_token[1][at], v[there])
    rest = torch.ones(pool * page, dtype=torch.bool, device=DEV)
    rest[at] = False
    assert all((t[rest] == 7.0).all() for t in by_token)
    # the same bits as the two calls apart
    kc2, vc2, ko = torch.full_like(kc, 7.0), torch.full_like(vc, 7.0), k.clone()
    moe.moe_rope_apply(rope, pos, k, ko)
    moe.moe_kv_append(attn, ko, v, torch.where(live, slots, -1), kc2, vc2)
    assert torch.equal(kc, kc2) and torch.equal(vc, vc2)


@pytest.mark.parametrize("rows,heads,dims,page,with_q", [(1, 16, 64, 16, True), (7, 5, 64, 64, True), (3, 1, 32, 128, False), (1500, 64, 64, 32, True)])
def test_latent_append_parity(rows, heads, dims, page, with_q):
    dt = torch.float16 if page == 64 else torch.bfloat16
    rope, f = handle(dims, dt, True, "yarn", 50000.0, 1.25)
    pool = -(-rows // page) + 2
    lat = moe.LatentAttention(heads, page, pool, 4, dt)
    pos = some_positions(rows, 100000, 13, gaps=rows > 6)
    slots = torch.randperm(pool * page, device=DEV)[:rows].int()
    if rows > 6:
        slots[2], slots[3] = -1, pool * page
    x = randn((rows, 576), dt, 14)
    q = randn((rows, heads, 192), dt, 15)
    before = q.clone()
    cache = torch.full(lat.cache_shape, 7.0, dtype=dt, device=DEV)
    part = q[:, :, 128:] if with_q else None
    ko = torch.full((rows, 72), 7.0, dtype=dt, device=DEV) if with_q else None
    moe.moe_latent_append(lat, rope, x[:, :512], x[:, 512:], pos, slots, cache, q=part, q_out=part, k_out=ko[:, :64] if with_q else None)
    live = pos >= 0
    if with_q:                                       # every row with a position, slot or none
        ref.check(ko[live][:, None, :64], [w[live] for w in ref.turn(x[:, None, 512:], pos, f, True, 1.25)], "k_out")
        assert (ko[~live] == 7.0).all() and (ko[:, 64:] == 7.0).all()
    if with_q:
        ref.check(q[:, :, 128:], ref.turn(before[:, :, 128:], pos, f, True, 1.25), "q")
    assert torch.equal(q[:, :, :128], before[:, :, :128]) and torch.equal(q[~live], before[~live])
    there = live & (slots >= 0) & (slots < pool * page)
    at, tokens = slots[there].long(), cache.view(-1, 576)
    assert torch.equal(tokens[at, :512], x[there, :512])
    ref.check(tokens[at, None, 512:], [w[there] for w in ref.turn(x[:, None, 512:], pos, f, True, 1.25)], "k")
    rest = torch.ones(pool * page, dtype=torch.bool, device=DEV)
    rest[at] = False
    assert (tokens[rest] == 7.0).all()


def test_captured_and_on_another_stream():
    rope, f = handle(128, torch.bfloat16, False)
    q, pos = randn((50, 8, 128), torch.bfloat16, 16), some_positions(50, 4000, 17)
    out = torch.empty_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    moe.moe_rope_apply(rope, pos, q, out, stream=side)
    side.synchronize()
    want = out.clone()
    ref.check(want, ref.turn(q, pos, f, False))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_rope_apply(rope, pos, q, out)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_empty_calls():
    rope, _ = handle(64, torch.bfloat16, False)
    attn, lat = moe.Attention(2, 1, 64, 16, 2, 2), moe.LatentAttention(2, 16, 2, 2)
    none = torch.empty(0, dtype=torch.int32, device=DEV)
    e = lambda *s: torch.empty(s, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    moe.moe_rope_apply(rope, none, e(0, 4, 64), e(0, 4, 64))
    moe.moe_rope_append(attn, rope, e(0, 2, 64), e(0, 1, 64), e(0, 1, 64), none, none, e(0, 2, 64), e(2, 1, 16, 64), e(2, 1, 16, 64))
    moe.moe_latent_append(lat, rope, e(0, 512), e(0, 64), none, none, e(2, 16, 576))
    torch.cuda.synchronize()


def test_refusals():
    rope, _ = handle(64, torch.bfloat16, False)
    q, pos = randn((4, 2, 64), torch.bfloat16, 18), some_positions(4, 9, 19)
    with pytest.raises(TypeError, match="q is"):
        moe.moe_rope_apply(rope, pos, q.half(), q)
    with pytest.raises(TypeError, match="positions is"):
        moe.moe_rope_apply(rope, pos.long(), q, q)
    with pytest.raises(ValueError, match="q_out of shape"):
        moe.moe_rope_apply(rope, pos, q, q[:3])
    with pytest.raises(ValueError, match="k and k_out"):
        moe.moe_rope_apply(rope, pos, q, q, k=q)
    with pytest.raises(ValueError, match="contiguous last axis"):
        moe.moe_rope_apply(rope, pos, q.transpose(1, 2).contiguous().transpose(1, 2), q)
    with pytest.raises(moe.MoEError) as e:                         # rows that overlap themselves
        moe.moe_rope_apply(rope, pos, q[:1].expand(4, 2, 64), q)
    assert e.value.status == 1
    with pytest.raises(moe.MoEError) as e:
        moe.moe_rope_apply(rope, pos, q[:, :, :48], q[:, :, :48])
    assert e.value.status == 2
    attn = moe.Attention(2, 1, 64, 16, 2, 2, torch.float16)
    cache = torch.zeros(attn.cache_shape, dtype=torch.float16, device=DEV)
    with pytest.raises(TypeError, match="handles of"):
        moe.moe_rope_append(attn, rope, q, q[:, :1], q[:, :1], pos, pos, q, cache, cache)
    wide = moe.Rope(128)
    attn = moe.Attention(2, 1, 64, 16, 2, 2)
    cache = torch.zeros(attn.cache_shape, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(moe.MoEError) as e:
        moe.moe_rope_append(attn, wide, q, q[:, :1], q[:, :1], pos, pos, q, cache, cache)
    assert e.value.status == 2
    lat = moe.LatentAttention(2, 16, 2, 2)
    cache, c = torch.zeros(lat.cache_shape, dtype=torch.bfloat16, device=DEV), randn((4, 576), torch.bfloat16, 20)
    with pytest.raises(ValueError, match="q and q_out"):
        moe.moe_latent_append(lat, rope, c[:, :512], c[:, 512:], pos, pos, cache, q=q)
    with pytest.raises(ValueError, match="cache of shape"):
        moe.moe_latent_append(lat, rope, c[:, :512], c[:, 512:], pos, pos, cache[:1])
    with pytest.raises(ValueError, match="slots of shape"):
        moe.moe_latent_append(lat, rope, c[:, :512], c[:, 512:], pos, pos[:2], cache)
    with pytest.raises(ValueError, match="c of shape"):
        moe.moe_latent_append(lat, rope, c, c[:, 512:], pos, pos, cache)
    with pytest.raises(ValueError, match="k_out of shape"):
        moe.moe_latent_append(lat, rope, c[:, :512], c[:, 512:], pos, pos, cache, k_out=c)
    with pytest.raises(moe.MoEError) as e:                         # in place: the cache's threads read it
        moe.moe_latent_append(lat, rope, c[:, :512], c[:, 512:], pos, pos, cache, k_out=c[:, 512:])
    assert e.value.status == 1
