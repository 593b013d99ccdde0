"""Latent and rotary calls right behind one another, nothing else between them: each may start before the one ahead has ended, and has to
read what that writes and to write what that reads only when it has.  Every chain is compared, bit for bit, with the same
calls a synchronisation apart; tree calls run over contexts long enough to be at work while the next call starts, on items that
stay whole (no join behind them) and on items that are cut (tables of capacity)."""
from types import SimpleNamespace

import pytest
import torch

from quantized_moe_expert_router_gb300 import moe
from test_gpu_attn import ints, offsets, randn
from test_gpu_latent import DEV, Latent, built  # noqa: F401  (built: the module's build fixture)

pytestmark = pytest.mark.gpu
HEADS, REQUESTS, CONTEXT, PAGE = 16, 400, 900, 64


def step(wide):
    """A decode step of many streams: whole items in a table as wide as the contexts, cut ones in a wide table."""
    c = Latent(HEADS, PAGE, torch.bfloat16, [CONTEXT - i % 37 for i in range(REQUESTS)], [1] * REQUESTS, seed=90)
    if wide:
        c.table = torch.cat([c.table, torch.full((REQUESTS, 2000), -1, dtype=torch.int32, device=DEV)], 1)
        c.lat = moe.LatentAttention(HEADS, PAGE, c.cache.shape[0], c.table.shape[1], c.dt)
    return c



def compare(make, calls, capture):
    """The state after the calls, with and without synchronisation between them, on fresh states each time."""
    want = None
    for rep in range(1 if capture else 8):
        state = make()
        torch.cuda.synchronize()
        if capture:
            calls(make(), lambda: None)                            # warm-up
            torch.cuda.synchronize()
            stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=stream):
                calls(state, lambda: None)
            graph.replay()
        else:
            calls(state, lambda: None)
        torch.cuda.synchronize()
        if want is None:
            want = make()
            torch.cuda.synchronize()
            calls(want, torch.cuda.synchronize)
            torch.cuda.synchronize()
        for k in want:
            if torch.is_tensor(want[k]):
                assert torch.equal(state[k].contiguous().view(torch.int16), want[k].contiguous().view(torch.int16)), f"{k}, turn {rep}"
        assert moe.moe_latent_get_device_status(state["c"].lat, state["ws"]) == 0


def tree(s, out, q="q"):
    c = s["c"]
    moe.moe_latent_tree(c.lat, s[q][:, :, :512], s[q][:, :, 512:], c.cu, c.cached, c.table, s["cache"], s[out], s["ws"])


def maker(wide, **more):
    c = step(wide)
    base = dict(q=c.q, cache=c.cache, **{k: v for k, v in more.items()})
    ws = moe.alloc_latent_workspace(c.lat, REQUESTS, REQUESTS)

    def make():
        s = {k: v.clone() for k, v in base.items()}
        s.update(c=c, ws=ws, out=torch.zeros((REQUESTS, HEADS, 512), dtype=c.dt, device=DEV))
        s["out2"] = torch.zeros_like(s["out"])
        return s
    return c, make


FORMS = pytest.mark.parametrize("wide", [False, True], ids=["whole", "cut"])
CAPTURED = pytest.mark.parametrize("capture", [False, True], ids=["eager", "captured"])


@FORMS
@CAPTURED
def test_rotation_in_place_of_what_the_tree_call_writes(wide, capture):
    _, make = maker(wide)
    rope, pos = moe.Rope(64), torch.arange(1, REQUESTS + 1, dtype=torch.int32, device=DEV)

    def calls(s, sync):
        tree(s, "out")
        sync()
        moe.moe_rope_apply(rope, pos, s["out"], s["out"])
        sync()
        moe.moe_rope_apply(rope, pos, s["q"][:, :, 512:], s["q"][:, :, 512:])       # what the tree call reads
    compare(make, calls, capture)


@FORMS
@CAPTURED
def test_append_into_slots_that_the_tree_call_reads(wide, capture):
    c, make = maker(wide, rows=randn((REQUESTS, 576), torch.bfloat16, 91))
    rope = moe.Rope(64, layout=moe.ROPE_INTERLEAVED)
    places = torch.arange(REQUESTS, device=DEV) % 800
    slots = (c.table[torch.arange(REQUESTS, device=DEV), places // PAGE] * PAGE + places % PAGE).int()
    pos = ints(list(range(REQUESTS)))

    def calls(s, sync):
        tree(s, "out")
        sync()
        moe.moe_latent_append(c.lat, rope, s["rows"][:, :512], s["rows"][:, 512:], pos, slots, s["cache"], q=s["q"][:, :, 512:], q_out=s["q"][:, :, 512:])
        sync()
        tree(s, "out2")
    compare(make, calls, capture)


@FORMS
@CAPTURED
def test_tree_and_prompt_calls_on_one_workspace(wide, capture):
    """Parts, statistics and counters of one call behind another's; a prompt whose queries a rotation turns right ahead of it."""
    n = 700
    c, make = maker(wide, pq=randn((n, HEADS, 192), torch.bfloat16, 92), pk=randn((n, HEADS, 128), torch.bfloat16, 93),
                    pr=randn((n, 64), torch.bfloat16, 94), pv=randn((n, HEADS, 128), torch.bfloat16, 95),
                    po=torch.zeros((n, HEADS, 128), dtype=torch.bfloat16, device=DEV))
    rope, pos, cu = moe.Rope(64), ints(list(range(n))), offsets([n])

    def calls(s, sync):
        tree(s, "out")
        sync()
        tree(s, "out2")
        sync()
        moe.moe_rope_apply(rope, pos, s["pq"][:, :, 128:], s["pq"][:, :, 128:], s["pr"][:, None], s["pr"][:, None])
        sync()
        moe.moe_latent_prompt(c.lat, s["pq"], s["pk"], s["pr"], s["pv"], cu, s["po"], s["ws"])
        sync()
        moe.moe_rope_apply(rope, pos, s["po"], s["po"])            # in place of the prompt's result
        sync()
        tree(s, "out")
    compare(make, calls, capture)


@CAPTURED
def test_rotated_keys_are_in_the_cache_when_attention_reads_them(capture):
    """moe_rope_append in place ahead of grouped-query attention, and again behind it into the slots that it reads."""
    B, hk, g, d, page, n = 64, 2, 4, 128, 16, 500
    width = -(-(n + 1) // page)
    attn = moe.Attention(hk * g, hk, d, page, B * width, width)
    table = torch.arange(B * width, dtype=torch.int32, device=DEV).view(B, width)
    cached, cu, pos = ints([n] * B), offsets([1] * B), ints([n] * B)
    slots = table[:, n // page] * page + n % page
    rope, lat = moe.Rope(d), moe.LatentAttention(1, 16, 1, 1)
    ws, status = moe.alloc_attn_workspace(attn, B, B), moe.alloc_latent_workspace(lat, 1, 1)
    kc, vc = (randn((B * width, hk, page, d), torch.bfloat16, 96 + i) for i in range(2))
    x = randn((B, hk * (g + 2), d), torch.bfloat16, 98)

    c = SimpleNamespace(lat=lat)

    def make():
        return dict(x=x.clone(), kc=kc.clone(), vc=vc.clone(), o1=torch.zeros((B, hk * g, d), dtype=torch.bfloat16, device=DEV),
                    o2=torch.zeros((B, hk * g, d), dtype=torch.bfloat16, device=DEV), c=c, ws=status)

    def calls(s, sync):
        q, k, v = s["x"][:, :hk * g], s["x"][:, hk * g:hk * (g + 1)], s["x"][:, hk * (g + 1):]
        for out in ("o1", "o2"):
            moe.moe_rope_append(attn, rope, q, k, v, pos, slots, q, s["kc"], s["vc"])
            sync()
            moe.moe_attn_tree(attn, q, cu, cached, table, s["kc"], s["vc"], s[out], ws)
            sync()
            moe.moe_rope_apply(rope, pos, k, k)
            sync()
    compare(make, calls, capture)
    assert moe.moe_attn_get_device_status(attn, ws) == 0
