"""The attention operators together, as a serving loop uses them around the
routed MoE layer.

One decoder block (random weights): rows -> q, k, v by one projection ->
attention -> output projection -> routed MoE layer.  Three streams are admitted
with prompts of different lengths; then every step verifies a small tree of
drafted rows per stream:

    moe_kv_plan     pages, slots, positions and tree masks from the lengths
    moe_rope_apply  queries and keys turned by the positions
    moe_kv_append   the rows' keys and values to their slots
    moe_attn_prompt (admission) or moe_attn_tree (verification)
    moe_route_forward
    moe_kv_append   again for the accepted rows, at their final slots

"Acceptance" takes each tree's longest path.  At the end the attention of the
accepted rows is compared with one moe_attn_prompt call over the whole accepted
sequences: the paged, stepwise computation has to give the same.

    python examples/paged_step.py [steps]
"""
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from quantized_moe_expert_router_gb300 import moe, synth  # noqa: E402

DEV = "cuda:0"
HIDDEN, Q_HEADS, KV_HEADS, HEAD_DIM = 512, 8, 2, 64
EXPERTS, TOP_K, INTERMEDIATE = 32, 4, 192
PAGE, POOL, TABLE = 16, 96, 24
PROMPTS = (70, 33, 5)
#: Parents of a drafted tree's rows: two branches from the context.
TREE = (-1, 0, 0, 1, -1, 4, 3)
PATH = (0, 1, 3, 6)                       # its longest path


class Block:
    """The block's weights, handles and buffers for up to `rows` rows of a step."""

    def __init__(self, rows):
        g = torch.Generator(device=DEV)
        g.manual_seed(0)
        width = (Q_HEADS + 2 * KV_HEADS) * HEAD_DIM
        self.wqkv = (torch.randn((HIDDEN, width), generator=g, device=DEV) * HIDDEN ** -0.5).bfloat16()
        self.wo = (torch.randn((Q_HEADS * HEAD_DIM, HIDDEN), generator=g, device=DEV) * HIDDEN ** -0.5).bfloat16()
        self.attn = moe.Attention(Q_HEADS, KV_HEADS, HEAD_DIM, PAGE, POOL, TABLE)
        self.rope = moe.Rope(HEAD_DIM)
        self.ws = moe.alloc_attn_workspace(self.attn, len(PROMPTS), rows)
        self.k_cache, self.v_cache = (torch.zeros((POOL, KV_HEADS, PAGE, HEAD_DIM), dtype=torch.bfloat16, device=DEV) for _ in range(2))
        self.layer = moe.Layer(EXPERTS, TOP_K, HIDDEN, INTERMEDIATE, rows)
        canon = synth.canonical_layer(0, 0, EXPERTS, HIDDEN, INTERMEDIATE)
        self.packed = moe.alloc_packed(self.layer)
        moe.moe_pack_weights(self.layer, {n: {f: torch.from_numpy(m[f]).to(DEV) for f in m} for n, m in canon.items()}, self.packed)
        self.router = torch.from_numpy(synth.router_weights(0, 0, EXPERTS, HIDDEN)).to(DEV)
        self.moe_ws = moe.alloc_workspace(self.layer, rows)

    def qkv(self, x):
        y = x @ self.wqkv
        n, a, b = x.shape[0], Q_HEADS * HEAD_DIM, KV_HEADS * HEAD_DIM
        return (y[:, :a].view(n, Q_HEADS, HEAD_DIM), y[:, a:a + b].view(n, KV_HEADS, HEAD_DIM), y[:, a + b:].view(n, KV_HEADS, HEAD_DIM))

    def experts(self, x):
        n = x.shape[0]
        ids = torch.empty((n, TOP_K), dtype=torch.int32, device=DEV)
        w = torch.empty((n, TOP_K), dtype=torch.float32, device=DEV)
        y = torch.empty((n, HIDDEN), dtype=torch.float32, device=DEV)
        moe.moe_route_forward(self.layer, x.view(torch.int16), n, self.router, None, self.packed, ids, w, y, self.moe_ws)
        return y


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def main(steps=3, accepted=None):
    """Runs the loop; returns the largest difference and the largest value.  A list `accepted` is given, by stream, the
    accepted rows' (q, k, v, stepwise attention)."""
    streams = len(PROMPTS)
    rows_max = sum(PROMPTS)
    block = Block(rows_max)
    attn = block.attn
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    free = torch.randperm(POOL, generator=g, device=DEV).int()
    table = torch.full((streams, TABLE), -1, dtype=torch.int32, device=DEV)
    info = torch.zeros(4, dtype=torch.int32, device=DEV)
    cached, fresh = [0] * streams, list(PROMPTS)
    history = [[] for _ in range(streams)]            # per stream: accepted (q, k, v, attention) rows
    for step in range(steps + 1):
        rows = sum(fresh)
        x = torch.randn((rows, HIDDEN), generator=g, device=DEV).bfloat16()      # stands for the block's input
        parents = ints(list(TREE) * streams) if step else None
        cu = torch.empty(streams + 1, dtype=torch.int32, device=DEV)
        slots, positions = (torch.empty(rows, dtype=torch.int32, device=DEV) for _ in range(2))
        mask = torch.empty(rows, dtype=torch.int64, device=DEV) if step else None
        moe.moe_kv_plan(attn, ints(cached), ints(fresh), free, table, cu, slots, positions, info, parents=parents, tree_mask=mask)
        q, k, v = block.qkv(x)
        moe.moe_rope_apply(block.rope, positions, q, q, k, k)
        moe.moe_kv_append(attn, k, v, slots, block.k_cache, block.v_cache)
        out = torch.empty((rows, Q_HEADS, HEAD_DIM), dtype=torch.bfloat16, device=DEV)
        if step == 0:
            moe.moe_attn_prompt(attn, q, k, v, cu, out, block.ws)
        else:
            moe.moe_attn_tree(attn, q, cu, ints(cached), table, block.k_cache, block.v_cache, out, block.ws, tree_mask=mask)
        hidden = x + out.view(rows, -1) @ block.wo
        y = block.experts(hidden.contiguous())
        if not torch.isfinite(y).all():
            raise RuntimeError(f"step {step}: non-finite output")
        # acceptance (on the host, as a sampler would): whole prompts, then each tree's longest path
        used = info.tolist()
        if used[3]:
            raise RuntimeError(f"step {step}: plan flags {used[3]}")
        free = free[used[1]:]
        keep = torch.full((rows,), -1, dtype=torch.int32, device=DEV)
        lo = 0
        for b, f in enumerate(fresh):
            path = list(range(f)) if step == 0 else list(PATH)
            at = torch.tensor(path, device=DEV) + lo
            keep[at] = slots[lo:lo + len(path)]
            history[b].append((q[at], k[at], v[at], out[at]))
            lo += f
            cached[b] += len(path)
        if step:
            moe.moe_kv_append(attn, k, v, keep, block.k_cache, block.v_cache)
            # pages that only rejected rows had reached go back to the free list
            for b in range(streams):
                have, held = -(-cached[b] // PAGE), int((table[b] >= 0).sum())
                if held > have:
                    free = torch.cat([table[b, have:held], free])
                    table[b, have:held] = -1
        fresh = [len(TREE)] * streams
        print(f"step {step}: {rows} rows, contexts {cached}, {int(used[1])} new pages, |y| {float(y.abs().mean()):.4f}")
    if accepted is not None:
        accepted += [tuple(torch.cat([r[i] for r in h]) for i in range(4)) for h in history]
    # the same rows by one call over the whole sequences
    q, k, v, got = (torch.cat([torch.cat([r[i] for r in h]) for h in history]) for i in range(4))
    lengths = [sum(r[0].shape[0] for r in h) for h in history]
    cu = ints([sum(lengths[:b]) for b in range(streams + 1)])
    want = torch.empty_like(got)
    moe.moe_attn_prompt(attn, q, k, v, cu, want, moe.alloc_attn_workspace(attn, streams, q.shape[0]))
    status = moe.moe_attn_get_device_status(attn, block.ws)
    if status:
        raise RuntimeError(f"device status {status}")
    off = float((got.float() - want.float()).abs().max())
    print(f"stepwise against whole sequences: largest difference {off:.4f}")
    return off, float(want.float().abs().max())


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 3)
