"""The latent attention's operators together, as a serving loop uses them around
the routed MoE layer.

One decoder block (random weights): rows -> queries, latent and key part by two
projections -> latent attention -> output projection -> routed MoE layer.  Three
streams are admitted with prompts of different lengths; then every step verifies
a small tree of drafted rows per stream:

    moe_latent_plan     pages, slots, positions and tree masks from the lengths
    moe_latent_append   the rows' latents and turned key parts to their slots; the
                        queries' rotary part is turned beside it
    moe_latent_prompt   (admission) on the latents' expansion to keys and values, or
    moe_latent_tree     (verification) over the cache, with the expansion's weights
                        multiplied into the queries and the output
    moe_route_forward
    moe_latent_append   again for the accepted rows, at their final slots

"Acceptance" takes each tree's longest path.  At the end the attention of the
accepted rows is compared with one moe_latent_prompt call over the whole accepted
sequences: the paged, stepwise, absorbed computation has to give the same as the
expanded one, but for the rounding of what each multiplies.

    python examples/latent_step.py [steps]
"""
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from quantized_moe_expert_router_gb300 import moe, synth  # noqa: E402

DEV = "cuda:0"
HIDDEN, HEADS = 512, 8
LATENT, ROPE, HEAD = moe.LATENT_DIM, moe.LATENT_ROPE, moe.LATENT_HEAD
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

        def weight(*shape, fan):
            return (torch.randn(shape, generator=g, device=DEV) * fan ** -0.5).bfloat16()
        self.wq = weight(HIDDEN, HEADS * (HEAD + ROPE), fan=HIDDEN)
        self.wc = weight(HIDDEN, LATENT + ROPE, fan=HIDDEN)
        self.wk, self.wv = (weight(HEADS, HEAD, LATENT, fan=LATENT) for _ in range(2))     # a head's K and V
        self.wo = weight(HEADS * HEAD, HIDDEN, fan=HEADS * HEAD)
        self.attn = moe.LatentAttention(HEADS, PAGE, POOL, TABLE)
        self.rope = moe.Rope(ROPE, 50000.0, moe.ROPE_INTERLEAVED)
        self.ws = moe.alloc_latent_workspace(self.attn, len(PROMPTS), rows)
        self.cache = torch.zeros(self.attn.cache_shape, dtype=torch.bfloat16, device=DEV)
        self.layer = moe.Layer(EXPERTS, TOP_K, HIDDEN, INTERMEDIATE, rows)
        canon = synth.canonical_layer(0, 0, EXPERTS, HIDDEN, INTERMEDIATE)
        self.packed = moe.alloc_packed(self.layer)
        moe.moe_pack_weights(self.layer, {n: {f: torch.from_numpy(m[f]).to(DEV) for f in m} for n, m in canon.items()}, self.packed)
        self.router = torch.from_numpy(synth.router_weights(0, 0, EXPERTS, HIDDEN)).to(DEV)
        self.moe_ws = moe.alloc_workspace(self.layer, rows)

    def project(self, x):
        """Queries [rows][heads][192], latents [rows][512], key parts [rows][64] (views of one projection)."""
        y = x @ self.wc
        return (x @ self.wq).view(-1, HEADS, HEAD + ROPE), y[:, :LATENT], y[:, LATENT:]

    def expanded(self, q, c, r, cu):
        """Attention of packed prompts on keys and values of every head."""
        k, v = ((c @ w.view(HEADS * HEAD, LATENT).T).view(-1, HEADS, HEAD) for w in (self.wk, self.wv))
        out = torch.empty((q.shape[0], HEADS, HEAD), dtype=torch.bfloat16, device=DEV)
        moe.moe_latent_prompt(self.attn, q, k, r, v, cu, out, self.ws)
        return out

    def absorbed(self, q, cu, cached, table, mask):
        """Attention over the cache: K goes into the query, V into the output (a product a head)."""
        qk = torch.bmm(q[:, :, :HEAD].transpose(0, 1), self.wk).transpose(0, 1)
        o = torch.empty((HEADS, q.shape[0], LATENT), dtype=torch.bfloat16, device=DEV)
        moe.moe_latent_tree(self.attn, qk, q[:, :, HEAD:], cu, cached, table, self.cache, o.transpose(0, 1), self.ws, tree_mask=mask)
        return torch.bmm(o, self.wv.transpose(1, 2)).transpose(0, 1)

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
    """Runs the loop; returns the largest difference and the largest value.  A list `accepted` is given the block and, by
    stream, the accepted rows' (turned q, latent, turned key part, stepwise attention, position)."""
    streams = len(PROMPTS)
    block = Block(sum(PROMPTS) + steps * streams * len(PATH))
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    free = torch.randperm(POOL, generator=g, device=DEV).int()
    table = torch.full((streams, TABLE), -1, dtype=torch.int32, device=DEV)
    info = torch.zeros(4, dtype=torch.int32, device=DEV)
    cached, fresh = [0] * streams, list(PROMPTS)
    history = [[] for _ in range(streams)]
    for step in range(steps + 1):
        rows = sum(fresh)
        x = torch.randn((rows, HIDDEN), generator=g, device=DEV).bfloat16()      # stands for the block's input
        parents = ints(list(TREE) * streams) if step else None
        cu = torch.empty(streams + 1, dtype=torch.int32, device=DEV)
        slots, positions = (torch.empty(rows, dtype=torch.int32, device=DEV) for _ in range(2))
        mask = torch.empty(rows, dtype=torch.int64, device=DEV) if step else None
        moe.moe_latent_plan(block.attn, ints(cached), ints(fresh), free, table, cu, slots, positions, info, parents=parents, tree_mask=mask)
        q, c, r = block.project(x)
        turned = torch.empty((rows, ROPE), dtype=torch.bfloat16, device=DEV)
        moe.moe_latent_append(block.attn, block.rope, c, r, positions, slots, block.cache, q=q[:, :, HEAD:], q_out=q[:, :, HEAD:], k_out=turned)
        out = block.absorbed(q, cu, ints(cached), table, mask) if step else block.expanded(q, c, turned, cu)
        hidden = x + out.reshape(rows, -1) @ block.wo
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
            history[b].append((q[at], c[at], turned[at], out[at], positions[at]))
            lo += f
            cached[b] += len(path)
        if step:
            moe.moe_latent_append(block.attn, block.rope, c, r, positions, keep, block.cache)
            # pages that only rejected rows had reached go back to the free list
            for b in range(streams):
                have, held = -(-cached[b] // PAGE), int((table[b] >= 0).sum())
                if held > have:
                    free = torch.cat([table[b, have:held], free])
                    table[b, have:held] = -1
        fresh = [len(TREE)] * streams
        print(f"step {step}: {rows} rows, contexts {cached}, {int(used[1])} new pages, |y| {float(y.abs().mean()):.4f}")
    whole = [tuple(torch.cat([s[i] for s in h]) for i in range(5)) for h in history]
    if accepted is not None:
        accepted += [block] + whole
    # the same rows by one call over the whole sequences
    q, c, r, got = (torch.cat([h[i] for h in whole]) for i in range(4))
    lengths = [h[0].shape[0] for h in whole]
    want = block.expanded(q, c, r, ints([sum(lengths[:b]) for b in range(streams + 1)]))
    status = moe.moe_latent_get_device_status(block.attn, block.ws)
    if status:
        raise RuntimeError(f"device status {status}")
    off = float((got.float() - want.float()).abs().max())
    print(f"stepwise and absorbed against whole and expanded: largest difference {off:.4f}")
    return off, float(want.float().abs().max())


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 3)
