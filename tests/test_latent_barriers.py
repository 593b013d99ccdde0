"""The barriers of lat_tree_kernel, and of attn_wide_kernel's ring of pieces, under every
role held back (host only): no wait is ever two phases behind its barrier."""
import os
import random

import pytest

import attn_barriers as ab
import latent_barriers as lb

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "quantized_moe_expert_router_gb300", "csrc")
TREE, WIDE = (open(os.path.join(CSRC, n)).read() for n in ("latent_tree.cu", "attn_wide.cu"))
SOFT = [f"soft{h}{w}" for h in range(2) for w in range(4)]
TREE_ROLES = ["copy", "s", "o", "q", "scores", "values", "tiles", "qcopies"] + SOFT
RINGS = [(4, 2), (5, 3)]                               # halves, key parts: 64 rows, and 32 or 16


def tree(items, ring, seed=0, often=0.5, **kw):
    for pick in ab.schedules(len(items), TREE_ROLES):
        ab.run(lb.Tree(ab.counts(TREE), items, *ring, lb.moves_by(seed, often), **kw), pick)


def test_the_kernel_has_the_modelled_barriers():
    count = ab.counts(TREE)
    assert count["p_full"] == 8 and count["sched_empty"] == 11
    assert all(count[n] == 1 for n in ("kv_full", "kv_empty", "q_full", "q_empty", "s_full", "pv_done", "sched_full"))
    assert "kHalves = N == 64 ? 4 : 5" in TREE and "kParts = N == 64 ? 2 : 3" in TREE
    assert "s_full[2], p_full[2], pv_done[2]" in TREE
    assert "kStages = 7;                // pieces" in WIDE


@pytest.mark.parametrize("ring", RINGS)
@pytest.mark.parametrize("often", [0.0, 0.5, 1.0])
@pytest.mark.parametrize("items", [[dict(n=1, m0=0)] * 7, [dict(n=2, m0=1)] * 5, [dict(n=7, m0=6), dict(n=1, m0=1)] * 3, [dict(n=12, m0=10)]])
def test_tree_no_wait_is_overtaken(items, ring, often):
    tree(items, ring, often=often)


@pytest.mark.parametrize("seed", range(30))
def test_tree_no_wait_is_overtaken_random_items(seed):
    rng = random.Random(seed)
    tree(lb.random_tree_items(rng, rng.randint(1, 6), rng.choice([1, 2, 4, 7])), rng.choice(RINGS), seed, rng.choice([0.1, 0.5]))


def test_the_model_finds_an_overtaken_wait():
    """One pv_done for all tiles: the products of an item's last two tiles may both be done when a softmax warp looks."""
    with pytest.raises((ab.Aliased, ab.Stuck)):
        tree([dict(n=4, m0=3)] * 3, RINGS[0], split_done=False)


@pytest.mark.parametrize("items", [
    [dict(n=1, m0=0, n0=1, n1=1, twin=False)] * 7, [dict(n=1, m0=1, n0=1, n1=0, twin=False), dict(n=1, m0=0, n0=1, n1=0, twin=False)] * 4,
    [dict(n=2, m0=2, n0=1, n1=1, twin=True), dict(n=2, m0=1, n0=1, n1=1, twin=True), dict(n=1, m0=0, n0=1, n1=0, twin=True)] * 3,
    [dict(n=3, m0=0, n0=2, n1=3, twin=False)] * 5, [dict(n=9, m0=8, n0=9, n1=9, twin=False), dict(n=1, m0=1, n0=1, n1=1, twin=False)] * 3,
])
def test_prompt_no_wait_is_overtaken(items):
    prompt(items)


@pytest.mark.parametrize("seed", range(30))
def test_prompt_no_wait_is_overtaken_random_items(seed):
    rng = random.Random(seed)
    prompt(ab.random_items(rng, rng.randint(1, 7), rng.choice([1, 2, 3, 6])))


def prompt(items):
    for pick in ab.schedules(len(items), ["copy", "mma", "help2", "help3", "pipe", "tiles", "q"] + SOFT):
        ab.run(lb.Prompt(ab.counts(WIDE), items), pick)
