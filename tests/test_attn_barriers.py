"""attn_wide_kernel's barriers under every role held back (host only): no wait is
ever two phases behind its barrier, whatever the items."""
import os
import random

import pytest

import attn_barriers as ab

SOURCE = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "quantized_moe_expert_router_gb300", "csrc",
                           "attn_wide.cu")).read()
COUNTS = ab.counts(SOURCE)
ROLES = ["copy", "mma", "help2", "help3", "pipe", "tiles", "q"] + [f"soft{h}{w}" for h in range(2) for w in range(4)]


def sweep(items, stages, **kw):
    for pick in ab.schedules(len(items), ROLES):
        ab.run(ab.Model(COUNTS, items, stages, **kw), pick)


def test_the_kernel_has_the_modelled_barriers():
    """Both helper warps arrive on v_clean, which has a barrier per item parity; q_empty is waited for once, by the warp that copies Q."""
    assert COUNTS["v_clean"] == 2 and COUNTS["v_posted"] == 1 and COUNTS["q_full"] == 1 and COUNTS["q_empty"] == 1
    assert COUNTS["sched_empty"] == 11 and COUNTS["p_full"] == 4
    assert "v_clean[2][3]" in SOURCE and "v_next" not in SOURCE
    assert SOURCE.count("&s.q_empty, (uint32_t)(i - 1)") == 1 and "warp == kApWHelp && i > 0" in SOURCE


@pytest.mark.parametrize("stages", [2, 4])
@pytest.mark.parametrize("items", [
    [dict(n=1, m0=0, n0=1, n1=1, twin=False)] * 7,                       # prompts of one key tile
    [dict(n=1, m0=1, n0=1, n1=0, twin=False), dict(n=1, m0=0, n0=1, n1=0, twin=False)] * 4,   # without and with a masked tile
    [dict(n=2, m0=2, n0=1, n1=1, twin=True), dict(n=2, m0=1, n0=1, n1=1, twin=True), dict(n=1, m0=0, n0=1, n1=0, twin=True)] * 3,
    [dict(n=3, m0=0, n0=2, n1=3, twin=False)] * 5,
    [dict(n=9, m0=8, n0=9, n1=9, twin=False), dict(n=1, m0=1, n0=1, n1=1, twin=False)] * 3,
])
def test_no_wait_is_overtaken(items, stages):
    sweep(items, stages)


@pytest.mark.parametrize("seed", range(40))
def test_no_wait_is_overtaken_random_items(seed):
    rng = random.Random(seed)
    sweep(ab.random_items(rng, rng.randint(1, 9), rng.choice([1, 2, 3, 6])), rng.choice([2, 4]))


@pytest.mark.parametrize("plant", [dict(q_by_copier=False), dict(clean_by_item=False), dict(clean_by_item=False, q_by_copier=False)])
def test_the_model_finds_an_overtaken_wait(plant):
    """One v_clean behind a v_next, or both helper warps behind q_empty: a helper warp that is held back is overtaken."""
    items = [dict(n=1, m0=1, n0=1, n1=0, twin=False), dict(n=1, m0=0, n0=1, n1=0, twin=False)] * 4
    with pytest.raises((ab.Aliased, ab.Stuck)):
        sweep(items, 4, **plant)
