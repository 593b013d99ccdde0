"""Far positions on the GPU: the angle of a position near 2^31 is that of a near one, to the last unit that the kernel takes."""
from decimal import Decimal, getcontext

import pytest
import torch

from quantized_moe_expert_router_gb300 import moe
from test_gpu_rope import DEV, built  # noqa: F401  (built: the module's build fixture)

pytestmark = pytest.mark.gpu
PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")


def fractions(f, positions):
    """Turns that positions make at f radians each, without the whole ones, times 2^64 (whole numbers)."""
    getcontext().prec = 90
    per = int(Decimal(f) / (2 * PI) * 2 ** 128)
    return [(p * per % 2 ** 128) >> 64 for p in positions]


@pytest.mark.parametrize("pair", [0, 1, 5])
def test_the_last_positions_are_as_good_as_the_first(pair):
    """Positions below 2^31 whose angle is just above a whole turn: the sine is so small that f16 resolves an angle's error of
    2^-24.  A handle whose pair 0 turns 2^-32 (1 + 2^-40) of a turn a position gives the same angle, in units of 2^-32 turns as the
    kernel takes them, at the position of that number: the results have to be the same bits.  Turns are held to
    2^-65, so 2^31 of them are off by a fourth of a unit: positions whose angle lies in the middle third of one."""
    far = moe.Rope(16, 100.0, moe.ROPE_HALF, dtype=torch.float16)
    f = moe.moe_rope_frequencies(far)[pair]
    tries = [2 ** 31 - 1 - 7 * i for i in range(300000)]
    found = [(p, x >> 32) for p, x in zip(tries, fractions(f, tries))
             if 1e-5 < x / 2 ** 64 < 6e-5 and 0.34 < (x & 0xFFFFFFFF) / 2 ** 32 < 0.66]
    assert len(found) >= 4
    near = moe.Rope(16, 100.0, moe.ROPE_HALF, moe.ROPE_LINEAR, factor=float(2 ** 32 / (2 * PI) * (1 - Decimal(2) ** -40)), dtype=torch.float16)
    out = []
    for rope, i, at in ((far, pair, 0), (near, 0, 1)):
        x = torch.zeros((len(found), 1, 16), dtype=torch.float16, device=DEV)
        x[:, :, i] = 1.0
        moe.moe_rope_apply(rope, torch.tensor([y[at] for y in found], dtype=torch.int32, device=DEV), x, x)
        out.append(torch.stack([x[:, 0, i], x[:, 0, i + 8]]))
    assert (out[1][1] > 0).all() and torch.equal(out[0], out[1])
