"""examples/paged_step.py row by row: the stepwise attention of every accepted row
against its definition in 64 bits over the accepted sequence, element by element
with the bounds of ``attn_ref`` (a row sees what was accepted before it and itself)."""
import importlib.util
import os

import pytest
import torch

import attn_ref as ref
from test_gpu_attn import built  # noqa: F401  (the module's build fixture)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def streams(built):  # noqa: F811
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "paged_step.py")
    spec = importlib.util.spec_from_file_location("paged_step", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    rows = []
    example.main(5, accepted=rows)
    assert [q.shape[0] for q, *_ in rows] == [n + 5 * len(example.PATH) for n in example.PROMPTS]
    return rows


def test_every_accepted_row(streams):
    for b, (q, k, v, got) in enumerate(streams):
        vis = torch.ones((q.shape[0],) * 2, dtype=torch.bool, device=q.device).tril()
        ref.check(got, None, ref.attend(q, k, v, vis, q.shape[2] ** -0.5), f"stream {b}")


@pytest.mark.parametrize("what", ["dropped", "foreign"])
def test_a_wrong_set_of_tokens_would_be_seen(streams, what):
    """The reference with a token less, or with one of the row's successors: no row of a step is within the bounds then."""
    for q, k, v, got in streams:
        n = q.shape[0]
        vis = torch.ones((n, n), dtype=torch.bool, device=q.device).tril()
        for row in range(n - 8, n - 1):
            wrong = vis[row:row + 1].clone()
            wrong[0, row + 1 if what == "foreign" else row // 2] = what == "foreign"
            with pytest.raises(AssertionError):
                ref.check(got[row:row + 1], None, ref.attend(q[row:row + 1], k, v, wrong, q.shape[2] ** -0.5))
