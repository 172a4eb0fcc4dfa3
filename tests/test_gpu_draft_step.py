"""The example's steps: every sequence's tokens, lengths and pages add up, and
the same steps give the same tokens."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import draft_step
    return draft_step


@pytest.mark.parametrize("block", [16, 64])
@pytest.mark.parametrize("K", [0, 1, 5])
def test_steps_add_up(example, K, block):
    B, steps = 5, 7
    told, s, accepted = example.run(steps=steps, B=B, K=K, block=block, pages=60)
    assert sum(map(len, told)) == B * steps + accepted
    assert 0 <= accepted <= B * steps * K
    assert s["cached"].tolist() == [len(t) for t in told]
    # held pages cover the last block; with the free ones they are all
    want = [-(-c // block) for c in s["cached"].tolist()]
    assert all(h >= w for h, w in zip(s["held"].tolist(), want))
    free = s["free_pos"].tolist()
    assert free[1] - free[0] + int(s["held"].sum()) == s["pages"]
    end = s["end_free"].tolist()
    assert end[1] - end[0] == s["pages"] and s["end_held"].tolist() == [0] * B
    queue = s["free_ids"][[i % s["pages"] for i in range(*end)]].tolist()
    assert sorted(queue) == list(range(s["pages"]))


def test_the_same_steps_again(example):
    """The same seed gives the same tokens, bit for bit."""
    a = example.run(steps=4, B=6, K=3, pages=60, seed=3)
    b = example.run(steps=4, B=6, K=3, pages=60, seed=3)
    assert a[0] == b[0] and a[2] == b[2]
