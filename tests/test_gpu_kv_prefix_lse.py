"""The log-sum-exp of the attention over a shared prefix: a number wherever a row sees a
token, -inf where it sees none, never NaN for finite inputs."""
import numpy as np
import pytest
import torch

import prefix_util as pu
from test_gpu_kv_prefix import ok, with_wide

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dbv():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import draft_block_verification_gb300 as m
    return m


def check_lse(c, got):
    pu.check(c, got)
    _, lse, _, size = pu.exact(c)
    gl = got["lse"].double()
    some = torch.isfinite(lse)
    assert torch.equal(torch.isfinite(gl), some) and (gl[~some] == -float("inf")).all()
    tol = 2.0 ** -16 * size + 2.0 ** -19 * (1 + lse.abs())
    assert ((gl - lse).abs() <= tol)[some].all()


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("D,block", [(64, 16), (128, 64), (128, 128)])
@pytest.mark.parametrize("P", [0, 16, 257, 1000])
@pytest.mark.parametrize("tree", [False, True])
def test_lengths(dbv, tree, P, D, block, wide):
    c = pu.make(70 + P + block, *with_wide([P], [3], [5, 0, 40], [1, 7, 3], wide), 2, 4, D, block,
                tree=tree, pow2=False)
    check_lse(c, pu.run(dbv, c))
    ok(dbv)


@pytest.mark.parametrize("wide", [False, True])
def test_rows_that_see_nothing(dbv, wide):
    """No prefix, no context, masks of which many rows are empty."""
    prefix, sizes, after, new = with_wide([0], [3], [0, 0, 0], [4, 9, 1], wide)
    after = [0] * len(after)
    c = pu.make(71, prefix, sizes, after, new, 2, 4, 128, 16, tree=True)
    r = np.random.RandomState(3)
    c["mask"][r.rand(len(c["mask"])) < 0.5] = 0
    got = pu.run(dbv, c)
    _, lse, _, _ = pu.exact(c)
    assert torch.isinf(lse).any()
    check_lse(c, got)
    assert (got["out"][torch.isinf(lse)] == 0).all()
    ok(dbv)


def test_groups_and_prompts(dbv):
    c = pu.make(72, [300, 64, 1025, 40], [3, 2, 1, 4], [0, 9, 70, 3, 3, 100, 0, 1, 2, 500],
                [3, 0, 5, 7, 1, 9, 133, 2, 0, 400], 2, 3, 128, 16, tree=False, pow2=False)
    check_lse(c, pu.run(dbv, c))
    ok(dbv)
