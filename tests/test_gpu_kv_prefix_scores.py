"""Attention over a shared prefix with scores far from 0, on both sides of what a
maximum in fp32 can tell apart."""
import numpy as np
import pytest
import torch

import kv_util
import prefix_util as pu
from test_gpu_kv_prefix import ok, with_wide

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dbv():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import draft_block_verification_gb300 as m
    return m


def two_heights(c, seed, far, sign):
    """Keys of 256 or 128 in one element, queries with one element: a row's largest
    score, some 2^far log2 units (row by row down to 2^(far - 6)), is that of many
    tokens, all others are half (sign < 0: twice) of it.  Returns the scale."""
    r = np.random.RandomState(seed)
    codes = c["codes"][0]
    dead = codes == 0x7F
    high = r.rand(*codes.shape[:3]) < 0.3
    codes[:] = 0
    codes[..., 3] = np.where(high, *(int(kv_util.e4m3_encode(np.array([x]))[0]) for x in (256.0, 128.0)))
    codes[dead] = 0x7F
    c["scale"][0][:] = 2.0 ** 6
    T, Hq, D = c["q"].shape
    # 256 * 2^6 * 2^(far - 15) [1, 2) * scale / ln 2
    q = torch.zeros((T, Hq, D), device="cuda")
    x = 2.0 ** (far - 15 - r.randint(0, 7, (T, Hq))) * r.uniform(1, 2, (T, Hq))
    q[..., 3] = sign * torch.as_tensor(x, dtype=torch.float32, device="cuda")
    c["q"] = q.bfloat16()
    return float(np.float32(r.uniform(0.7, 1.4)))


def check_heights(c, got, scale):
    """Tolerances.  Scores of one height are the same number, so nothing is lost
    between them: what is left is the output's rounding (2^-8 of its size) and the
    weights' (2^-8 + 2^-11 of sum w|v| / sum w).  Where the two heights are 2^9 apart
    and more the lower weighs nothing; below that (size under 2^11) a score's error
    counts, 2^-15 of its size at most.  lse is a sum in fp32: 2^-20 of its size."""
    want, lse, mag, size = pu.exact(c, scale)
    assert torch.isfinite(lse).all()
    near = torch.where(size < 2.0 ** 11, 2.0 ** -15 * size, 0.0)[..., None]
    tol = 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -11 + near) * mag
    out, gl = got["out"].double(), got["lse"].double()
    bad = ~((out - want).abs() <= tol)
    assert not bad.any(), (bad.nonzero()[:4], out[bad][:4], want[bad][:4], tol[bad][:4])
    assert ((gl - lse).abs() <= 2.0 ** -20 * lse.abs() + 2.0 ** -16).all()


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("pow2", [True, False])
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("far", [10, 14, 17, 20, 24, 27, 29, 33, 60])
def test_scores_far_from_zero(dbv, far, sign, pow2, wide):
    c = pu.make(30 + far, *with_wide([900], [4], [0, 40, 3, 130], [1, 5, 2, 1], wide), 2, 4, 128, 16,
                pow2=pow2)
    scale = two_heights(c, far, far, sign)
    check_heights(c, pu.run(dbv, c, scale=scale), scale)
    ok(dbv)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("far", [16, 28, 45])
def test_far_scores_of_many_rows(dbv, far, D):
    """Draft trees of 40 and prompts: both parts on the prefix kernel, masked tiles, a
    span cut by many CTAs."""
    c = pu.make(31 + far, [5000], [5], [200, 0, 17, 300, 64], [40, 33, 90, 60, 45], 1, 3, D, 64,
                tree=True, pow2=False)
    scale = two_heights(c, far, far, 1.0)
    check_heights(c, pu.run(dbv, c, scale=scale), scale)
    # heights by page, so that maxima move from tile to tile, up and down
    for p in range(0, len(c["codes"][0]), 3):
        k = c["codes"][0][p, :, :, 3]
        k[k != 0x7F] = int(kv_util.e4m3_encode(np.array([128.0]))[0])
    check_heights(c, pu.run(dbv, c, scale=scale), scale)
    ok(dbv)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("spread", [1e5, 1e6, 1e9, 1e15])
def test_large_queries(dbv, spread, wide):
    """Ordinary keys, large queries.  Which token wins is within a score's error; the
    result is finite and among the values, the sum as large as the largest score."""
    c = pu.make(34, *with_wide([1100], [3], [7, 0, 90], [3, 1, 9], wide), 2, 4, 128, 32, pow2=False,
                spread=spread)
    got = pu.run(dbv, c)
    _, lse, _, size = pu.exact(c)
    assert torch.isfinite(got["out"]).all() and torch.isfinite(got["lse"]).all()
    assert float(got["out"].abs().max()) <= 448.0 * float(c["scale"][1].max()) * (1 + 2.0 ** -7)
    assert ((got["lse"].double() - lse).abs() <= 2.0 ** -15 * size + 2.0 ** -19 * (1 + lse.abs())).all()
    ok(dbv)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("scale,spread", [(0.0, 1.0), (None, 2.0 ** -110), (-0.1, 2.0 ** -105)])
def test_hidden_tokens_beside_a_factor_of_zero(dbv, scale, spread, tree, wide):
    """Scores that are 0 whatever the key, among tiles of new tokens: key scales of
    2^-40, which a page of zeros has.  Weights are alike for all that a row sees."""
    prefix, sizes, after, new = with_wide([300], [3], [7, 0, 90], [3, 1, 40], wide)
    c = pu.make(35, prefix, sizes, after, new, 2, 4, 128, 32, tree=tree, pow2=False, spread=spread)
    c["scale"][0][::2] = 2.0 ** -40
    got = pu.run(dbv, c, scale=scale)
    pu.check(c, got, scale)
    _, lse, _, _ = pu.exact(c, scale)
    some = torch.isfinite(lse)
    assert torch.isfinite(got["lse"][some]).all()
    assert ((got["lse"][some].double() - lse[some]).abs() <= 2.0 ** -16).all()
    ok(dbv)
