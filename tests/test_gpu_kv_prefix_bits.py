"""What the attention over a shared prefix keeps of its weights and values: few tokens
count, so that no rounding is averaged away."""
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


def few(c, seed, n):
    """Of every page one token in n counts, with a score of -2 to 6 for q = 1 in one
    element; the others' are 40 below and more.  Queries 1 to 2."""
    r = np.random.RandomState(seed)
    codes = c["codes"][0]
    dead = codes == 0x7F
    x = r.choice([-2, -1.5, -1.25, -1, -0.5, 0.5, 1, 1.5, 2, 2.5, 3.5, 5, 6], codes.shape[:3]) * 8
    x = np.where(r.rand(*codes.shape[:3]) < 1.0 / n, x, -448.0)
    codes[:] = 0
    codes[..., 7] = kv_util.e4m3_encode(x)
    codes[dead] = 0x7F
    c["scale"][0][:] = 0.125
    q = torch.zeros(c["q"].shape, device="cuda")
    q[..., 7] = torch.as_tensor(r.uniform(1, 2, q.shape[:2]), dtype=torch.float32, device="cuda")
    c["q"] = q.bfloat16()


def check_bits(c, got):
    """Tolerances.  The output's rounding, 2^-8 of its size.  A weight's, 2^-11 of itself
    (of sum w|v| / sum w), and 2^-12 for the exponential, log2 of a scale's fraction and
    the score's factor (a score is one product here, within 2^-22 of itself, 2^-18 in all
    for scores below 2^4).  Weights far below the largest: 2^-30 of it each."""
    want, lse, mag, size = pu.exact(c, 1.0)
    assert float(size.max()) < 130 and torch.isfinite(lse).all()
    top = 448.0 * float(c["scale"][1].max())
    tol = 2.0 ** -8 * want.abs() + (2.0 ** -11 + 2.0 ** -12) * mag + float(c["kv"].max()) * 2.0 ** -30 * top
    out, gl = got["out"].double(), got["lse"].double()
    bad = ~((out - want).abs() <= tol)
    assert not bad.any(), (bad.sum(), bad.nonzero()[:4], out[bad][:4], want[bad][:4], tol[bad][:4])
    assert ((gl - lse).abs() <= 2.0 ** -16 * (1 + lse.abs())).all()


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("pow2", [True, False])
@pytest.mark.parametrize("D,block,n", [(128, 16, 64), (64, 64, 300), (128, 128, 200)])
def test_weights_keep_eleven_bits(dbv, D, block, n, pow2, wide):
    c = pu.make(50 + n, *with_wide([1500], [4], [0, 40, 3, 130], [1, 5, 2, 1], wide), 2, 4, D, block,
                pow2=pow2)
    few(c, n, n)
    check_bits(c, pu.run(dbv, c, scale=1.0))
    ok(dbv)


@pytest.mark.parametrize("tree", [False, True])
def test_many_rows_keep_eleven_bits(dbv, tree):
    """Both parts on the prefix kernel, masked tiles, one and both slots of a unit."""
    c = pu.make(51, [2100, 300], [3, 2], [200, 0, 17, 300, 64], [40, 33, 90, 60, 45], 1, 3, 128, 64,
                tree=tree, pow2=False)
    few(c, 51, 40)
    check_bits(c, pu.run(dbv, c, scale=1.0))
    ok(dbv)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("spread", [5, 9, 30])
def test_pages_of_unlike_value_scales(dbv, spread, D):
    """Some tiles' values lie too far apart for fp16 and go to bf16: a weight is held to
    2^-8 there.  Tokens of all pages count alike, |v| is much the same whatever the page."""
    c = pu.make(52, [2100, 300], [3, 2], [200, 0, 17, 300, 64], [40, 33, 90, 60, 45], 1, 3, D, 16,
                pow2=False)
    r = np.random.RandomState(spread)
    up = r.randint(0, 2, c["scale"][1].shape) * (r.rand(*c["scale"][1].shape) < 0.2)
    c["scale"][1] *= np.float32(2.0) ** (up * spread).astype(np.float32)
    small = up[..., None, None] > 0
    live = c["codes"][1] != 0x7F
    v = c["codes"][1]
    near0 = kv_util.e4m3_encode(r.uniform(-2, 2, v.shape) * 2.0 ** -min(spread, 9))
    v[:] = np.where(small & live, near0, v)
    pu.check(c, pu.run(dbv, c))
    ok(dbv)


@pytest.mark.parametrize("far", [0, 20])
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("P", [256, 304, 700])
def test_a_stored_value_of_nan(dbv, P, wide, far):
    """A token before the new ones whose value holds NaN, in a shared page or a
    sequence's own: rows that see it are NaN there, no other row is, wherever the
    shared tokens end in a tile."""
    prefix, sizes, after, new = with_wide([P], [3], [10, 0, 90], [4, 6, 5], wide)
    c = pu.make(53, prefix, sizes, after, new, 2, 4, 128, 16, far=far)
    for at, rows in ((3, slice(0, 15)), (P // 16 * 16 - 1, slice(0, 15)), (P + 80, slice(10, 15))):
        seq = 2 if at >= P else 0
        page, row = c["table"][seq, at // 16], at % 16
        was = c["codes"][1][page, 1, row, 9]
        c["codes"][1][page, 1, row, 9] = 0xFF
        got = pu.run(dbv, c)["out"]
        c["codes"][1][page, 1, row, 9] = was
        lost = torch.zeros(got.shape[:2], dtype=torch.bool, device="cuda")
        lost[rows, 4:] = True  # heads of cache head 1
        assert got[..., 9].isnan().equal(lost), at
        assert got[~lost].isfinite().all(), at
    if wide:  # a sequence of many rows: its own context
        lo = sum(new[:3])
        at = 40
        page, row = c["table"][3, at // 16], at % 16
        c["codes"][1][page, 0, row, 5] = 0x7F
        got = pu.run(dbv, c)["out"]
        lost = torch.zeros(got.shape[:2], dtype=torch.bool, device="cuda")
        lost[lo:, :4] = True
        assert got[..., 5].isnan().equal(lost) and got[~lost].isfinite().all()
    ok(dbv)
