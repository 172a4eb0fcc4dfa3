"""Attention over the paged cache where rows see nothing in a part of the work,
scores are very low, and masked places hold NaN."""
import numpy as np
import pytest
import torch

from test_gpu_kv_units import call, case, check, reference, tiles

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dbv():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import draft_block_verification_gb300 as m
    return m


@pytest.mark.parametrize("B", [1, 200])
@pytest.mark.parametrize("new,G,H", [(130, 1, 2), (140, 4, 1), (260, 2, 1)])
def test_low_scores_beside_tiles_that_a_row_does_not_see(dbv, B, new, G, H):
    """Blocks of new tokens across borders of 128: the early rows see nothing of
    the later tiles, and every score that they do see is about -110 (-250), so
    that a maximum of 0 for what is not seen would flush all of theirs."""
    for low in (110.0, 250.0):
        c = case(B + new, [0] * B, [new] * B, H, G, 128, 64)
        if B > 1:  # several tiles a CTA, so that one CTA joins both pairs' sums
            assert tiles(c) > torch.cuda.get_device_properties(0).multi_processor_count
        q = c["q"].float().abs() + 0.5
        c["q"] = q.bfloat16()
        live = c["cache"][0] != 0x7F
        key = (torch.rand(live.shape, device="cuda") * 16 + 208).to(torch.float8_e4m3fn)
        c["cache"][0] = torch.where(live, key.view(torch.uint8) | 0x80, c["cache"][0])
        c["scale"][0][:] = 2.0 ** -6
        # a row's mean score is -low for its mean |q| of about 1.3
        f = low / (128 * 1.3 * 216 * 2.0 ** -6)
        out = call(dbv, c, scale=f)
        check(c, out, f)
        assert torch.isfinite(out["lse"]).all()


def check_rows(c, out, lost):
    """Rows of `lost` [T, Hq] are NaN, the others as the reference has them."""
    for b in range(len(c["kv"])):
        lo, hi = int(c["cu"][b]), int(c["cu"][b + 1])
        want, lse, tol, rel = reference(c, b)
        got, gl, bad = out["out"][lo:hi].double(), out["lse"][lo:hi].double(), lost[lo:hi]
        assert torch.isnan(got[bad]).all() and torch.isnan(gl[bad]).all(), b
        ok = ~bad
        assert ((got - want).abs() <= tol)[ok].all(), b
        assert torch.equal(torch.isinf(gl[ok]), torch.isinf(lse[ok])), b
        ok &= torch.isfinite(lse)
        assert ((gl - lse).abs() <= rel)[ok].all(), b


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new,G,lens", [(1, 4, [300, 40000]), (5, 4, [1000] * 60), (9, 8, [700]),
                                        (33, 4, [2000, 90])])
def test_queries_that_are_not_finite(dbv, new, G, lens, D):
    """A row whose query holds NaN or an infinity is NaN, in units of one CTA and
    in shared ones, and no other row is."""
    B, H = len(lens), 2
    c = case(new, lens, [new] * B, H, G, D, 32)
    clean = dict(c, q=c["q"].clone())
    r = np.random.RandomState(D)
    lost = torch.zeros(c["q"].shape[:2], dtype=torch.bool, device="cuda")
    for i, bad in enumerate((float("nan"), float("inf"), -float("inf"))):
        for _ in range(max(1, B // 4)):
            t, h, d = r.randint(c["q"].shape[0]), r.randint(H * G), r.randint(D)
            c["q"][t, h, d] = bad
            lost[t, h] = True
    check_rows(clean, call(dbv, c), lost)
    dbv.default_handle(c["q"].device).sync_status()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new,G,lens", [(4, 4, [300, 128, 0]), (20, 1, [100, 250] * 100),
                                        (33, 2, [2000, 90]), (60, 2, [200, 77]),
                                        (150, 1, [60, 0])])
@pytest.mark.parametrize("side", [0, 1])
@pytest.mark.parametrize("tree", [False, True])
def test_new_tokens_that_are_nan(dbv, tree, side, new, G, lens, D):
    """NaN in the key or value of some new tokens: rows that see one are NaN, the
    rows that do not are as if its bytes were zero."""
    B, H, block = len(lens), 2, 32
    c = case(new, lens, [new] * B, H, G, D, block, tree=tree)
    r = np.random.RandomState(D + new)
    clean = dict(c, cache=[x.clone() for x in c["cache"]])
    lost = torch.zeros(c["q"].shape[:2], dtype=torch.bool, device="cuda")
    for b in range(0, B, 1 if B < 10 else 3):
        for j in (new - 1, new // 2 + r.randint(new // 2)):
            if tree and j == new - 1:  # one that no row sees
                c["mask"][c["cu"][b]:c["cu"][b + 1], j // 32] &= ~np.uint32(1 << (j % 32))
            p, h, d = lens[b] + j, r.randint(H), r.randint(D)
            page = int(c["table"][b, p // block])
            c["cache"][side][page, h, p % block, d] = r.choice([0x7F, 0xFF])
            clean["cache"][side][page, h, p % block] = 0
            for i in range(new):
                t = int(c["cu"][b]) + i
                sees = (c["mask"][t, j // 32] >> (j % 32)) & 1 if tree else j <= i
                if sees:
                    lost[t, h * G:(h + 1) * G] = True
    assert lost.any() and not lost.all()
    check_rows(clean, call(dbv, c), lost)
    dbv.default_handle(c["q"].device).sync_status()
