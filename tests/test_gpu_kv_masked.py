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
