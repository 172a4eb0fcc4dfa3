"""Attention over the paged cache where the pages' value scales lie far apart:
every page's values count with the same precision, whatever the others' scales."""
import pytest
import torch

from test_gpu_kv_units import call, case, check, tiles

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dbv():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import draft_block_verification_gb300 as m
    return m


SHAPES = [  # lens, new, H, G, D, block
    ([500], 1, 2, 4, 128, 64),
    ([300, 41, 900], 5, 2, 4, 64, 16),
    ([100] * 150, 9, 2, 4, 128, 32),
    ([600] * 100, 17, 2, 3, 64, 128),
    ([9000, 20000], 12, 2, 4, 128, 16),
    ([1500, 260], 33, 1, 4, 128, 64),
    ([400] * 90, 60, 1, 2, 128, 16),
]


def spread(c, kind, seed):
    """Value scales of the pages of c, in place."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = c["scale"][1]
    r = torch.rand(s.shape, generator=g, device="cuda")
    if kind == "outlier":       # one page in five, 2^16 over the others
        s.mul_(torch.where(r < 0.2, 2.0 ** 16, 1.0))
    elif kind == "two":         # 2^12 apart, evenly
        s.mul_(torch.where(r < 0.5, 2.0 ** 12, 1.0))
    elif kind == "wide":        # anything from 2^-38 to 2^-2
        s.copy_(torch.exp2(-38 + 36 * r))
    elif kind == "ends":        # the ends of the range and the middle
        s.copy_(torch.exp2(40.0 * torch.floor(r * 3) - 40))
    elif kind == "zeros":       # pages of zeros, at the least scale
        none = r < 0.3
        s.masked_fill_(none, 2.0 ** -40)
        c["cache"][1][none] = 0
    # channel d has values only in the pages up to a scale that rises with d, so that
    # the first channels come from the pages of the least scales alone
    e = torch.log2(s).floor()
    top = e.min() + (e.max() - e.min()) * torch.linspace(0, 1, c["D"], device="cuda")
    c["cache"][1].masked_fill_((e[..., None] > top)[:, :, None], 0)
    # (what lies past a sequence's end stays NaN)
    for b, L in enumerate(c["kv"]):
        if L % c["block"]:
            c["cache"][1][int(c["table"][b, L // c["block"]]), :, int(L % c["block"]):] = 0x7F


@pytest.mark.parametrize("kind", ["outlier", "two", "wide", "ends", "zeros"])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_value_scales_far_apart(dbv, shape, kind):
    lens, new, H, G, D, block = SHAPES[shape]
    c = case(shape, lens, [new] * len(lens), H, G, D, block, tree=shape % 3 == 1)
    spread(c, kind, shape)
    out = call(dbv, c)
    check(c, out)
    again = call(dbv, c)
    assert torch.equal(out["out"], again["out"]) and torch.equal(out["lse"], again["lse"])
    dbv.default_handle(c["q"].device).sync_status()


@pytest.mark.parametrize("apart", [12, 16, 18, 30])
def test_small_values_beside_an_outlier_page(dbv, apart):
    """A page whose scale is large for a value that this channel does not have:
    the channel's output comes from the other page alone."""
    D, block = 128, 64
    c = case(1, [block], [block], 1, 1, D, block)
    c["q"].zero_()                                   # equal weights
    one = kv_code(1.0)
    c["cache"][1].fill_(one)
    first, second = (int(c["table"][0, i]) for i in range(2))
    c["cache"][1][first] = 0
    c["cache"][1][first, 0, 0, 5] = kv_code(448.0)   # the outlier, in channel 5
    c["scale"][1][first], c["scale"][1][second] = 2.0 ** (apart - 8), 2.0 ** -8
    check(c, call(dbv, c))
    out = call(dbv, c)["out"][:, 0].double()
    n = torch.arange(1, block + 1, device="cuda").double()
    want = n / (block + n) * 2.0 ** -8
    assert ((out[:, 6] - want).abs() <= 2.0 ** -7 * want).all()


def kv_code(x):
    return int(torch.tensor([x]).to(torch.float8_e4m3fn).view(torch.uint8)[0])


def test_low_scores_in_one_scale_class(dbv):
    """Classes whose rows see little or nothing, and scores far below zero."""
    c = case(4, [0] * 40, [150] * 40, 2, 1, 128, 16)
    assert tiles(c) >= 160
    spread(c, "wide", 9)
    c["q"] = (c["q"].float().abs() + 0.5).bfloat16()
    live = c["cache"][0] != 0x7F
    key = (torch.rand(live.shape, device="cuda") * 16 + 208).to(torch.float8_e4m3fn)
    c["cache"][0] = torch.where(live, key.view(torch.uint8) | 0x80, c["cache"][0])
    c["scale"][0][:] = 2.0 ** -6
    f = 120.0 / (128 * 1.3 * 216 * 2.0 ** -6)
    check(c, call(dbv, c, scale=f), f)


def test_nan_and_empty_rows_with_scales_far_apart(dbv):
    c = case(5, [130, 0], [40, 33], 2, 2, 64, 16, tree=True)
    spread(c, "wide", 3)
    c["mask"][3] = 0
    c["mask"][50] = 0
    c["q"][7, 1, 3] = float("nan")
    out = call(dbv, c)
    assert torch.isnan(out["out"][7, 1]).all() and torch.isnan(out["lse"][7, 1])
    c["q"][7, 1] = 0
    fine = call(dbv, c)
    out["out"][7, 1], out["lse"][7, 1] = fine["out"][7, 1], fine["lse"][7, 1]
    check(c, out)
    assert (out["out"][50] == 0).all() and torch.isinf(out["lse"][50]).all()
