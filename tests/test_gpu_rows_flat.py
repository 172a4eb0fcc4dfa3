"""sv_sample_rows on long rows of equal or nearly equal logits, where a whole row
weighs far more than the tokens that top-k keeps."""
import pytest
import torch

from test_gpu_rows import check, full

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dbv():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import draft_block_verification_gb300 as m
    return m


def k_of(R, k):
    return full(R, k, torch.int32)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [65536, 65537, 131072, 262144, 1 << 20])
def test_top_k_with_top_p_on_equal_rows(dbv, V, dtype):
    """All logits are equal: the kept tokens are the first ones by id."""
    for fill in (0.0, 3.5, -100.0):
        x = torch.full((3, V), fill, dtype=dtype, device="cuda")
        u = torch.tensor([0.03, 0.5, 0.97], device="cuda")
        for k in (1, 2, 50, 4096, 4097, 60000):
            check(dbv, x, u, k=k_of(3, k), p=full(3, 0.95))
        check(dbv, x, u, k=k_of(3, 50), p=full(3, 0.617), m=full(3, 0.5))
        check(dbv, x, u, k=k_of(3, 50), p=full(3, 0.0))
    out = dbv.sv_sample_rows(torch.zeros((1, V), dtype=dtype, device="cuda"), u[:1],
                             top_k=k_of(1, 50), top_p=full(1, 0.95))
    assert out["kept"].tolist() == [48] and out["token"].tolist() == [1]


@pytest.mark.parametrize("V", [65536, 131072, 1 << 20])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_top_k_with_top_p_on_nearly_equal_rows(dbv, V, dtype):
    """Positive logits within 2^-7 of each other: few values in bf16, many in
    fp32; and rows of which more than half are equal to the largest."""
    g = torch.Generator(device="cuda").manual_seed(V)
    R = 4
    u = torch.rand(R, generator=g, device="cuda")
    near = (1 + torch.rand((R, V), generator=g, device="cuda") * 2.0 ** -7).to(dtype)
    half = torch.where(torch.rand((R, V), generator=g, device="cuda") < 0.6, 2.0,
                       torch.randn((R, V), generator=g, device="cuda").clamp(max=1.9)).to(dtype)
    for x in (near, half):
        for k in (3, 50, 1000, 4096, 5000):
            for p in (0.3, 0.617, 0.983):
                check(dbv, x, u, k=k_of(R, k), p=full(R, p))
        check(dbv, x, u, k=k_of(R, 64), p=full(R, 0.7), T=full(R, 50.0))


def test_infinities_share_the_weight(dbv):
    """More +inf logits than the list holds, with both filters."""
    V = 131072
    x = torch.zeros((2, V), device="cuda")
    x[0, :] = float("inf")
    x[1, ::2] = float("inf")
    u = torch.tensor([0.4, 0.8], device="cuda")
    for k in (7, 50, 4096, 50000):
        check(dbv, x, u, k=k_of(2, k), p=full(2, 0.777))
