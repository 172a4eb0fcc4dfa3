"""Reading the cache back rounds a product once, beside the middle of two bf16 steps too."""
import numpy as np
import pytest
import torch

import kv_util
from test_gpu_kv_read import dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dbv():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import draft_block_verification_gb300 as m
    return m


def once(x):
    """fp64 to bf16's values, ties to even (a product has 28 bits, exact in fp64)."""
    m, e = np.frexp(x)
    return np.ldexp(np.rint(m * 256), e - 8)


def beside(n, seed):
    """Scales whose product with 9, 11, 13 or 15 eighths lies beside a middle, not in it,
    where fp32 has the middle itself."""
    r = np.random.RandomState(seed)
    found = []
    while len(found) < n:
        a = r.choice([9, 11, 13, 15]) / 8
        mid = (2 * r.randint(128, 256) + 1) / 512 * 2.0 ** r.randint(-9, 4)
        s = np.float32(mid / a)
        if np.float32(np.float32(a) * s) == mid and float(s) * a != mid:
            found.append(s)
    return np.array(found, np.float32)


@pytest.mark.parametrize("aligned", [True, False])
def test_products_beside_a_middle(dbv, aligned):
    pages, H, D, block = 64, 4, 64, 16
    r = np.random.RandomState(1)
    eighths = kv_util.e4m3_encode(np.array([9, 11, 13, 15]) / 8)
    codes = [eighths[r.randint(0, 4, (pages, H, block, D))] | (r.randint(0, 2, (pages, H, block, D)) << 7)
             for _ in "kv"]
    for c in codes:
        c[:, :, 3] = r.randint(0, 256, c[:, :, 3].shape)  # (any byte, NaN too)
    scale = [beside(pages * H, 2 + i).reshape(pages, H) for i in range(2)]
    T = pages * block
    wide = [torch.zeros((T, H * D + 5), dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    out = None if aligned else [w[:, 1:1 + H * D].unflatten(1, (H, D)) for w in wide]
    k, v = (dev(c.astype(np.uint8), torch.uint8).view(torch.float8_e4m3fn) for c in codes)
    got = dbv.sv_kv_read(k, v, *(dev(s, torch.float32) for s in scale),
                         dev(np.arange(pages)[None].astype(np.int32)), dev([0, T]), T, out=out)
    for n, c, s in zip("kv", codes, scale):
        exact = kv_util.e4m3_decode(c.astype(np.uint8)) * s.astype(np.float64)[:, :, None, None]
        exact = exact.transpose(0, 2, 1, 3).reshape(T, H, D)
        want, twice = once(exact), once(exact.astype(np.float32).astype(np.float64))
        assert (want != twice)[~np.isnan(want)].sum() > 1000  # (what rounding twice would give)
        have = got[n].double().cpu().numpy()
        assert np.array_equal(np.isnan(have), np.isnan(want))
        assert np.array_equal(have[~np.isnan(want)], want[~np.isnan(want)])
    dbv.default_handle(torch.device("cuda", 0)).sync_status()
