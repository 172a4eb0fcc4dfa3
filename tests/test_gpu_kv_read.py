"""Tokens read back from the paged 8-bit cache: every element equals the byte's
value times its scale, rounded once."""
import numpy as np
import pytest
import torch

import kv_util

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dbv():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import draft_block_verification_gb300 as m
    return m


def dev(a, dtype=torch.int32):
    return torch.as_tensor(np.asarray(a), dtype=dtype, device="cuda")


def case(seed, first, n, H, D, block, pow2=True):
    r = np.random.RandomState(seed)
    want = [-(-(f + k) // block) for f, k in zip(first, n)]
    pages = sum(want) + 2
    ids, at = r.permutation(pages), 0
    table = np.full((len(n), max(want + [1])), -1, np.int32)
    for b, w in enumerate(want):
        table[b, :w] = ids[at:at + w]
        at += w
    codes = [r.randint(0, 256, (pages, H, block, D)).astype(np.uint8) for _ in range(2)]
    scale = [(2.0 ** r.randint(-9, 3, (pages, H)) if pow2 else
              np.exp(r.uniform(-5, 3, (pages, H)))).astype(np.float32) for _ in range(2)]
    return dict(first=first, n=n, table=table, codes=codes, scale=scale, block=block,
                cu=np.append(0, np.cumsum(n)).astype(np.int32))


def expected(c, side, dtype):
    rows = []
    for b, (f, k) in enumerate(zip(c["first"], c["n"])):
        p = f + np.arange(k)
        page, off = c["table"][b, p // c["block"]], p % c["block"]
        v = kv_util.e4m3_decode(c["codes"][side][page, :, off]).astype(np.float32)
        rows.append(v * c["scale"][side][page][:, :, None])
    x = np.concatenate(rows) if rows else np.zeros((0,) + c["codes"][0].shape[1::2])
    return torch.as_tensor(x, dtype=torch.float32).to(dtype)


def run(dbv, c, rows=None, **kw):
    k, v = (dev(a, torch.uint8).view(torch.float8_e4m3fn) for a in c["codes"])
    ks, vs = (dev(a, torch.float32) for a in c["scale"])
    return dbv.sv_kv_read(k, v, ks, vs, dev(c["table"]), dev(c["cu"]),
                          int(c["cu"][-1]) if rows is None else rows, first=dev(c["first"]), **kw)


def same(got, want):
    got = got.cpu()
    nan = want.isnan()
    return torch.equal(got.isnan(), nan) and torch.equal(got[~nan], want[~nan])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("block", [16, 32, 64, 128])
@pytest.mark.parametrize("H,D", [(1, 64), (3, 128), (8, 64), (5, 64)])
def test_every_element(dbv, H, D, block, dtype):
    for pow2 in (True, False):
        c = case(H + block, [0, 5, 0, 127, 300, 16], [1, 40, 0, 2, 129, 16], H, D, block, pow2)
        got = run(dbv, c, dtype=dtype)
        assert all(same(got[n], expected(c, i, dtype)) for i, n in enumerate("kv"))
    dbv.default_handle(torch.device("cuda", 0)).sync_status()


@pytest.mark.parametrize("B,n", [(1, 1), (1, 5000), (300, 7), (1000, 1)])
def test_many_rows_and_sequences(dbv, B, n):
    r = np.random.RandomState(B)
    c = case(B, r.randint(0, 90, B).tolist(), r.randint(0, n + 1, B).tolist(), 2, 64, 16)
    got = run(dbv, c)
    assert all(same(got[m], expected(c, i, torch.bfloat16)) for i, m in enumerate("kv"))


def test_rows_behind_the_last_sequence_stay(dbv):
    c = case(1, [3, 0], [20, 9], 2, 128, 32)
    out = [torch.full((40, 2, 128), 3.0, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    got = run(dbv, c, rows=40, out=out)
    for i, n in enumerate("kv"):
        assert got[n] is out[i] and (out[i][29:] == 3.0).all()
        assert same(out[i][:29], expected(c, i, torch.bfloat16))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_strided_outputs(dbv, dtype):
    """Heads before tokens, and rows off 16 bytes."""
    c = case(2, [0, 33], [50, 21], 3, 64, 16)
    T = 71
    a = torch.zeros((3, T, 64), dtype=dtype, device="cuda").transpose(0, 1)
    wide = torch.zeros((T, 3 * 64 + 5), dtype=dtype, device="cuda")
    b = wide[:, 1:1 + 3 * 64].unflatten(1, (3, 64))
    run(dbv, c, dtype=dtype, out=(a, b))
    assert same(a, expected(c, 0, dtype)) and same(b, expected(c, 1, dtype))
    assert (wide[:, 0] == 0).all() and (wide[:, 193:] == 0).all()


def test_what_append_wrote_comes_back(dbv):
    """Append, then read: within half a step of e4m3 (2^-4 of the element, 2^-10
    of the scale below the normal ones).  Appending that again gives the same values:
    they are multiples of e4m3's steps at the scale they had, and where rounding has
    brought a page's largest down to 448 of half that scale, twice each byte's value is
    one of e4m3's too."""
    r = np.random.RandomState(4)
    T, H, D, block = 100, 4, 128, 32
    k, v = (torch.as_tensor(r.randn(T, H, D), dtype=torch.float32, device="cuda") for _ in "kv")
    cache = [torch.zeros((4, H, block, D), dtype=torch.float8_e4m3fn, device="cuda") for _ in "kv"]
    scale = [torch.ones((4, H), device="cuda") for _ in "kv"]
    slot = torch.arange(T, dtype=torch.int32, device="cuda")
    dbv.sv_kv_append(k, v, slot, *cache, *scale)
    got = dbv.sv_kv_read(*cache, *scale, dev([[0, 1, 2, 3]]), dev([0, T]), T, dtype=torch.float32)
    for n, x, s in (("k", k, scale[0]), ("v", v, scale[1])):
        step = s[torch.arange(T) // block][:, :, None] * 2.0 ** -10
        assert ((got[n] - x).abs() <= torch.maximum(x.abs() * 2.0 ** -4, step)).all()
    dbv.sv_kv_append(got["k"], got["v"], slot, *cache, *scale)
    again = dbv.sv_kv_read(*cache, *scale, dev([[0, 1, 2, 3]]), dev([0, T]), T,
                           dtype=torch.float32)
    assert all(torch.equal(again[n], got[n]) for n in "kv")


def test_out_of_range_rows_are_latched_and_left(dbv):
    h = dbv.default_handle(torch.device("cuda", 0))
    for what in ("page", "low page", "first", "beyond", "sums"):
        c = case(3, [0, 10], [20, 20], 2, 64, 16)
        if what == "page":
            c["table"][0, 1] = len(c["codes"][0])
        elif what == "low page":
            c["table"][0, 1] = -1
        elif what == "first":
            c["first"] = [-30, 10]
        elif what == "beyond":
            c["first"] = [0, 10 ** 6]
        else:
            c["cu"] = np.array([4, 20, 40], np.int32)
        out = [torch.full((40, 2, 64), 9.0, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
        run(dbv, c, rows=40, out=out)
        with pytest.raises(dbv.SVError) as e:
            h.sync_status()
        assert e.value.status == dbv.SV_ERR_DEVICE_BOUNDS
        left = {"page": range(16, 20), "low page": range(16, 20), "first": range(20),
                "beyond": range(20, 40), "sums": range(4)}[what]
        assert all((o[list(left)] == 9.0).all() for o in out)
    h.sync_status()


def test_in_a_graph_and_on_another_stream(dbv):
    c = case(5, [0, 3, 70], [200, 100, 5], 2, 128, 64)
    want = [expected(c, i, torch.bfloat16) for i in range(2)]
    k, v = (dev(a, torch.uint8).view(torch.float8_e4m3fn) for a in c["codes"])
    args = [k, v, *(dev(a, torch.float32) for a in c["scale"]), dev(c["table"]), dev(c["cu"]), 305]
    first = dev(c["first"])
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        out = dbv.sv_kv_read(*args, first=first)
    g.replay()
    s = torch.cuda.Stream()
    other = dbv.sv_kv_read(*args, first=first, stream=s)
    torch.cuda.synchronize()
    for i, n in enumerate("kv"):
        assert same(out[n], want[i]) and same(other[n], want[i])
