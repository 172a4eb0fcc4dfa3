"""Attention over the paged cache where every CTA has several tiles and units:
stages that are used again, sums carried from tile to tile, units that CTAs
share, several units a CTA.  The reference is a plain fp64 form on the GPU."""
import numpy as np
import pytest
import torch

import kv_util

pytestmark = pytest.mark.gpu

CLASS = 6  # value scales less than 2^6 apart share the weights' last step


@pytest.fixture(scope="module")
def dbv():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import draft_block_verification_gb300 as m
    return m


def case(seed, lens, new, H, G, D, block, tree=False, spread=1.0, qscale=1.0):
    """Sequences of lens[b] + new[b] tokens in shuffled pages, on the GPU.  Bytes
    past a sequence's end are NaN.  Value scales lie within 2^spread."""
    r = np.random.RandomState(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    lens, new = np.asarray(lens), np.asarray(new)
    kv = lens + new
    want = -(-kv // block)
    pages = int(want.sum()) + 2
    order = r.permutation(pages)[:want.sum()]
    table = np.full((len(kv), max(int(want.max()), 1)), -1, np.int32)
    at = 0
    for b, w in enumerate(want):
        table[b, :w] = order[at:at + w]
        at += w
    dev = dict(device="cuda")
    cache = [(torch.randn((pages, H, block, D), generator=g, **dev) * 60).clamp_(-448, 448)
             .to(torch.float8_e4m3fn).view(torch.uint8) for _ in range(2)]
    for b, L in enumerate(kv):
        if L % block:
            for c in cache:
                c[int(table[b, L // block]), :, int(L % block):] = 0x7F
    scale = [torch.exp2(torch.rand((pages, H), generator=g, **dev) * spread - 8)
             for _ in range(2)]
    T = int(new.sum())
    q = (torch.randn((T, H * G, D), generator=g, **dev) * qscale).bfloat16()
    cu = np.append(0, np.cumsum(new)).astype(np.int32)
    mask = None
    if tree:
        words = max(1, -(-int(new.max()) // 32))
        mask = np.zeros((T, words), np.uint32)
        for b, n in enumerate(new):
            for i in range(n):
                t = cu[b] + i
                if i and r.rand() < 0.9:
                    mask[t] = mask[cu[b] + r.randint(i)]
                if r.rand() < 0.95:
                    mask[t, i // 32] |= np.uint32(1 << (i % 32))
    return dict(q=q, cache=cache, scale=scale, table=table, kv=kv, cu=cu, mask=mask, block=block,
                H=H, G=G, D=D)


def tiles(c):
    """Tiles of 128 tokens of the call, over all units."""
    n = np.diff(c["cu"]) * c["G"]
    return int((-(-c["kv"] // 128) * -(-n // 128)).sum()) * c["H"]


def call(dbv, c, **kw):
    i32 = lambda a: torch.as_tensor(np.asarray(a), dtype=torch.int32, device="cuda")  # noqa: E731
    m = None if c["mask"] is None else i32(c["mask"].view(np.int32))
    return dbv.sv_kv_attention(c["q"], *c["cache"], *c["scale"], i32(c["table"]), i32(c["kv"]),
                               i32(c["cu"]), mask=m, want_lse=True, **kw)


def decoded(codes):
    t = np.concatenate([kv_util.e4m3_decode(np.arange(256))])
    return torch.as_tensor(t, dtype=torch.float64, device="cuda")[codes.long()]


def reference(c, b, softmax_scale=None):
    """(out, lse, tolerance of out, tolerance of lse) of sequence b in fp64.

    The tolerance of an output: its rounding to bf16, 2^-8 of it and 2^-133; a
    weight w of a value of scale s is held as w s in two parts of e4m3, off by
    (2^-8 + 2^-11) of itself and by 2^-17.5 of the largest w s among the row's
    tokens whose scales are less than 2^CLASS apart, which reaches the output
    times the 8-bit value; a score is a sum of 256 exact products in fp32
    (2^-16 of sum |q||k|), of queries that are off by 2^-17 of the row's largest,
    and its exponential and the sums are off by 2^-16 of the score's size + 1."""
    H, G, D, block = c["H"], c["G"], c["D"], c["block"]
    L, lo, hi = int(c["kv"][b]), int(c["cu"][b]), int(c["cu"][b + 1])
    n = hi - lo
    pages = torch.as_tensor(c["table"][b, :-(-L // block)].astype(np.int64), device="cuda")
    vals, s = [], None
    for x, y in zip(c["cache"], c["scale"]):
        code = decoded(x[pages]).transpose(0, 1).reshape(H, -1, D)[:, :L]
        s = y[pages].double().t().repeat_interleave(block, 1)[:, :L]
        vals.append((code, s))
    K = vals[0][0] * vals[0][1][..., None]
    code, s = vals[1]
    sees = torch.as_tensor(np.stack([
        kv_util.sees(i, n, L - n, L, None if c["mask"] is None else c["mask"][lo + i])
        for i in range(n)]), device="cuda").repeat_interleave(G, 0)  # [n G, L]
    K = torch.where(sees.any(0)[:, None], K, 0.0)
    code = torch.where(sees.any(0)[:, None], code, 0.0)
    q = c["q"][lo:hi].double().reshape(n, H, G, D).transpose(0, 1).reshape(H, n * G, D)
    f = D ** -0.5 if softmax_scale is None else softmax_scale
    z = (q @ K.transpose(1, 2) * f).masked_fill(~sees, -np.inf)
    top = z.amax(2, keepdim=True)
    top = torch.where(top == -np.inf, 0.0, top)
    w = torch.exp(z - top)
    mass = w.sum(2, keepdim=True)
    some = mass > 0
    mass = torch.where(some, mass, 1.0)
    out = (w * s[:, None]) @ code / mass
    mag = (w * s[:, None]) @ code.abs() / mass
    e = torch.floor(torch.log2(s)).long()
    step = torch.zeros_like(out)
    for x in e.unique().tolist():  # tokens of one scale exponent at a time
        near = (e - x).abs() < CLASS
        most = (w * torch.where(near, s, 0.0)[:, None]).amax(2, keepdim=True)
        step += most * ((sees & (e == x)[:, None]).double() @ code.abs())
    size = ((q.abs() @ K.abs().transpose(1, 2)).masked_fill(~sees, 0.0).amax(2, keepdim=True)
            + q.abs().amax(2, keepdim=True) * K.abs().sum(2).amax(1)[:, None, None]) * abs(f)
    rel = 2.0 ** -15 * size + 2.0 ** -15 * (1 + torch.abs(top))
    tol = 2.0 ** -8 * out.abs() + 2.0 ** -133 + (2.0 ** -8 + 2.0 ** -11 + rel) * mag + \
        2.0 ** -17.5 * step / mass
    lse = torch.where(some, top + torch.log(mass), -np.inf)
    back = lambda t: t.reshape(H, n, G, -1).transpose(0, 1).reshape(n, H * G, -1)  # noqa: E731
    return back(out), back(lse)[..., 0], back(tol), back(rel)[..., 0]


def check(c, out, softmax_scale=None, sequences=None):
    for b in range(len(c["kv"])) if sequences is None else sequences:
        lo, hi = int(c["cu"][b]), int(c["cu"][b + 1])
        if lo == hi:
            continue
        want, lse, tol, rel = reference(c, b, softmax_scale)
        got, gl = out["out"][lo:hi].double(), out["lse"][lo:hi].double()
        bad = ~((got - want).abs() <= tol)
        assert not bad.any(), (b, bad.nonzero()[:3].tolist(), got[bad][:3], want[bad][:3])
        assert torch.equal(torch.isinf(gl), torch.isinf(lse)), b
        ok = torch.isfinite(lse)
        assert ((gl - lse).abs()[ok] <= rel[ok]).all(), b


# rows of a unit: those where some warps have a query row less than others (5, 9,
# 10, 13 to 15), the borders of the products' widths, more than one row block
MANY = [(1, 5), (1, 9), (2, 5), (1, 13), (2, 7), (3, 5), (1, 1), (4, 4), (17, 1), (8, 4),
        (11, 3), (16, 3), (16, 4), (13, 5), (24, 4), (25, 4), (32, 4), (43, 3), (40, 7)]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new,G", MANY)
def test_several_units_a_cta(dbv, new, G, D):
    """Short sequences of unequal length: spans end inside units, and a CTA that
    joins a shared unit goes on to others.  The same again, bit for bit."""
    r = np.random.RandomState(new * 16 + G)
    B, H = 300 if new * G <= 64 else 130, 2
    c = case(new + G, r.randint(0, 900, B), np.full(B, new), H, G, D, 32, tree=new == 11)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert tiles(c) > 3 * sms
    out = call(dbv, c)
    check(c, out)
    for _ in range(20):
        again = call(dbv, c)
        assert torch.equal(out["out"], again["out"]) and torch.equal(out["lse"], again["lse"])
    dbv.default_handle(c["q"].device).sync_status()


@pytest.mark.parametrize("new,G,D,block", [(1, 5, 128, 16), (5, 6, 64, 128), (9, 4, 64, 16),
                                           (17, 4, 128, 64), (12, 8, 128, 32), (30, 4, 64, 32),
                                           (33, 4, 128, 16)])
def test_long_units_shared_by_many_ctas(dbv, new, G, D, block):
    """Tens of tiles a CTA, pages looked up in many windows."""
    H = 2
    lens = [60000, 33333, 127, 70001]
    c = case(new, lens, [new, max(1, new - 1), new, 1], H, G, D, block, tree=new == 12)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert tiles(c) > 8 * sms
    out = call(dbv, c)
    check(c, out)
    again = call(dbv, c)
    assert torch.equal(out["out"], again["out"]) and torch.equal(out["lse"], again["lse"])
    dbv.default_handle(c["q"].device).sync_status()


@pytest.mark.parametrize("new,G", [(1, 4), (4, 8), (12, 4), (20, 6)])
@pytest.mark.parametrize("rising", [True, False])
def test_maximum_that_moves(dbv, rising, new, G):
    """Scores that rise along the sequence, by tens from tile to tile, or fall:
    every CTA has several tiles, so sums are rescaled."""
    H, D, block, L = 2, 128, 64, 80000
    c = case(3, [L] * 3, [new] * 3, H, G, D, block)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert tiles(c) > 4 * sms
    p = torch.arange(c["table"].shape[1] * block, device="cuda") / (L + new)
    f = (p if rising else 1 - p).clamp(0, 1)[:, None] * 300 + torch.zeros(D, device="cuda")
    code = f.to(torch.float8_e4m3fn).view(torch.uint8).reshape(-1, block, D)
    for b in range(3):
        c["cache"][0][torch.as_tensor(c["table"][b].astype(np.int64), device="cuda")] = \
            code[:, None]
    c["scale"][0][:] = 2.0 ** -6
    c["q"] = c["q"].abs()
    check(c, call(dbv, c, scale=1.0), 1.0)
