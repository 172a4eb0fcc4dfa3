"""Norms of queries and keys with the rotation, against the formula in 64 bits."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dbv():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import draft_block_verification_gb300 as m
    return m


def formula(x, pos, inv_freq, w, eps, inter):
    """(y, size): the result in 64 bits, and |x'_a| + |x'_b| of each element's pair."""
    x = x.double()
    if w is not None:
        x = x / ((x * x).mean(-1, keepdim=True) + eps).sqrt() * w.double()
    y, size = x.clone(), x.abs()
    r = 0 if inv_freq is None else 2 * len(inv_freq)
    if r:
        t = (pos.double()[:, None] * inv_freq.double())[:, None]
        i = torch.arange(r // 2, device=x.device)
        ia, ib = (2 * i, 2 * i + 1) if inter else (i, i + r // 2)
        a, b = x[..., ia], x[..., ib]
        y[..., ia] = a * t.cos() - b * t.sin()
        y[..., ib] = b * t.cos() + a * t.sin()
        size[..., ia] = size[..., ib] = a.abs() + b.abs()
    return y, size


def check(dbv, q, k, pos, inv_freq, qw=None, kw=None, eps=1e-6, inter=False, dtype=None, **more):
    """Tolerances.  Half a step of the output's type (2^-8 of bf16, 2^-24 of fp32);
    before it, of |x'_a| + |x'_b|: the sum of squares within 24 steps of 2^-24 (half
    of that in the root), the root 2^-22, products and cosines 2^-22, the angle
    2^-32 turns and its rounding to 24 bits 2^-22 -- 2^-19 in all."""
    got = dbv.sv_qk_norm_rope(q, k, pos, inv_freq, q_weight=qw, k_weight=kw, eps=eps,
                              interleaved=inter, dtype=dtype, **more)
    for x, w, n in ((q, qw, "q"), (k, kw, "k")):
        if x is None:
            assert got[n] is None
            continue
        want, size = formula(x, pos, inv_freq, w, eps, inter)
        y = got[n]
        assert y.dtype == (dtype or x.dtype)
        half = torch.finfo(y.dtype).eps / 2
        live = pos >= 0
        bad = ~((y.double() - want).abs() <= half * want.abs() + 2.0 ** -19 * size)[live]
        assert not bad.any(), (n, bad.nonzero()[:4], y[live][bad][:4], want[live][bad][:4])
    return got


def inputs(seed, T, Hq, H, D, rot, dtype=torch.bfloat16, far=5000, spread=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn((T, Hq + 2 * H, D), generator=g, device="cuda") * spread).to(dtype)
    pos = torch.randint(0, far, (T,), generator=g, device="cuda").to(torch.int32)
    f = (10000.0 ** -(torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / max(rot, 1)))
    w = [torch.rand(D, generator=g, device="cuda") + 0.5 for _ in range(2)]
    return x[:, :Hq], x[:, Hq:Hq + H], pos, f.float(), w


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("D,rot", [(64, 64), (128, 128), (256, 256), (512, 512), (96, 96), (80, 80),
                                   (128, 64), (128, 32), (96, 48), (64, 18), (128, 2), (16, 16),
                                   (32, 32), (18, 6), (198, 198), (130, 44), (2, 2), (48, 48),
                                   (510, 256)])
def test_head_sizes(dbv, D, rot, norm, inter):
    q, k, pos, f, w = inputs(D + rot, 37, 6, 2, D, rot)
    w = w if norm else [None, None]
    check(dbv, q, k, pos, f, *w, inter=inter)


@pytest.mark.parametrize("T,Hq,H", [(1, 32, 8), (1, 1, 1), (2, 5, 5), (33, 7, 1), (1088, 32, 8),
                                    (5000, 3, 1), (1, 100, 30)])
@pytest.mark.parametrize("D", [64, 128, 96, 42])
def test_tokens_and_heads(dbv, T, Hq, H, D):
    q, k, pos, f, w = inputs(T + D, T, Hq, H, D, D)
    check(dbv, q, k, pos, f, *w)


@pytest.mark.parametrize("D,rot", [(128, 128), (64, 30)])
@pytest.mark.parametrize("i", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("o", [torch.bfloat16, torch.float32])
def test_types(dbv, i, o, D, rot):
    q, k, pos, f, w = inputs(1, 50, 4, 2, D, rot, dtype=i)
    for inter in (False, True):
        check(dbv, q, k, pos, f, *w, inter=inter, dtype=o)


def test_far_positions(dbv):
    """Angles at positions up to the last of 31 bits, in fp32 where it shows."""
    q, k, pos, f, w = inputs(2, 64, 2, 1, 128, 128, dtype=torch.float32)
    pos = torch.cat([torch.arange(2 ** 31 - 32, 2 ** 31), torch.tensor([0, 1, 2, 3]),
                     2 ** torch.arange(28)]).to(device="cuda", dtype=torch.int32)
    check(dbv, q, k, pos, f)
    # frequencies of every size and sign
    f = torch.tensor([1.0, -1.0, 1.9999, 0.0, 1e-38, 1e-42, 2.0 ** -20, 0.1], device="cuda")
    for inter in (False, True):
        check(dbv, q, k, torch.clamp(pos, max=1 << 22), f, inter=inter)


def test_only_one_weight_or_side(dbv):
    q, k, pos, f, w = inputs(3, 20, 4, 2, 128, 128)
    check(dbv, q, k, pos, f, w[0], None)
    check(dbv, q, k, pos, f, None, w[1])
    check(dbv, q, None, pos, f, w[0], None)
    check(dbv, None, k, pos, f, None, w[1])
    check(dbv, q, k, pos, None, *w)
    got = check(dbv, q, k, pos, None)
    assert torch.equal(got["q"], q) and torch.equal(got["k"], k)


def test_small_and_large_heads(dbv):
    """eps where a head is nothing, and elements far from 1."""
    q, k, pos, f, w = inputs(4, 30, 4, 2, 64, 64)
    q[3] = 0
    k[5, 1] = 0
    q[7] *= 1e-12
    q[8] *= 1e15
    check(dbv, q, k, pos, f, *w)
    check(dbv, q, k, pos, f, *w, eps=0.25)
    got = dbv.sv_qk_norm_rope(q, k, pos, f, q_weight=w[0], k_weight=w[1])
    assert (got["q"][3] == 0).all()


def test_not_finite_stays_in_its_head(dbv):
    for D in (128, 42):
        q, k, pos, f, w = inputs(5, 9, 4, 2, D, D)
        q[2, 1, 3] = float("nan")
        k[4, 0, 1] = float("inf")
        for ws in (w, [None, None]):
            got = dbv.sv_qk_norm_rope(q, k, pos, f, q_weight=ws[0], k_weight=ws[1])
            lost = got["q"].isfinite().all(-1).logical_not().nonzero().tolist()
            assert lost == [[2, 1]]
            lost = got["k"].isfinite().all(-1).logical_not().nonzero().tolist()
            assert lost == [[4, 0]]


@pytest.mark.parametrize("D", [128, 96, 42])
def test_skipped_tokens_and_places(dbv, D):
    """Negative positions are left; outputs in place, in views, heads first.  (Rows
    off 16 bytes go another way, which adds and multiplies in another order: their
    results are within the tolerance, not the same bits.  fp32 sums of D squares in
    two orders differ by up to D 2^-24, and where that moves a result across the
    middle of two bf16 values its rounding differs by a step.)"""
    q, k, pos, f, w = inputs(6, 40, 4, 2, D, D)
    pos[3] = -1
    pos[30:] = -1
    want = dbv.sv_qk_norm_rope(q, k, pos, f, q_weight=w[0], k_weight=w[1])
    out = (torch.full((4, 40, D), 5.0, dtype=torch.bfloat16, device="cuda").transpose(0, 1),
           torch.full((40, 2 * D + 3), 5.0, dtype=torch.bfloat16,
                      device="cuda")[:, 1:1 + 2 * D].unflatten(1, (2, D)))
    check(dbv, q, k, pos, f, *w, out=out)
    live = pos >= 0
    for o in out:
        assert (o[~live] == 5.0).all()
    before = [q.clone(), k.clone()]
    got = dbv.sv_qk_norm_rope(q, k, pos, f, q_weight=w[0], k_weight=w[1], out=(q, k))
    for x, b, n in zip((q, k), before, "qk"):
        assert got[n] is x and torch.equal(x[live], want[n][live])
        assert torch.equal(x[~live], b[~live])


def test_broadcast_inputs(dbv):
    """Strides of zero in the inputs: one token's head for all."""
    q, k, pos, f, w = inputs(7, 12, 4, 2, 128, 128)
    check(dbv, q[:1, :1].expand(12, 4, 128), k[:, :1].expand(12, 2, 128), pos, f, *w)


def test_refusals_of_the_binding(dbv):
    q, k, pos, f, w = inputs(8, 5, 4, 2, 64, 64)
    bad = [dict(k=k.float()), dict(k=k[:4]), dict(pos=pos.long()), dict(pos=pos[:4]),
           dict(inv_freq=f.double()), dict(q_weight=w[0].bfloat16()), dict(k_weight=w[1][:3]),
           dict(dtype=torch.float16), dict(q=q.half(), k=k.half()),
           dict(out=(q[:, :2], None)), dict(q=q.transpose(1, 2))]
    for b in bad:
        a = dict(q=q, k=k, pos=pos, inv_freq=f)
        a.update(b)
        with pytest.raises(ValueError):
            dbv.sv_qk_norm_rope(**a)
    with pytest.raises(dbv.SVError):
        dbv.sv_qk_norm_rope(q, k, pos, torch.ones(40, device="cuda"))
    with pytest.raises(dbv.SVError):  # an output that is the other's input
        dbv.sv_qk_norm_rope(q[:, :2], k, pos, f, out=(k, None))


def test_in_a_graph_and_on_another_stream(dbv):
    q, k, pos, f, w = inputs(9, 300, 8, 2, 128, 128)
    want = dbv.sv_qk_norm_rope(q, k, pos, f, q_weight=w[0], k_weight=w[1])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = dbv.sv_qk_norm_rope(q, k, pos, f, q_weight=w[0], k_weight=w[1])
    g.replay()
    s = torch.cuda.Stream()
    other = dbv.sv_qk_norm_rope(q, k, pos, f, q_weight=w[0], k_weight=w[1], stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(out[n], want[n]) and torch.equal(other[n], want[n]) for n in "qk")


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("D,rot,off", [(128, 32, 0), (128, 20, 0), (96, 48, 1), (64, 0, 0)])
def test_what_is_not_rotated_stays_apart(dbv, D, rot, off, inter):
    """Infinities and NaN: without a norm they reach the other element of their own
    pair, and none that is not rotated but themselves; the rest keeps its bits."""
    T = 6
    whole = torch.randn((T, 2, D + 8), device="cuda").bfloat16()
    x = whole[:, :, off:off + D]
    pos = torch.arange(1, T + 1, device="cuda", dtype=torch.int32)
    f = torch.rand(rot // 2, device="cuda") + 0.1 if rot else None
    clean = dbv.sv_qk_norm_rope(x, None, pos, f, interleaved=inter)["q"]
    for d in range(0, D, 5):
        x[d % T, d % 2, d] = float("inf") if d % 3 else float("nan")
    bad = ~x.isfinite()
    reach = bad.clone()
    i = torch.arange(rot // 2, device="cuda")
    a, b = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
    reach[..., a] |= bad[..., b]
    reach[..., b] |= bad[..., a]
    got = dbv.sv_qk_norm_rope(x, None, pos, f, interleaved=inter)["q"]
    assert torch.equal(~got.isfinite(), reach)
    assert torch.equal(got[~reach], clean[~reach])
    assert torch.equal(got[..., rot:].nan_to_num(7.0), x[..., rot:].nan_to_num(7.0))


@pytest.mark.parametrize("Hq,H,D,rot,inter", [(32, 8, 128, 128, False), (7, 3, 96, 48, True),
                                              (1, 40, 64, 64, False), (5, 2, 256, 32, False)])
@pytest.mark.parametrize("given", [torch.bfloat16, torch.float32])
def test_many_tokens(dbv, Hq, H, D, rot, inter, given):
    """So many that a warp takes all of a token's heads."""
    q, k, pos, f, w = inputs(10, 5000, Hq, H, D, rot, given, far=1 << 20)
    pos[77] = pos[4999] = -1
    check(dbv, q, k, pos, f, *w, inter=inter, dtype=torch.bfloat16)
    check(dbv, q, k, pos, f, w[0], None, inter=inter)
