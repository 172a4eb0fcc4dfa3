"""sv_sample_rows against the definition in fp64 (numpy): tokens and kept
counts are equal wherever no decision of the definition lies within 1e-11 of
its border (weights are decided to 2^-44); probabilities agree within fp32
rounding of a quotient of exact sums."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

BORDER = 1e-11          # relative distance from a border that leaves a decision open
PROB_RTOL = 2.0 ** -22  # one rounding to fp32 and the weights' own error; and
                        # half the least fp32 step, 2^-150


@pytest.fixture(scope="module")
def dbv():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import draft_block_verification_gb300 as m
    return m


def reference(x, u, T, k, p, m):
    """(token, prob, kept, open): open where fp64 itself does not tell."""
    x = np.where(np.isnan(x), -np.inf, x.astype(np.float64))
    top = x.max()
    if top == -np.inf:
        return -1, 0.0, 0, False
    if T == 0:
        return int(np.argmax(x)), 1.0, 1, False
    if top == np.inf:
        x = np.where(x == np.inf, 0.0, -np.inf)
        top = 0.0
    d = (x - top) / T
    w = np.exp(d)
    order = np.argsort(-x, kind="stable")
    finite = int((x > -np.inf).sum())
    n = min(k, finite) if k > 0 else finite
    is_open = False
    run = np.cumsum(w[order[:n]])
    if p < 1:
        goal = p * run[-1]
        n = min(n, int((run < goal).sum()) + 1)
        is_open |= bool((np.abs(run[:-1] - goal) < BORDER * run[-1]).any()) and p > 0
    if m > 0:
        is_open |= bool((np.abs(d - np.log(m)) < 1e-13).any()) and m < 1
        n = min(n, int((d >= np.log(m)).sum()))
    n = max(n, 1)
    ids = np.sort(order[:n])
    run = np.cumsum(w[ids])
    goal = u * run[-1]
    past = np.nonzero(run > goal)[0]
    at = int(past[0]) if len(past) else int(np.nonzero(w[ids] > 0)[0][-1])
    if 0 < u < 1:
        is_open |= bool((np.abs(run[:-1] - goal) < BORDER * run[-1]).any())
    return int(ids[at]), w[ids[at]] / run[-1], n, is_open


def check(dbv, x, u, T=None, k=None, p=None, m=None, most_open=0.02):
    R = x.shape[0]
    host = x.float().cpu().numpy()
    par = []
    for v, off in ((T, 1.0), (k, 0), (p, 1.0), (m, 0.0)):
        par.append(np.full(R, off) if v is None else v.cpu().numpy())
    out = dbv.sv_sample_rows(x, u, temperature=T, top_k=k, top_p=p, min_p=m)
    torch.cuda.synchronize()
    token, prob, kept = (out[n].cpu().numpy() for n in ("token", "prob", "kept"))
    uh = u.cpu().numpy().astype(np.float64)
    opened = 0
    for r in range(R):
        rt, rp, rk, is_open = reference(host[r], uh[r], float(par[0][r]), int(par[1][r]),
                                        float(par[2][r]), float(par[3][r]))
        if is_open:
            opened += 1
            continue
        what = (r, uh[r], [float(a[r]) for a in par])
        assert kept[r] == rk, (what, kept[r], rk)
        assert token[r] == rt, (what, token[r], rt)
        assert abs(prob[r] - rp) <= PROB_RTOL * rp + 2.0 ** -150, (what, prob[r], rp)
    assert opened <= max(1, most_open * R)
    dbv.default_handle(x.device).sync_status()


def rows(R, V, dtype, spread, seed, lift=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((R, V), generator=g, device="cuda") * spread
    if lift:
        top = torch.randint(0, V, (R, min(V, 12)), generator=g, device="cuda")
        x.scatter_add_(1, top, torch.rand(top.shape, generator=g, device="cuda") * 10)
    return x.to(dtype), torch.rand(R, generator=g, device="cuda")


def full(R, v, dtype=torch.float32):
    return torch.full((R,), v, dtype=dtype, device="cuda")


def mixed(R, seed):
    g = np.random.RandomState(seed)
    f = lambda v, t: torch.tensor(g.choice(v, R), dtype=t, device="cuda")  # noqa: E731
    return dict(T=f([0.0, 0.5, 0.7, 1.0, 1.3, 4.0], torch.float32),
                k=f([0, 0, 1, 2, 40, 1000, 5000, 1 << 30], torch.int32),
                p=f([1.0, 0.0, 0.3, 0.8, 0.95, 0.999], torch.float32),
                m=f([0.0, 0.0, 0.02, 0.3, 1.0], torch.float32))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [1, 2, 7, 8, 257, 1000, 4096, 4097, 4104, 32003, 50257])
def test_mixed_filters(dbv, V, dtype):
    R = 48
    x, u = rows(R, V, dtype, 2.0, V)
    check(dbv, x, u, **mixed(R, V))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("spread", [0.05, 1.0, 2.0, 6.0])
def test_wide_rows(dbv, spread, dtype):
    """Kept sets from one token to most of a row of 128,256."""
    R = 24
    x, u = rows(R, 128256, dtype, spread, 5, lift=spread > 1)
    check(dbv, x, u, **mixed(R, 77))
    check(dbv, x, u, p=full(R, 0.9))
    check(dbv, x, u)


def test_largest_vocabulary(dbv):
    x, u = rows(2, 1 << 20, torch.bfloat16, 1.0, 9)
    check(dbv, x, u, p=full(2, 0.95))
    with pytest.raises(dbv.SVError) as e:
        dbv.sv_sample_rows(torch.zeros((1, (1 << 20) + 8), device="cuda"), u[:1])
    assert e.value.status == dbv.SV_ERR_UNSUPPORTED


@pytest.mark.parametrize("V", [100, 9000, 40000])
@pytest.mark.parametrize("levels", [1, 2, 5])
def test_ties(dbv, V, levels):
    """Few distinct logits: the boundary cuts through equals by id, also where
    more of them are equal than the list holds."""
    R = 40
    g = torch.Generator(device="cuda").manual_seed(levels)
    x = torch.randint(0, levels, (R, V), generator=g, device="cuda").float()
    u = torch.rand(R, generator=g, device="cuda")
    k = torch.randint(1, V, (R,), generator=g, device="cuda", dtype=torch.int32)
    check(dbv, x, u, k=k, most_open=1.0)
    check(dbv, x, u, k=k, p=full(R, 0.617), most_open=1.0)
    check(dbv, x, u, p=full(R, 0.531), most_open=1.0)
    check(dbv, x, u, m=full(R, 0.5))


def test_unaligned_rows(dbv):
    R, V = 9, 5001
    for dtype in (torch.bfloat16, torch.float32):
        base, u = rows(R, V + 6, dtype, 2.0, 3)
        check(dbv, base[:, 3:3 + V], u, **mixed(R, 4))
        wide, u = rows(2 * R, V + 7, dtype, 2.0, 4)  # 5008 a row: whole vectors
        check(dbv, wide[::2, :V], u[:R].contiguous(), **mixed(R, 5))


def test_masked_and_special_logits(dbv):
    for V in (33, 5000):
        for dtype in (torch.bfloat16, torch.float32):
            x, u = rows(12, V, dtype, 1.0, V)
            low = torch.finfo(dtype).min
            x[0] = -float("inf")
            x[1, :] = low
            x[2, 1:] = -float("inf")
            x[3, 3:] = low
            x[4, 5] = float("inf")
            x[5, 2:9] = float("inf")
            x[6, ::3] = float("nan")
            x[7] = float("nan")
            x[8, :-1] = -float("inf")
            x[9] = torch.finfo(dtype).max
            x[10, ::2] = -float("inf")
            x[11, 1::2] = -0.0
            x[11, ::2] = 0.0
            for kw in (dict(), dict(k=full(12, 4, torch.int32)), dict(p=full(12, 0.7)),
                       dict(m=full(12, 0.25)), dict(T=full(12, 0.0)),
                       dict(k=full(12, 9, torch.int32), p=full(12, 0.6), m=full(12, 0.1))):
                check(dbv, x, u, most_open=1.0, **kw)


def test_ends_of_u_and_temperature(dbv):
    x, _ = rows(8, 6000, torch.float32, 2.0, 1)
    for u in (0.0, 1.0, 1e-30, 1.0 - 2.0 ** -24):
        for T in (2.0 ** -20, 0.01, 100.0):
            check(dbv, x, full(8, u), T=full(8, T), p=full(8, 0.9), most_open=1.0)
            check(dbv, x, full(8, u), T=full(8, T), most_open=1.0)


def test_bad_parameters_are_latched(dbv):
    x, u = rows(4, 100, torch.float32, 1.0, 1)
    h = dbv.default_handle(x.device)
    nan = float("nan")
    for kw in (dict(temperature=[1, -1, 1, 1]), dict(temperature=[1, nan, 1, 1]),
               dict(temperature=[1, 1e-8, 1, 1]), dict(top_p=[1, -0.1, 1, 1]),
               dict(top_p=[1, nan, 1, 1]), dict(min_p=[0, 1.5, 0, 0]), dict(top_k=[0, -3, 0, 0])):
        name, v = next(iter(kw.items()))
        t = torch.tensor(v, dtype=torch.int32 if name == "top_k" else torch.float32,
                         device="cuda")
        out = dbv.sv_sample_rows(x, u, **{name: t})
        assert out["token"].tolist()[1] == -1 and out["kept"].tolist()[1] == 0
        assert all(v >= 0 for v in out["token"].tolist()[2:])
        with pytest.raises(dbv.SVError) as e:
            h.sync_status()
        assert e.value.status == dbv.SV_ERR_DEVICE_BOUNDS
    h.sync_status()


def test_refusals_and_empty(dbv):
    x, u = rows(4, 100, torch.float32, 1.0, 1)
    for bad in (lambda: dbv.sv_sample_rows(x.half(), u), lambda: dbv.sv_sample_rows(x, u[:3]),
                lambda: dbv.sv_sample_rows(x, u.double()), lambda: dbv.sv_sample_rows(x[0], u),
                lambda: dbv.sv_sample_rows(x.t(), u),
                lambda: dbv.sv_sample_rows(x, u, top_k=u)):
        with pytest.raises(ValueError):
            bad()
    out = dbv.sv_sample_rows(x[:0], u[:0])
    assert out["token"].numel() == 0


def test_another_stream_and_a_graph(dbv):
    x, u = rows(6, 40000, torch.bfloat16, 2.0, 2)
    p = full(6, 0.9)
    want = dbv.sv_sample_rows(x, u, top_p=p)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = dbv.sv_sample_rows(x, u, top_p=p)
    torch.cuda.synchronize()
    assert all(torch.equal(want[n], got[n]) for n in want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        again = dbv.sv_sample_rows(x, u, top_p=p)
    u2 = torch.rand_like(u)
    want = dbv.sv_sample_rows(x, u2, top_p=p)
    u.copy_(u2)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(want[n], again[n]) for n in want)
