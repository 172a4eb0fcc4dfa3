"""The paged 8-bit cache on the GPU: plan, append and attention against the
plain numpy forms of kv_util."""
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


# --------------------------------------------------------------------------
# Plan
# --------------------------------------------------------------------------
class Pool:
    """The plain form: a queue of pages and the sequences' tables."""

    def __init__(self, B, cols, ring, block, seed):
        r = np.random.RandomState(seed)
        self.block, self.ring = block, ring
        self.ids = r.permutation(ring).astype(np.int32)
        self.head, self.tail = 0, ring
        first = int(r.randint(ring))
        self.ids = np.roll(self.ids, first)
        self.head += first
        self.tail += first
        self.table = np.full((B, cols), -1, np.int32)
        self.held = np.zeros(B, np.int32)

    def step(self, cached, new, cap):
        want = -(-(cached + new) // self.block)
        if np.maximum(want - self.held, 0).sum() > self.tail - self.head:
            return None
        ids, head, tail = self.ids.copy(), self.head, self.tail
        slot, pos = [], []
        for b, (c, n, w) in enumerate(zip(cached, new, want)):
            for j in range(self.held[b], w):
                self.table[b, j] = ids[head % self.ring]
                head += 1
            for j in range(w, self.held[b]):
                self.ids[tail % self.ring] = self.table[b, j]
                tail += 1
            p = np.arange(c, c + n)
            slot.append(self.table[b, p // self.block] * self.block + p % self.block)
            pos.append(p)
        self.head, self.tail, self.held = head, tail, want.astype(np.int32)
        pad = np.full(cap - new.sum(), -1)
        return dict(kv_len=cached + new, cu_new=np.append(0, np.cumsum(new)), held=want,
                    free_pos=[head, tail], slot=np.concatenate(slot + [pad]),
                    pos=np.concatenate(pos + [pad]))


@pytest.mark.parametrize("B,block", [(1, 16), (2, 128), (31, 16), (64, 64), (1000, 32),
                                     (1024, 16), (1025, 16), (5000, 16)])
def test_plan_over_many_steps(dbv, B, block):
    """Sequences grow, lose rejected drafts, end and start again: the state
    stays equal to the plain form's, and no page is ever held twice."""
    r = np.random.RandomState(B)
    cols, ring, cap = 12, 9 * B + 3, 40 * B + 5
    pool = Pool(B, cols, ring, block, B)
    table, ids = dev(pool.table), dev(pool.ids)
    held, free_pos = dev(pool.held), dev([pool.head, pool.tail], torch.int64)
    cached = np.zeros(B, np.int64)
    for step in range(8):
        new = r.randint(0, 40, B)
        cached[r.rand(B) < 0.1] = 0
        new = np.where(r.rand(B) < 0.1, 0, new)
        new = np.minimum(new, cols * block - cached)
        before = (pool.head, pool.tail)
        want = pool.step(cached, new, cap)
        assert want is not None
        out = dbv.sv_kv_plan(dev(cached), dev(new), held, table, ids, free_pos, block, cap)
        for n in want:
            assert np.array_equal(out[n].cpu().numpy(), np.asarray(want[n])), (n, step, before)
        got = table.cpu().numpy()
        live = np.arange(cols) < pool.held[:, None]
        assert np.array_equal(got[live], pool.table[live])
        assert np.array_equal(ids.cpu().numpy(), pool.ids)
        pages = got[live]
        queue = pool.ids[np.arange(pool.head, pool.tail) % ring]
        assert len(set(pages)) == len(pages)
        assert not set(pages) & set(queue) and len(pages) + len(queue) == ring
        held, free_pos = out["held"], out["free_pos"]
        cached = np.maximum(cached + new - r.randint(0, 20, B), 0)
    dbv.default_handle(table.device).sync_status()


def test_plan_again_gives_the_same(dbv):
    pool = Pool(6, 8, 40, 16, 3)
    table, ids = dev(pool.table), dev(pool.ids)
    held, fp = dev(pool.held), dev([pool.head, pool.tail], torch.int64)
    c, n = dev([0] * 6), dev([1, 17, 0, 64, 33, 5])
    first = dbv.sv_kv_plan(c, n, held, table, ids, fp, 16, 130)
    kept = table.clone()
    again = dbv.sv_kv_plan(c, n, held, table, ids, fp, 16, 130)
    assert all(torch.equal(first[k], again[k]) for k in first) and torch.equal(kept, table)


@pytest.mark.parametrize("kind,status", [
    ("pages", 3), ("tokens", 6), ("negative", 6), ("cols", 6), ("held", 6), ("queue", 6)])
def test_plan_that_cannot_be_served_changes_nothing(dbv, kind, status):
    pool = Pool(4, 4, 9, 16, 1)
    table, ids = dev(pool.table), dev(pool.ids)
    cached, new, held = [0, 0, 0, 0], [16, 32, 5, 0], [0, 0, 0, 0]
    head, tail, cap = pool.head, pool.tail, 64
    if kind == "pages":
        tail = head + 3
    elif kind == "tokens":
        cap = 52
    elif kind == "negative":
        new[2] = -1
    elif kind == "cols":
        new[1] = 65
        cap = 200
    elif kind == "held":
        held[3] = 5
    else:
        tail = head + 10
    fp = dev([head, tail], torch.int64)
    kept = table.clone(), ids.clone()
    out = dbv.sv_kv_plan(dev(cached), dev(new), dev(held), table, ids, fp, 16, cap)
    with pytest.raises(dbv.SVError) as e:
        dbv.default_handle(table.device).sync_status()
    assert e.value.status == status
    assert torch.equal(table, kept[0]) and torch.equal(ids, kept[1])
    assert out["kv_len"].tolist() == cached and out["held"].tolist() == held
    assert out["cu_new"].tolist() == [0] * 5 and out["free_pos"].tolist() == [head, tail]
    assert set(out["slot"].tolist()) == {-1} and set(out["pos"].tolist()) == {-1}


def test_plan_of_nothing(dbv):
    e = dev([])
    out = dbv.sv_kv_plan(e, e, e, dev(np.zeros((0, 3))), dev([4, 5]), dev([0, 2], torch.int64),
                         16, 3)
    assert out["cu_new"].tolist() == [0] and out["slot"].tolist() == [-1] * 3
    assert out["free_pos"].tolist() == [0, 2]


# --------------------------------------------------------------------------
# Append
# --------------------------------------------------------------------------
def make_slots(r, lens, new, block, pages):
    """A shuffled table and the slots of `new` tokens after `lens` tokens."""
    want = [-(-(c + n) // block) for c, n in zip(lens, new)]
    order = r.permutation(pages)[:sum(want)]
    table, at, slot = np.full((len(lens), max(max(want), 1)), -1, np.int32), 0, []
    for b, w in enumerate(want):
        table[b, :w] = order[at:at + w]
        at += w
        p = np.arange(lens[b], lens[b] + new[b])
        slot.append(table[b, p // block] * block + p % block)
    return table, np.concatenate(slot).astype(np.int32)


def check_append(dbv, x, slot, codes, scale, block):
    """x: two [T, H, D] torch tensors; codes, scale: numpy pairs."""
    c = [dev(a, torch.uint8) for a in codes]
    s = [dev(a, torch.float32) for a in scale]
    for _ in range(2):  # the second time changes nothing
        dbv.sv_kv_append(x[0], x[1], dev(slot), c[0].view(torch.float8_e4m3fn),
                         c[1].view(torch.float8_e4m3fn), s[0], s[1])
        for i in range(2):
            want, ws = kv_util.append(x[i].float().cpu().numpy(), slot, codes[i], scale[i], block)
            assert np.array_equal(s[i].cpu().numpy(), ws.astype(np.float32))
            got = c[i].cpu().numpy()
            assert np.array_equal(got, want), np.argwhere(got != want)[:5]


def random_cache(r, pages, H, block, D):
    codes = [r.randint(0, 255, (pages, H, block, D)).astype(np.uint8) for _ in range(2)]
    for c in codes:
        c[(c & 127) == 127] = 3
    scale = [2.0 ** r.randint(-9, -2, (pages, H)).astype(np.float64) for _ in range(2)]
    return codes, scale


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D,block,H", [(128, 64, 8), (64, 16, 1), (128, 16, 3), (64, 128, 2),
                                       (128, 128, 2), (64, 32, 5)])
def test_append(dbv, D, block, H, dtype):
    r = np.random.RandomState(D + block)
    lens = [0, 1, block - 1, block, 3 * block + 5, 7, 2 * block - 2]
    new = [1, 2 * block + 3, 2, block, 17, 0, 1]
    table, slot = make_slots(r, lens, new, block, 40)
    codes, scale = random_cache(r, 40, H, block, D)
    x = [torch.as_tensor(r.randn(len(slot), H, D) * np.exp(r.randn(len(slot), 1, 1) * 2),
                         dtype=dtype, device="cuda") for _ in range(2)]
    check_append(dbv, x, slot, codes, scale, block)
    dbv.default_handle(x[0].device).sync_status()


def test_append_many_tokens(dbv):
    """Windows of 32 tokens: long runs, and a run's start anywhere in a window."""
    r = np.random.RandomState(5)
    lens, new = r.randint(0, 70, 40), r.randint(0, 150, 40)
    table, slot = make_slots(r, lens, new, 32, 400)
    codes, scale = random_cache(r, 400, 4, 32, 64)
    x = [torch.as_tensor(r.randn(len(slot), 4, 64), dtype=torch.bfloat16, device="cuda")
         for _ in range(2)]
    check_append(dbv, x, slot, codes, scale, 32)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_append_strides_padding_and_order(dbv, dtype):
    """Views into a fused projection, an odd offset, skipped tokens, one run
    alone, runs in falling order of their pages."""
    r = np.random.RandomState(8)
    H, D, block = 3, 64, 16
    slot = np.array([-1, 37, 38, -1, -5, 5, 0 + 16 * 9, 1 + 16 * 9, -1, 16 * 4 + 15, 16 * 3],
                    np.int32)
    for off, row in ((0, 2 * H * D + 8), (1, 2 * H * D + 3)):
        whole = torch.as_tensor(r.randn(len(slot), row + off), dtype=dtype, device="cuda")
        k = whole[:, off:off + H * D].unflatten(1, (H, D))
        v = whole[:, off + H * D:off + 2 * H * D].unflatten(1, (H, D))
        codes, scale = random_cache(r, 12, H, block, D)
        check_append(dbv, [k, v], slot, codes, scale, block)
    t = torch.as_tensor(r.randn(H, len(slot), D), dtype=dtype, device="cuda").transpose(0, 1)
    check_append(dbv, [t, t], slot, codes, scale, block)


def test_append_special_values(dbv):
    """Zeros, the borders of the scale, saturation, NaN and infinities, and
    values so small or large that the scale's ends are met."""
    H, D, block = 1, 64, 16
    x = np.zeros((9, H, D), np.float32)
    x[1, 0, 3] = 448.0
    x[2, 0, 3] = np.nextafter(np.float32(448.0), np.float32(1e9))
    x[3, 0, :] = np.linspace(-3e38, 3e38, D)
    x[4, 0, :] = 1e-40
    x[5, 0, 7] = np.nan
    x[5, 0, 8] = 5.0
    x[6, 0, 7] = np.inf
    x[6, 0, 8] = -np.inf
    x[7, 0, :] = np.nan
    x[8, 0, 0] = 2.0 ** -50
    slot = (np.arange(9) * block).astype(np.int32)
    codes, scale = random_cache(np.random.RandomState(1), 10, H, block, D)
    t = torch.as_tensor(x, device="cuda")
    check_append(dbv, [t, t], slot, codes, scale, block)


def test_append_slot_beyond_the_cache_is_latched(dbv):
    H, D, block, pages = 2, 64, 16, 3
    r = np.random.RandomState(2)
    codes, scale = random_cache(r, pages, H, block, D)
    x = torch.as_tensor(r.randn(2, H, D), dtype=torch.float32, device="cuda")
    c = [dev(a, torch.uint8) for a in codes]
    s = [dev(a, torch.float32) for a in scale]
    dbv.sv_kv_append(x, x, dev([pages * block, 4]), c[0], c[1], s[0], s[1])
    with pytest.raises(dbv.SVError) as e:
        dbv.default_handle(x.device).sync_status()
    assert e.value.status == dbv.SV_ERR_DEVICE_BOUNDS
    want, _ = kv_util.append(x.cpu().numpy(), np.array([-1, 4]), codes[0], scale[0], block)
    assert np.array_equal(c[0].cpu().numpy(), want)


# --------------------------------------------------------------------------
# Attention
# --------------------------------------------------------------------------
def attend_case(r, lens, new, H, G, D, block, tree=False, pow2=False, spread=1.0):
    """lens: tokens before the new ones.  Every byte that no token may see is
    NaN, in live pages and in others."""
    pages = sum(-(-(c + n) // block) for c, n in zip(lens, new)) + 2
    table, slot = make_slots(r, lens, new, block, pages)
    kv = np.array(lens) + np.array(new)
    codes = [kv_util.e4m3_encode(r.randn(pages, H, block, D) * 60) for _ in range(2)]
    scale = [(2.0 ** r.randint(-8, -3, (pages, H)) if pow2 else
              np.exp(r.uniform(-5, -3, (pages, H)))).astype(np.float32) for _ in range(2)]
    live = np.zeros((pages, block), bool)
    for b, L in enumerate(kv):
        p = np.arange(L)
        live[table[b, p // block], p % block] = True
    for c in codes:
        c[~np.broadcast_to(live[:, None], (pages, H, block))] = 0x7F
    T = int(np.sum(new))
    q = torch.as_tensor(r.randn(T, H * G, D) * spread, dtype=torch.bfloat16, device="cuda")
    cu = np.append(0, np.cumsum(new)).astype(np.int32)
    mask = None
    if tree:
        words = max(1, -(-max(new) // 32))
        mask = np.zeros((T, words), np.uint32)
        for b, n in enumerate(new):
            for i in range(n):
                t = cu[b] + i
                if i and r.rand() < 0.9:
                    mask[t] = mask[cu[b] + r.randint(i)]
                if r.rand() < 0.95:
                    mask[t, i // 32] |= np.uint32(1 << (i % 32))
    return dict(q=q, codes=codes, scale=scale, table=table, kv=kv, cu=cu, mask=mask, block=block)


def run_attend(dbv, c, **kw):
    m = None if c["mask"] is None else dev(c["mask"].view(np.int32))
    k, v = (dev(a, torch.uint8).view(torch.float8_e4m3fn) for a in c["codes"])
    ks, vs = (dev(a, torch.float32) for a in c["scale"])
    return dbv.sv_kv_attention(c["q"], k, v, ks, vs, dev(c["table"]), dev(c["kv"]),
                               dev(c["cu"]), mask=m, want_lse=True, **kw)


def check_attend(c, out, softmax_scale=None):
    """Tolerances.  An output is rounded to bf16 (2^-8 of its size); a weight is
    held to 8 bits or more (2^-8 of sum w|v| / sum w) down to 2^-24 of the
    largest; a score is a sum of up to 256 exact products in fp32 (2^-16 of
    sum |q||k| at worst), its exponential within 2^-20 of a score's size."""
    want, lse, mag, size = kv_util.attend(
        c["q"].float().cpu().numpy().astype(np.float64), c["codes"], c["scale"], c["table"],
        c["kv"], c["cu"], c["block"], c["mask"], softmax_scale)
    got = out["out"].float().cpu().numpy()
    L = c["kv"].max()
    top = 448.0 * max(s.max() for s in c["scale"])
    tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + 2.0 ** -15 * size[..., None]) * mag + \
        L * 2.0 ** -24 * top * (mag > 0)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], want[bad][:4], tol[bad][:4])
    gl = out["lse"].cpu().numpy()
    assert np.array_equal(np.isinf(gl), np.isinf(lse))
    ok = np.isfinite(lse)
    assert (np.abs(gl[ok] - lse[ok]) <= 2.0 ** -16 * size[ok] + 2.0 ** -19 * (
        1 + np.abs(lse[ok]))).all()


CASES = [
    # lens, new, H, G, D, block
    ([0], [1], 1, 1, 128, 16),
    ([0], [1], 2, 4, 64, 64),
    ([1], [1], 8, 4, 128, 64),
    ([127], [1], 1, 8, 128, 64),
    ([128], [1], 1, 8, 128, 128),
    ([126, 0, 300], [2, 5, 17], 2, 4, 128, 64),
    ([0, 63, 64, 65], [64, 1, 9, 33], 1, 3, 64, 16),
    ([500, 20, 1000, 3], [17, 17, 1, 8], 2, 4, 128, 32),
    ([200, 90], [7, 70], 1, 7, 128, 128),
    ([40, 700], [3, 20], 1, 16, 64, 32),
    ([333] * 5, [1, 0, 2, 0, 13], 3, 12, 128, 16),
    ([2600, 10], [5, 3], 2, 6, 64, 128),
    ([3000], [17], 1, 4, 128, 64),
]


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_attention(dbv, case, tree):
    lens, new, H, G, D, block = CASES[case]
    r = np.random.RandomState(case)
    c = attend_case(r, lens, new, H, G, D, block, tree=tree, spread=[0.3, 1.0, 4.0][case % 3])
    out = run_attend(dbv, c)
    check_attend(c, out)
    again = run_attend(dbv, c)  # bit for bit, whatever the order of the work
    assert torch.equal(out["out"], again["out"]) and torch.equal(out["lse"], again["lse"])
    dbv.default_handle(c["q"].device).sync_status()


def test_attention_one_page_dominates(dbv):
    """Scales that differ by 2^30 between pages, values and keys alike, and a
    page whose values are all zero at the least scale."""
    r = np.random.RandomState(3)
    c = attend_case(r, [300, 70], [4, 2], 2, 2, 128, 32, pow2=True)
    c["scale"][1][:] = (2.0 ** r.randint(-30, 0, c["scale"][1].shape)).astype(np.float32)
    first = c["table"][0, 0]
    c["codes"][1][first] = 0
    c["scale"][1][first] = 2.0 ** -40
    c["scale"][0][first] *= 8
    out = run_attend(dbv, c)
    want, lse, mag, size = kv_util.attend(
        c["q"].float().cpu().numpy().astype(np.float64), c["codes"], c["scale"], c["table"],
        c["kv"], c["cu"], 32)
    got = out["out"].float().cpu().numpy()
    # the weights' last step is relative to the largest weighted value, not to the sum
    tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + 2.0 ** -15 * size[..., None]) * mag
    top = mag.max(-1, keepdims=True)
    assert (np.abs(got - want) <= tol + 2.0 ** -12 * top).all()


def test_attention_rows_that_see_nothing(dbv):
    r = np.random.RandomState(4)
    c = attend_case(r, [0, 50], [5, 3], 2, 3, 64, 16, tree=True)
    c["mask"][:] = 0
    out = run_attend(dbv, c)
    check_attend(c, out)
    assert (out["out"][:5] == 0).all() and torch.isinf(out["lse"][:5]).all()


def test_attention_sharp_and_shifted_scores(dbv):
    """Scores of some hundreds, rising along the sequence (the running maximum
    moves in every tile) or falling, and a scale of 0 or below."""
    r = np.random.RandomState(6)
    for rising in (True, False):
        c = attend_case(r, [900], [6], 1, 4, 128, 64, spread=0.2)
        for b, L in enumerate(c["kv"]):
            for p in range(L):
                f = p / L if rising else 1 - p / L
                code = kv_util.e4m3_encode(np.full(128, 300.0 * f))
                c["codes"][0][c["table"][b, p // 64], :, p % 64] = code
        c["q"].abs_()
        check_attend(c, run_attend(dbv, c, scale=0.5), 0.5)
        check_attend(c, run_attend(dbv, c, scale=0.0), 0.0)
        check_attend(c, run_attend(dbv, c, scale=-0.25), -0.25)


def test_attention_strided_queries(dbv):
    r = np.random.RandomState(7)
    c = attend_case(r, [100, 9], [3, 11], 2, 4, 128, 64)
    T, Hq, D = c["q"].shape
    for off in (0, 1):
        wide = torch.zeros((T, 2, Hq, D + 8), dtype=torch.bfloat16, device="cuda")
        q = wide[:, 1, :, off:off + D]
        q.copy_(c["q"])
        a = run_attend(dbv, dict(c, q=q))
        b = run_attend(dbv, c)
        assert torch.equal(a["out"], b["out"])


def test_attention_offsets_beyond_32_bits(dbv):
    """Pages that lie past 4 GB in caches of 4.6 GB each."""
    r = np.random.RandomState(8)
    small = attend_case(r, [150, 70], [4, 2], 8, 2, 128, 64)
    want = run_attend(dbv, small)
    pages = 70000
    n = small["codes"][0].shape[0]
    big = [torch.empty((pages, 8, 64, 128), dtype=torch.uint8, device="cuda") for _ in range(2)]
    scale = [torch.ones((pages, 8), device="cuda") for _ in range(2)]
    for i in range(2):
        big[i][pages - n:] = dev(small["codes"][i], torch.uint8)
        scale[i][pages - n:] = dev(small["scale"][i], torch.float32)
    table = np.where(small["table"] >= 0, small["table"] + pages - n, -1)
    got = dbv.sv_kv_attention(small["q"], big[0], big[1], scale[0], scale[1], dev(table),
                              dev(small["kv"]), dev(small["cu"]), want_lse=True)
    assert torch.equal(want["out"], got["out"]) and torch.equal(want["lse"], got["lse"])
    # and the append writes there
    x = torch.randn((3, 8, 128), device="cuda")
    slot = dev([(pages - 1) * 64 + 60 + i for i in range(3)])
    dbv.sv_kv_append(x, x, slot, big[0], big[1], scale[0], scale[1])
    w, _ = kv_util.append(x.cpu().numpy(), np.array([60, 61, 62]),
                          small["codes"][0][-1:], small["scale"][0][-1:], 64)
    assert np.array_equal(big[0][-1].cpu().numpy(), w[0])


def test_attention_bad_pages_and_lengths_are_latched(dbv):
    r = np.random.RandomState(9)
    h = dbv.default_handle(torch.device("cuda", 0))
    c = attend_case(r, [100, 40], [3, 2], 2, 2, 64, 16)
    good = run_attend(dbv, c)
    for kind in ("page", "negative", "length", "short"):
        d = dict(c, table=c["table"].copy(), kv=c["kv"].copy())
        if kind == "page":
            d["table"][0, 2] = c["codes"][0].shape[0]
        elif kind == "negative":
            d["table"][0, 2] = -7
        elif kind == "length":
            d["kv"][0] = c["table"].shape[1] * 16 + 1
        else:
            d["kv"][0] = 2  # fewer tokens than new ones
        out = run_attend(dbv, d)
        with pytest.raises(dbv.SVError) as e:
            h.sync_status()
        assert e.value.status == dbv.SV_ERR_DEVICE_BOUNDS
        assert torch.equal(out["out"][3:], good["out"][3:])  # the other sequence
    h.sync_status()


def test_attention_padding_rows_another_stream_and_a_graph(dbv):
    """T larger than the new tokens (a fixed shape under a graph), lengths that
    change between replays, and a call on another stream."""
    r = np.random.RandomState(10)
    c = attend_case(r, [700, 30, 200], [5, 2, 9], 2, 4, 128, 32)
    q = torch.cat([c["q"], torch.full((4, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")])
    want = run_attend(dbv, c)["out"]
    got = run_attend(dbv, dict(c, q=q))["out"]
    assert torch.equal(got[:16], want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = run_attend(dbv, c)["out"]
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    k, v = (dev(a, torch.uint8) for a in c["codes"])
    ks, vs = (dev(a, torch.float32) for a in c["scale"])
    table, kv, cu = dev(c["table"]), dev(c["kv"]), dev(c["cu"])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = dbv.sv_kv_attention(q, k, v, ks, vs, table, kv, cu)["out"]
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[:16], want)
    kv2 = kv - dev([100, 0, 150])  # an earlier step of the same sequences
    want = dbv.sv_kv_attention(q, k, v, ks, vs, table, kv2, cu)["out"].clone()
    kv.copy_(kv2)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[:16], want[:16])


def test_refusals(dbv):
    r = np.random.RandomState(11)
    c = attend_case(r, [20], [2], 1, 2, 64, 16)
    for kw in (dict(q=c["q"].float()), dict(q=c["q"][0]), dict(q=c["q"].transpose(1, 2)),
               dict(q=c["q"][..., :32]), dict(table=c["table"][0]),
               dict(cu=np.array([0, 1, 2])), dict(mask=np.zeros((1, 1), np.uint32))):
        with pytest.raises((ValueError, dbv.SVError)):
            run_attend(dbv, dict(c, **kw))
