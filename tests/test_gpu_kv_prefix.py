"""Attention over a shared prefix: every row against its value in 64 bits, at
row counts, page sizes and lengths where units, tiles and spans end."""
import numpy as np
import pytest
import torch

import prefix_util as pu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dbv():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import draft_block_verification_gb300 as m
    return m


def ok(dbv):
    dbv.default_handle(torch.device("cuda", 0)).sync_status()


def with_wide(prefix, sizes, after, new, wide):
    """Few rows behind a short prefix are read for each sequence by itself.  wide:
    one more sequence, of its own group, whose rows are too many for that; then
    what is shared is read once, however short."""
    more = ([0], [1], [70], [9]) if wide else ([],) * 4
    return [x + y for x, y in zip((prefix, sizes, after, new), more)]


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("block", [16, 32, 64, 128])
@pytest.mark.parametrize("P", [0, 15, 16, 128, 130, 257, 1000])
def test_lengths_and_pages(dbv, P, block, D, wide):
    c = pu.make(P + block, *with_wide([P], [3], [5, 0, 40], [1, 1, 1], wide), 2, 4, D, block)
    pu.check(c, pu.run(dbv, c))
    ok(dbv)


@pytest.mark.parametrize("new,G", [([1, 1], 1), ([2, 3], 3), ([17, 16, 15], 4), ([31, 1, 32], 2),
                                   ([32] * 4, 1), ([43, 43, 43], 1), ([64, 64], 2),
                                   ([85, 86, 86], 1), ([50, 3, 77], 4), ([70] * 3, 7)])
def test_rows_of_a_unit(dbv, new, G):
    """Up to and past 128 and 256 query rows a head, one and several units."""
    n = len(new)
    c = pu.make(n + G, [700], [n], [9] * n, new, 2, G, 128, 32)
    pu.check(c, pu.run(dbv, c))
    ok(dbv)


@pytest.mark.parametrize("H,G,D,prefix,new", [
    (1, 8, 128, 20000, [1] * 4), (8, 4, 128, 3000, [5] * 8), (3, 2, 64, 9000, [40, 60, 70]),
    (2, 12, 64, 5000, [9] * 9), (1, 1, 128, 40000, [1, 1])])
def test_spans(dbv, H, G, D, prefix, new):
    """Units cut by many CTAs, CTAs with many units, spans that end in a tile."""
    n = len(new)
    c = pu.make(H + G, [prefix], [n], [300] * n, new, H, G, D, 64)
    pu.check(c, pu.run(dbv, c))
    ok(dbv)


@pytest.mark.parametrize("tree", [False, True])
def test_groups(dbv, tree):
    """Groups of unequal prefixes, one of a single sequence, sequences without new
    tokens, and one whose first sequence has none."""
    prefix, sizes = [300, 64, 1025, 40, 500], [3, 2, 1, 4, 3]
    new = [3, 0, 5, 7, 1, 9, 33, 2, 0, 4, 0, 6, 8]
    after = [0, 9, 70, 3, 3, 100, 0, 1, 2, 500, 20, 30, 40]
    c = pu.make(5, prefix, sizes, after, new, 2, 3, 128, 16, tree=tree, pow2=False)
    pu.check(c, pu.run(dbv, c))
    # sequences that are in no group
    part = np.array([3, 5, 9], np.int32)
    pu.check(c, pu.run(dbv, c, prefix_len=None, cu_group=pu.dev(part)))
    # a group without sequences
    part = np.array([0, 3, 3, 5, 6, 13], np.int32)
    pu.check(c, pu.run(dbv, c, prefix_len=None, cu_group=pu.dev(part)))
    ok(dbv)


def test_bounds_only_say_where_to_look(dbv):
    """Bounds below, at and above what is shared, none, and tables that part early."""
    c = pu.make(6, [400], [4], [80, 90, 7, 300], [2, 9, 1, 3], 2, 4, 64, 32)
    for p in (0, 31, 32, 100, 399, 416, 10 ** 9, -5):
        pu.check(c, pu.run(dbv, c, prefix_len=pu.dev([p])))
    pu.check(c, pu.run(dbv, c, prefix_len=None, cu_group=None))
    # a sequence whose third page is a copy of its own
    used = set(c["table"].reshape(-1).tolist())
    spare = next(i for i in range(len(c["codes"][0])) if i not in used)
    for a in c["codes"]:
        a[spare] = a[c["table"][2, 2]]
    for s in c["scale"]:
        s[spare] = s[c["table"][2, 2]]
    c["table"][2, 2] = spare
    pu.check(c, pu.run(dbv, c, prefix_len=None, cu_group=None))
    # new tokens inside the pages that are alike are not shared
    d = pu.make(7, [256], [2], [0, 0], [1, 1], 1, 2, 128, 128)
    d["table"][1] = d["table"][0]
    d["kv"][:] = 200
    d["kv"][1] = 131
    for a in d["codes"]:
        a[:] = np.where(a == 0x7F, 1, a)
    pu.check(d, pu.run(dbv, d, prefix_len=None))
    ok(dbv)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("far", [-30, -7, 12, 38])
@pytest.mark.parametrize("pow2", [True, False])
def test_value_scales_far_apart(dbv, far, pow2, wide):
    """Pages of a prefix whose value scales lie far apart: what a row has from
    pages of small scales keeps its bits."""
    c = pu.make(8, *with_wide([1100], [3], [0] * 3, [1, 2, 1], wide), 2, 4, 128, 16, pow2=pow2,
                far=far)
    # pages of large scales hold zeros; so the output is the others'
    big = np.arange(len(c["codes"][1])) % 2 == (1 if far > 0 else 0)
    c["codes"][1][big] &= 0x80
    c["scale"][0][:] = 2.0 ** -7
    got = pu.run(dbv, c)
    want, _, mag, size = pu.exact(c)
    # (no floor against the largest scale here: nothing of it comes in.  The tokens
    # behind the shared pages are a fraction of a page, of a class of their own.)
    tol = 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -15 * size[..., None]) * mag
    assert ((got["out"].double() - want).abs() <= tol).all()
    ok(dbv)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("scale", [0.0, -0.088, 1.0, 3e-5])
def test_softmax_scales(dbv, scale, wide):
    c = pu.make(9, *with_wide([600], [3], [30, 0, 5], [3, 1, 4], wide), 2, 4, 64, 64)
    pu.check(c, pu.run(dbv, c, scale=scale), scale)


def test_maxima_that_move(dbv):
    """Scores that grow along the prefix, so that sums are rescaled tile by tile,
    and rows that rise at different tiles."""
    c = pu.make(10, [4000], [5], [3] * 5, [9, 17, 30, 1, 8], 1, 4, 128, 64)
    order = c["table"][0, :4000 // 64]
    grow = 2.0 ** (np.arange(len(order)) // 7 - 12.0)
    c["scale"][0][order, 0] = grow.astype(np.float32)
    pu.check(c, pu.run(dbv, c))


@pytest.mark.parametrize("wide", [False, True])
def test_rows_that_are_not_finite(dbv, wide):
    """A query of NaN or infinity gives a row of NaN and no other; so does a new
    token of NaN for the rows that see it."""
    c = pu.make(11, *with_wide([500], [3], [10, 0, 3], [4, 6, 5], wide), 2, 4, 128, 32)
    c["q"][2, 1, 5] = float("nan")
    c["q"][7, 3, 100] = float("inf")
    got = pu.run(dbv, c)
    lost = torch.zeros(got["lse"].shape, dtype=torch.bool, device="cuda")
    lost[2, 1] = lost[7, 3] = True
    assert got["out"][lost].isnan().all() and got["lse"][lost].isnan().all()
    assert got["out"][~lost].isfinite().all()
    c["q"][2, 1, 5] = c["q"][7, 3, 100] = 0.0
    pos = int(c["kv"][1]) - 3
    page, row = c["table"][1, pos // 32], pos % 32
    c["codes"][1][page, 0, row, 9] = 0x7F
    got = pu.run(dbv, c)["out"].isnan().any(-1)
    want = torch.zeros_like(got)
    want[7:10, :4] = True  # tokens 3, 4 and 5 of sequence 1, heads of cache head 0
    assert torch.equal(got, want)


@pytest.mark.parametrize("wide", [False, True])
def test_rows_that_see_only_the_prefix(dbv, wide):
    """A mask that leaves a new token nothing of its own sequence."""
    c = pu.make(12, *with_wide([64], [2], [0, 0], [3, 4], wide), 1, 4, 128, 64, tree=True)
    c["mask"][:] = 0
    pu.check(c, pu.run(dbv, c))
    ok(dbv)


@pytest.mark.parametrize("wide", [False, True])
def test_strided_queries(dbv, wide):
    """Views into a projection, on and off 16 bytes, and a broadcast head."""
    c = pu.make(13, *with_wide([300], [3], [5, 6, 7], [2, 1, 4], wide), 2, 4, 64, 16)
    q = c["q"]
    T, Hq, D = q.shape
    for width, off in ((3 * Hq * D, 8), (Hq * D + 3, 1)):
        whole = torch.zeros((T, width + off), dtype=torch.bfloat16, device="cuda")
        view = whole[:, off:off + Hq * D].unflatten(1, (Hq, D))
        view.copy_(q)
        c["q"] = view
        pu.check(c, pu.run(dbv, c))
    c["q"] = q.transpose(0, 1).contiguous().transpose(0, 1)
    pu.check(c, pu.run(dbv, c))
    c["q"] = q[:, :1].expand(T, Hq, D)
    pu.check(c, pu.run(dbv, c))


def test_rows_behind_the_last_sequence_stay(dbv):
    c = pu.make(14, [200], [2], [5, 6], [3, 2], 2, 2, 128, 16)
    a, k = pu.tensors(c)
    T, Hq, D = c["q"].shape
    a[0] = torch.cat([c["q"], c["q"]])
    L = dbv.lib()
    h = dbv.default_handle(torch.device("cuda", 0))
    out = torch.full((2 * T, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    size = L.sv_kv_prefix_work_bytes(h.ptr, 2 * T, Hq, 2, D, 2, 1)
    work = torch.empty(size, dtype=torch.uint8, device="cuda")
    p = [t.data_ptr() for t in a]
    rc = L.sv_kv_prefix_attention(
        h.ptr, p[0], Hq * D, D, 2 * T, Hq, 2, D, *p[1:5], 16, a[1].shape[0], p[5],
        a[5].shape[1], p[6], p[7], 2, None, None, 1, None, 0, D ** -0.5, out.data_ptr(), None,
        work.data_ptr(), size, torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    want = pu.run(dbv, c)["out"]
    assert torch.equal(out[:T], want) and (out[T:] == 7.0).all()
    # a workspace that is a byte too small
    rc = L.sv_kv_prefix_attention(
        h.ptr, p[0], Hq * D, D, 2 * T, Hq, 2, D, *p[1:5], 16, a[1].shape[0], p[5],
        a[5].shape[1], p[6], p[7], 2, None, None, 1, None, 0, D ** -0.5, out.data_ptr(), None,
        work.data_ptr(), size - 1, torch.cuda.current_stream().cuda_stream)
    assert rc == dbv.SV_ERR_INVALID_ARG


def test_nothing_of_the_workspace_is_read(dbv):
    """The same result whatever the workspace held, and the same bits again."""
    c = pu.make(15, [3000], [4], [5, 0, 64, 90], [9, 20, 33, 1], 4, 4, 128, 64)
    want = pu.run(dbv, c)
    for fill in (0x00, 0xFF, 0x7F):
        a, k = pu.tensors(c)
        size = dbv.lib().sv_kv_prefix_work_bytes(
            dbv.default_handle(torch.device("cuda", 0)).ptr, *c["q"].shape[:2], 4, 128, 4, 1)
        torch.full((size,), fill, dtype=torch.uint8, device="cuda")  # (goes back to the pool)
        got = pu.run(dbv, c)
        assert all(torch.equal(got[n], want[n]) for n in want)


def test_streams_and_graphs(dbv):
    """Calls on two streams at once, one of them from two graphs of one handle."""
    cs = [pu.make(16, [6000], [6], [100] * 6, [5] * 6, 2, 4, 128, 64),
          pu.make(17, [900], [20], [60] * 20, [9] * 20, 2, 4, 64, 32)]
    want = [pu.run(dbv, c) for c in cs]
    calls = []
    for c in cs:
        a, k = pu.tensors(c)
        p, g = pu.dev(c["prefix"]), pu.dev(c["group"])
        calls.append(lambda a=a, k=k, p=p, g=g: dbv.sv_kv_prefix_attention(*a, p, cu_group=g, **k))
    torch.cuda.synchronize()
    graphs, outs = [], []
    for f in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(f())
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(4)]
    got = [[], []]
    torch.cuda.synchronize()
    for _ in range(30):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(calls[i]())
            with torch.cuda.stream(streams[2 + i]):
                graphs[i].replay()
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x[n], want[i][n]) for x in got[i] for n in x)
        assert all(torch.equal(outs[i][n], want[i][n]) for n in want[i])
    ok(dbv)


def test_a_stream_that_is_not_the_current_one(dbv):
    c = pu.make(18, [700], [3], [5] * 3, [3] * 3, 2, 4, 128, 64)
    want = pu.run(dbv, c)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for given in (s, s.cuda_stream):
        got = pu.run(dbv, c, stream=given)
        s.synchronize()
        torch.cuda.synchronize()
        assert all(torch.equal(got[n], want[n]) for n in want)


def test_bad_lengths_and_groups_are_latched(dbv):
    c = pu.make(19, [200], [3], [5, 6, 7], [3, 2, 1], 2, 2, 128, 16)
    h = dbv.default_handle(torch.device("cuda", 0))

    def latched():
        with pytest.raises(dbv.SVError) as e:
            h.sync_status()
        assert e.value.status == dbv.SV_ERR_DEVICE_BOUNDS

    for group in ([0, 2, 1, 3], [-1, 3], [0, 4], [3, 0]):
        got = pu.run(dbv, c, prefix_len=None, cu_group=pu.dev(group))
        latched()
        pu.check(c, got)  # nothing is shared, the rows are right
    for name, i, v in (("kv", 1, 1), ("kv", 2, 10 ** 6), ("cu", 3, 99)):
        d = dict(c, **{name: c[name].copy()})
        d[name][i] = v
        a, k = pu.tensors(d)
        dbv.sv_kv_prefix_attention(*a, **k)
        latched()
    d = dict(c, table=c["table"].copy())
    d["table"][:, 3] = len(c["codes"][0])  # a shared page beyond the cache
    a, k = pu.tensors(d)
    dbv.sv_kv_prefix_attention(*a, **k)
    latched()
    pu.check(c, pu.run(dbv, c))
    ok(dbv)


@pytest.mark.parametrize("new,H,G,D,block", [([2000, 3, 40], 1, 2, 64, 64), ([700, 900], 2, 1, 128, 16),
                                             ([1, 33, 16, 17, 32, 8], 2, 1, 128, 32),
                                             ([4, 5, 4, 5, 1], 1, 8, 64, 128)])
def test_rows_on_both_sides(dbv, new, H, G, D, block):
    """Sequences of up to 32 rows a head and of more, in one group; whole prompts."""
    n = len(new)
    c = pu.make(n + H, [530], [n], [700 + 50 * i for i in range(n)], new, H, G, D, block)
    pu.check(c, pu.run(dbv, c))
    ok(dbv)


@pytest.mark.parametrize("after,new,G,D", [([30000, 20000], [1, 1], 3, 128), ([25000], [1], 8, 64),
                                           ([9000, 17, 40000], [2, 4, 3], 7, 64)])
@pytest.mark.parametrize("far", [0, 9])
def test_own_tokens_in_many_ranges(dbv, after, new, G, D, far):
    """Few sequences with long contexts of their own, which many warps share."""
    n = len(new)
    c = pu.make(n + G, [64], [n], after, new, 1, G, D, 64, pow2=far == 0, far=far)
    pu.check(c, pu.run(dbv, c))
    ok(dbv)


def test_many_sequences(dbv):
    """Thousands of sequences and groups: more tasks than warps, and spans."""
    r = np.random.RandomState(3)
    sizes = [int(x) for x in r.randint(1, 6, 900)]
    B = sum(sizes)
    c = pu.make(4, [int(x) for x in r.randint(1, 70, 900)], sizes,
                [int(x) for x in r.randint(0, 40, B)], [int(x) for x in r.randint(0, 3, B)],
                1, 2, 64, 16)
    pu.check(c, pu.run(dbv, c))
    ok(dbv)


@pytest.mark.parametrize("far", [-40, 7, 30])
def test_own_scales_far_apart(dbv, far):
    """What a sequence has of its own, behind no prefix: pages of small value scales
    keep their bits beside pages of large ones that hold zeros."""
    c = pu.make(20, [0], [3], [700, 45, 130], [1, 3, 8], 2, 4, 128, 16, far=far)
    big = np.arange(len(c["codes"][1])) % 2 == (1 if far > 0 else 0)
    c["codes"][1][big] &= 0x80
    c["scale"][0][:] = 2.0 ** -7
    got = pu.run(dbv, c)
    want, _, mag, size = pu.exact(c)
    tol = 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -15 * size[..., None]) * mag
    assert ((got["out"].double() - want).abs() <= tol).all()
    ok(dbv)


def test_sequences_out_of_order(dbv):
    """cu_new that goes back: more rows than there are, in all.  Latched; what lies
    behind the outputs and the workspace is left alone, and the next call is right."""
    c = pu.make(21, [64], [1], [20], [40], 2, 2, 128, 16)
    B = 300
    d = dict(c, cu=np.append(np.tile([0, 40], B // 2), 0).astype(np.int32),
             table=np.repeat(c["table"], B, 0), kv=np.repeat(c["kv"], B))
    a, k = pu.tensors(d)
    dbv.sv_kv_prefix_attention(*a, **k)
    h = dbv.default_handle(torch.device("cuda", 0))
    with pytest.raises(dbv.SVError) as e:
        h.sync_status()
    assert e.value.status == dbv.SV_ERR_DEVICE_BOUNDS
    pu.check(c, pu.run(dbv, c))
    ok(dbv)


def test_masks_of_fewer_words(dbv):
    """New tokens beyond a mask's words are seen by none."""
    c = pu.make(22, [96], [3], [5, 0, 9], [70, 40, 3], 2, 2, 64, 32, tree=True)
    full = c["mask"]
    c["mask"] = np.ascontiguousarray(full[:, :2])
    got = pu.run(dbv, c)
    c["mask"] = full & np.array([2 ** 32 - 1, 2 ** 32 - 1, 0], np.uint32)
    pu.check(c, got)
    ok(dbv)


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_units_that_are_not_cut(dbv, D, tree):
    """More small units than CTAs, beside some that are cut; the same bits each time,
    whichever CTA takes them."""
    r = np.random.RandomState(7)
    sizes = [40, 1, 30]
    B = sum(sizes)
    new = [int(x) for x in r.randint(5, 24, B)]
    after = [int(x) for x in r.randint(0, 300, B)]
    after[5], after[50], new[60] = 5000, 4000, 300
    c = pu.make(23, [900, 50, 2500], sizes, after, new, 4, 4, D, 32, tree=tree)
    want = pu.run(dbv, c)
    pu.check(c, want)
    for _ in range(5):
        got = pu.run(dbv, c)
        assert all(torch.equal(got[n], want[n]) for n in want)
    ok(dbv)
