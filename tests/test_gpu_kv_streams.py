"""Calls of sv_kv_attention on one handle from several streams, and in a graph."""
import pytest
import torch

from test_gpu_kv_units import call, case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dbv():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import draft_block_verification_gb300 as m
    return m


def cases():
    """Calls whose units are shared by CTAs."""
    return [case(1, [4000, 9000], [3, 5], 2, 4, 128, 64),
            case(2, [700] * 40, [9] * 40, 2, 4, 64, 32)]


def prepared(dbv, c):
    """The call with its tensors already on the device."""
    t = lambda a: torch.as_tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    table, kv, cu = t(c["table"]), t(c["kv"]), t(c["cu"])
    return lambda h=None: dbv.sv_kv_attention(c["q"], *c["cache"], *c["scale"], table, kv, cu,
                                              want_lse=True, handle=h)


def same(a, b):
    return all(torch.equal(a[n], b[n]) for n in a)


def test_streams_overlap_on_one_handle(dbv):
    cs = cases()
    want = [call(dbv, c) for c in cs]
    runs = [prepared(dbv, c) for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(100):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(runs[i]())
    torch.cuda.synchronize()
    for i in range(2):
        assert all(same(g, want[i]) for g in got[i])
    dbv.default_handle(torch.device("cuda", 0)).sync_status()


def test_a_graph_beside_another_stream(dbv):
    cs = cases()
    want = [call(dbv, c) for c in cs]
    runs = [prepared(dbv, c) for c in cs]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = runs[0]()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(50):
        g.replay()
        with torch.cuda.stream(s):
            got.append(runs[1]())
    torch.cuda.synchronize()
    assert same(out, want[0]) and all(same(x, want[1]) for x in got)


def test_more_streams_than_workspaces(dbv):
    cs = cases()
    want = [call(dbv, c) for c in cs]
    runs = [prepared(dbv, c) for c in cs]
    h = dbv.Handle()
    streams = [torch.cuda.Stream() for _ in range(24)]
    torch.cuda.synchronize()
    try:
        for turn in range(2):
            got = []
            for i, s in enumerate(streams):
                with torch.cuda.stream(s):
                    got.append(runs[(i + turn) % 2](h))
            torch.cuda.synchronize()
            assert all(same(x, want[(i + turn) % 2]) for i, x in enumerate(got))
        h.sync_status()
    finally:
        h.close()


def test_a_capture_needs_an_earlier_call(dbv):
    run = prepared(dbv, cases()[0])
    h = dbv.Handle()
    try:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            torch.zeros(1, device="cuda")
            with pytest.raises(dbv.SVError) as e:
                run(h)
        assert e.value.status == dbv.SV_ERR_UNSUPPORTED
        run(h)
        h.sync_status()
    finally:
        h.close()
