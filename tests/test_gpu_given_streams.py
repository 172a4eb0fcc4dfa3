"""Calls with stream=: what they allocate belongs to that stream, so that calls on it and
on the current one may be in flight together."""
import pytest
import torch

import prefix_util as pu
from test_gpu_kv_prefix import ok

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dbv():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import draft_block_verification_gb300 as m
    return m


@pytest.mark.parametrize("raw", [False, True])
def test_results_are_of_the_given_stream(dbv, raw):
    """A block that the current stream has given back, and may still use, is not taken."""
    c = pu.make(40, [600], [4], [5] * 4, [9] * 4, 2, 4, 128, 32)
    q = c["q"]
    pos = torch.arange(q.shape[0], dtype=torch.int32, device="cuda")
    freq = torch.full((64,), 0.1, device="cuda")
    a, k = pu.tensors(c)
    size = dbv.lib().sv_kv_prefix_work_bytes(
        dbv.default_handle(torch.device("cuda", 0)).ptr, *q.shape[:2], 2, 128, 4, 1)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    # blocks of the sizes that the calls ask for
    old = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in (q.numel() * 2, size) * 2]
    span = [(t.data_ptr(), t.data_ptr() + t.numel()) for t in old]
    del old
    for call in (lambda **kw: dbv.sv_kv_prefix_attention(*a, **k, **kw),
                 lambda **kw: dbv.sv_kv_attention(*a, **k, **kw),
                 lambda **kw: {"q": dbv.sv_qk_norm_rope(q, None, pos, freq, **kw)["q"]}):
        got = call(stream=s.cuda_stream if raw else s)
        for t in got.values():
            assert not any(lo <= t.data_ptr() < hi for lo, hi in span)
        torch.cuda.synchronize()
    ok(dbv)


def test_calls_on_two_streams_without_waits(dbv):
    """Calls on the current stream and on a given one in turn, never synchronised: each
    has a workspace to itself."""
    cs = [pu.make(41, [3000], [12], [40] * 12, [7] * 12, 2, 4, 128, 64),
          pu.make(42, [2000, 500], [10, 9], [60] * 19, [40] * 19, 2, 4, 64, 32)]
    want = [pu.run(dbv, c) for c in cs]
    calls = []
    for c in cs:
        a, k = pu.tensors(c)
        p, g = pu.dev(c["prefix"]), pu.dev(c["group"])
        calls.append(lambda stream, a=a, k=k, p=p, g=g: dbv.sv_kv_prefix_attention(
            *a, p, cu_group=g, stream=stream, **k))
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for i in range(60):
        which = i % 2 ^ (i // 20 & 1)
        got.append((which, calls[which](None if i % 2 else s)))
    torch.cuda.synchronize()
    for which, x in got:
        assert all(torch.equal(x[n], want[which][n]) for n in x)
    ok(dbv)
