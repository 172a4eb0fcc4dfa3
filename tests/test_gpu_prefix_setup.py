"""A prefix attention that cannot run takes no other call with it."""
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


def test_a_setup_that_fails_is_that_calls_own(dbv, monkeypatch):
    c = pu.make(60, [200], [2], [5, 6], [3, 2], 2, 2, 128, 16)
    want = pu.run(dbv, c)
    monkeypatch.setenv("SV_FAULT_INJECT", "sv_kv_prefix_setup:5")
    h = dbv.Handle()
    try:
        with pytest.raises(dbv.SVError) as e:
            pu.run(dbv, c, handle=h)
        assert e.value.status == dbv.SV_ERR_UNSUPPORTED
        monkeypatch.delenv("SV_FAULT_INJECT")
        with pytest.raises(dbv.SVError):
            pu.run(dbv, c, handle=h)
        a, k = pu.tensors(c)
        out = dbv.sv_kv_attention(*a, handle=h, **k)
        h.sync_status()
        pu.check(c, out)
        logits = torch.randn((2, 4, 1000), device="cuda")
        acc, _ = dbv.sv_verify_greedy(logits, logits[:, :3].argmax(-1).int(), handle=h)
        h.sync_status()
        assert acc.tolist() == [3, 3]
    finally:
        h.close()
    got = pu.run(dbv, c)
    assert all(torch.equal(got[n], want[n]) for n in want)
