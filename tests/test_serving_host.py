"""Host side of the calls around the cache's attention: refusals that answer
before anything touches a GPU."""
import pytest
import torch

from test_kv_host import OK, attend_args, h, lib  # noqa: F401  (fixtures)


def prefix_args(**kw):
    a = dict(q=OK, qt=64, qh=64, T=4, Hq=4, H=2, D=64, kc=OK, vc=OK, ks=OK, vs=OK, block=64,
             pages=4, table=OK, cols=4, kv=OK, cu=OK, B=2, prefix=OK, group=OK, groups=1,
             mask=None, words=0, scale=0.125, out=OK, lse=None, work=OK, size=1 << 40, stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), 1), (dict(q=OK + 1), 1), (dict(qt=-1), 1), (dict(T=-1), 1), (dict(Hq=0), 1),
    (dict(Hq=3), 1), (dict(H=0), 1), (dict(D=80), 5), (dict(kc=OK + 4), 1), (dict(vs=None), 1),
    (dict(block=65), 1), (dict(pages=0), 1), (dict(table=None), 1), (dict(cols=0), 1),
    (dict(kv=None), 1), (dict(cu=None), 1), (dict(B=-1), 1), (dict(mask=OK, words=0), 1),
    (dict(scale=float("inf")), 1), (dict(out=None), 1), (dict(out=OK + 2), 1),
    (dict(T=1 << 30), 5), (dict(cols=1 << 26), 5), (dict(groups=0), 1),
    (dict(group=None, groups=2), 1), (dict(work=None), 1), (dict(work=OK + 8), 1),
    (dict(size=100), 1), (dict(T=1 << 27, Hq=16, H=16, groups=1 << 27, B=1 << 27), 5),
    (dict(B=1 << 30), 5), (dict(groups=1 << 30), 5)])
def test_prefix_refusals(lib, h, kw, want):  # noqa: F811
    assert lib.sv_kv_prefix_attention(h, *prefix_args(**kw)) == want


def test_prefix_work_bytes(lib, h):  # noqa: F811
    size = lambda *a: lib.sv_kv_prefix_work_bytes(h, *a)  # noqa: E731
    # sums of a unit for each 256 rows of a head and each group: [D + 2][256] fp32
    unit = 256 * 66 * 4
    assert size(1024, 4, 2, 64, 2, 1) - size(4, 4, 2, 64, 2, 1) >= 2 * 8 * unit
    assert size(1024, 4, 2, 64, 9, 7) - size(1024, 4, 2, 64, 9, 1) >= 2 * 6 * unit
    assert size(4, 4, 2, 64, 2, 1) < size(4, 4, 2, 128, 2, 1)
    for bad in ((-1, 4, 2, 64, 2, 1), (4, 3, 2, 64, 2, 1), (4, 4, 2, 96, 2, 1),
                (4, 4, 2, 64, -2, 1), (4, 4, 2, 64, 2, 0), (1 << 30, 4, 2, 64, 2, 1),
                (4, 4, 2, 64, 1 << 30, 1)):
        assert size(*bad) == 0


def read_args(**kw):
    a = dict(kc=OK, vc=OK, ks=OK, vs=OK, H=2, D=64, block=64, pages=4, table=OK, cols=4,
             first=None, cu=OK, B=2, T=4, k=OK, v=2 * OK, dtype=1, kt=128, kh=64, vt=128, vh=64,
             stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(kc=None), 1), (dict(vc=OK + 8), 1), (dict(ks=None), 1), (dict(H=0), 1),
    (dict(H=40000), 5), (dict(D=96), 5), (dict(block=24), 1), (dict(pages=0), 1),
    (dict(pages=1 << 30), 5), (dict(table=None), 1), (dict(cols=0), 1), (dict(cols=1 << 26), 5),
    (dict(cu=None), 1), (dict(B=-1), 1), (dict(T=-1), 1), (dict(k=None), 1), (dict(v=OK + 1), 1),
    (dict(dtype=0, k=OK + 2), 1), (dict(dtype=3), 1), (dict(kt=-1), 1), (dict(vh=-1), 1),
    (dict(v=OK), 1), (dict(kt=0), 1), (dict(vh=0), 1)])
def test_read_refusals(lib, h, kw, want):  # noqa: F811
    assert lib.sv_kv_read(h, *read_args(**kw)) == want


def rope_args(**kw):
    a = dict(q=OK, k=2 * OK, dtype=1, qt=256, qh=64, kt=128, kh=64, T=4, Hq=4, H=2, D=64, qw=OK,
             kw=OK, eps=1e-6, f=OK, rot=64, inter=0, pos=OK, qo=3 * OK, ko=4 * OK, odtype=1,
             qot=256, qoh=64, kot=128, koh=64, stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), 1), (dict(k=None), 1), (dict(q=OK + 1), 1), (dict(dtype=0, k=OK + 2), 1),
    (dict(dtype=2), 1), (dict(odtype=5), 1), (dict(qt=-1), 1), (dict(koh=-1), 1), (dict(T=-1), 1),
    (dict(Hq=-1), 1), (dict(D=63), 1), (dict(D=0), 1), (dict(D=514), 5), (dict(rot=-2), 1),
    (dict(rot=7), 1), (dict(rot=66), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1),
    (dict(f=None), 1), (dict(pos=None), 1), (dict(qo=None), 1), (dict(ko=4 * OK + 1), 1),
    (dict(odtype=0, qo=OK + 2), 1), (dict(qot=0), 1), (dict(koh=0), 1),
    (dict(qo=OK, qoh=32), 1), (dict(qo=OK, odtype=0), 1), (dict(qo=2 * OK), 1),
    (dict(ko=3 * OK), 1), (dict(ko=OK), 1), (dict(T=1 << 30), 5)])
def test_rope_refusals(lib, h, kw, want):  # noqa: F811
    assert lib.sv_qk_norm_rope(h, *rope_args(**kw)) == want


def test_null_handle_is_refused(lib):  # noqa: F811
    assert lib.sv_kv_prefix_attention(None, *prefix_args()) == 1
    assert lib.sv_kv_prefix_work_bytes(None, 4, 4, 2, 64, 2, 1) == 0
    assert lib.sv_kv_read(None, *read_args()) == 1
    assert lib.sv_qk_norm_rope(None, *rope_args()) == 1


def test_nothing_to_do_is_ok(lib, h):  # noqa: F811
    assert lib.sv_kv_prefix_attention(h, *prefix_args(T=0, q=None, out=None, work=None)) == 0
    assert lib.sv_kv_prefix_attention(h, *prefix_args(B=0)) == 0
    assert lib.sv_kv_read(h, *read_args(T=0, k=None, v=None)) == 0
    assert lib.sv_qk_norm_rope(h, *rope_args(T=0, q=None, k=None)) == 0
    assert lib.sv_qk_norm_rope(h, *rope_args(Hq=0, H=0, pos=None)) == 0


@pytest.mark.parametrize("call", ["sv_kv_prefix_attention", "sv_kv_read", "sv_qk_norm_rope"])
def test_fault_injection_answers_before_a_launch(lib, h, call, monkeypatch):  # noqa: F811
    args = {"sv_kv_prefix_attention": prefix_args, "sv_kv_read": read_args,
            "sv_qk_norm_rope": rope_args}[call]()
    monkeypatch.setenv("SV_FAULT_INJECT", "sv_kv_plan:2,%s:3" % call)
    assert getattr(lib, call)(h, *args) == 3


def test_binding_refuses_host_tensors():
    import draft_block_verification_gb300 as dbv
    z, i = torch.zeros((2, 8)), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        dbv.sv_kv_prefix_attention(z, z, z, z, z, i, i, i)
    with pytest.raises(ValueError):
        dbv.sv_kv_read(z, z, z, z, i, i, 2)
    with pytest.raises(ValueError):
        dbv.sv_qk_norm_rope(z, z, i, z)
