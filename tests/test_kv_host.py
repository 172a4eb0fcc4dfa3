"""Host side of the paged cache and sampling calls: refusals that answer before
anything touches a GPU, and the plain forms that the GPU tests compare with."""
import ctypes as C

import numpy as np
import pytest
import torch

import kv_util


@pytest.fixture(scope="module")
def lib():
    from draft_block_verification_gb300 import _build
    _build.build()
    import draft_block_verification_gb300 as dbv
    return dbv.lib()


@pytest.fixture(scope="module")
def h():
    """Memory in a handle's place: every refusal below answers before it is read."""
    return C.cast(C.create_string_buffer(1 << 16), C.c_void_p)


OK = 4096  # an aligned address that a refused call never follows


def plan_args(**kw):
    a = dict(B=2, block=64, cols=4, ring=8, cap=10, cached=OK, new=OK, held=OK, free_pos=OK,
             ids=OK, table=OK, kv=2 * OK, cu=OK, held_out=2 * OK, free_out=2 * OK, slot=OK,
             pos=OK, stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(B=-1), 1), (dict(block=48), 1), (dict(block=0), 1), (dict(block=256), 1),
    (dict(cols=0), 1), (dict(ring=0), 1), (dict(cap=-1), 1), (dict(cached=None), 1),
    (dict(new=None), 1), (dict(held=None), 1), (dict(free_pos=None), 1), (dict(ids=None), 1),
    (dict(table=None), 1), (dict(kv=None), 1), (dict(cu=None), 1), (dict(slot=None), 1),
    (dict(pos=None), 1), (dict(held_out=OK), 1), (dict(free_out=OK), 1), (dict(kv=OK), 1),
    (dict(B=16385), 5)])
def test_plan_refusals(lib, h, kw, want):
    assert lib.sv_kv_plan(h, *plan_args(**kw)) == want


def append_args(**kw):
    a = dict(k=OK, v=OK, dtype=1, kt=64, kh=64, vt=64, vh=64, T=4, H=2, D=64, block=64, pages=4,
             slot=OK, kc=OK, vc=OK, ks=OK, vs=OK, stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(k=None), 1), (dict(v=None), 1), (dict(k=OK + 1), 1), (dict(dtype=2), 1),
    (dict(dtype=0, v=OK + 2), 1), (dict(kt=-1), 1), (dict(vh=-1), 1), (dict(T=-1), 1),
    (dict(H=0), 1), (dict(D=96), 5), (dict(D=256), 5), (dict(block=63), 1), (dict(pages=0), 1),
    (dict(slot=None), 1), (dict(kc=None), 1), (dict(vc=OK + 8), 1), (dict(ks=None), 1),
    (dict(H=40000), 5), (dict(pages=1 << 30), 5)])
def test_append_refusals(lib, h, kw, want):
    assert lib.sv_kv_append(h, *append_args(**kw)) == want


def attend_args(**kw):
    a = dict(q=OK, qt=64, qh=64, T=4, Hq=4, H=2, D=64, kc=OK, vc=OK, ks=OK, vs=OK, block=64,
             pages=4, table=OK, cols=4, kv=OK, cu=OK, B=2, mask=None, words=0, scale=0.125,
             out=OK, lse=None, stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), 1), (dict(q=OK + 1), 1), (dict(qt=-1), 1), (dict(T=-1), 1), (dict(Hq=0), 1),
    (dict(Hq=3), 1), (dict(H=0), 1), (dict(D=80), 5), (dict(kc=OK + 4), 1), (dict(vs=None), 1),
    (dict(block=65), 1), (dict(pages=0), 1), (dict(table=None), 1), (dict(cols=0), 1),
    (dict(kv=None), 1), (dict(cu=None), 1), (dict(B=-1), 1), (dict(mask=OK, words=0), 1),
    (dict(scale=float("nan")), 1), (dict(out=None), 1), (dict(out=OK + 2), 1),
    (dict(T=1 << 30), 5), (dict(cols=1 << 26), 5)])
def test_attention_refusals(lib, h, kw, want):
    assert lib.sv_kv_attention(h, *attend_args(**kw)) == want


def rows_args(**kw):
    a = dict(x=OK, dtype=1, rs=100, R=2, V=100, u=OK, T=None, k=None, p=None, m=None, token=OK,
             prob=OK, kept=OK, stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), 1), (dict(x=OK + 1), 1), (dict(dtype=0, x=OK + 2), 1), (dict(dtype=7), 1),
    (dict(rs=99), 1), (dict(R=-1), 1), (dict(V=0), 1), (dict(u=None), 1), (dict(token=None), 1),
    (dict(prob=None), 1), (dict(kept=None), 1), (dict(V=(1 << 20) + 1, rs=1 << 21), 5)])
def test_rows_refusals(lib, h, kw, want):
    assert lib.sv_sample_rows(h, *rows_args(**kw)) == want


def test_null_handle_is_refused(lib):
    assert lib.sv_kv_plan(None, *plan_args()) == 1
    assert lib.sv_kv_append(None, *append_args()) == 1
    assert lib.sv_kv_attention(None, *attend_args()) == 1
    assert lib.sv_sample_rows(None, *rows_args()) == 1


def test_nothing_to_do_is_ok(lib, h):
    assert lib.sv_kv_append(h, *append_args(T=0, k=None, v=None, slot=None)) == 0
    assert lib.sv_kv_attention(h, *attend_args(T=0, q=None, out=None)) == 0
    assert lib.sv_kv_attention(h, *attend_args(B=0)) == 0
    assert lib.sv_sample_rows(h, *rows_args(R=0, x=None)) == 0


def test_binding_refuses_host_tensors():
    import draft_block_verification_gb300 as dbv
    z = torch.zeros((2, 8))
    with pytest.raises(ValueError):
        dbv.sv_sample_rows(z, z[:, 0])
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        dbv.sv_kv_plan(i, i, i, i[None], i, i, 16, 4)
    with pytest.raises(ValueError):
        dbv.sv_kv_append(z, z, i, z, z, z, z)
    with pytest.raises(ValueError):
        dbv.sv_kv_attention(z, z, z, z, z, i, i, i)


def test_codes_round_like_torch():
    """The plain encoder against torch's conversion, at every code, at every
    midpoint and around it, and on random values."""
    m = kv_util.MAGNITUDES
    mid = (m[1:] + m[:-1]) / 2
    r = np.random.RandomState(0).randn(4000) * 60
    x = np.concatenate([m, mid, mid * (1 + 2.0 ** -20), mid * (1 - 2.0 ** -20), r])
    x = np.concatenate([x, -x]).astype(np.float32).clip(-448, 448)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(kv_util.e4m3_encode(x), want)
    assert np.array_equal(kv_util.e4m3_decode(want),
                          torch.from_numpy(want).view(torch.float8_e4m3fn).double().numpy())


def test_needed_scale_at_its_borders():
    for e in (-40, -3, 0, 7, 39):
        top = 448.0 * 2.0 ** e
        assert kv_util.needed_scale(top) == 2.0 ** e
        assert kv_util.needed_scale(np.nextafter(top, np.inf)) == 2.0 ** (e + 1)
    assert kv_util.needed_scale(0.0) == 2.0 ** -40
    assert kv_util.needed_scale(np.inf) == 2.0 ** 40
