"""sv_kv_plan refuses outputs that are its inputs: every CTA reads the inputs
while others write the outputs."""
import ctypes as C

import pytest

from test_kv_host import h, lib, plan_args  # noqa: F401

OUT = dict(kv=1, cu=2, held_out=3, free_out=4, slot=5, pos=6)
IN = dict(cached=7, new=8, held=9, free_pos=10, ids=11, table=12)


@pytest.mark.parametrize("o", OUT)
@pytest.mark.parametrize("i", IN)
def test_plan_refuses_outputs_that_are_inputs(lib, h, o, i):  # noqa: F811
    apart = {k: v * 65536 for k, v in (OUT | IN).items()}
    assert lib.sv_kv_plan(h, *plan_args(**dict(apart, **{o: apart[i]}))) == 1


def test_plan_looks_at_addresses_after_the_limits(lib, h):  # noqa: F811
    assert lib.sv_kv_plan(h, *plan_args(B=16385, kv=4096)) == 5


def test_plan_of_nothing_has_no_addresses_to_compare(lib, monkeypatch):  # noqa: F811
    """Null outputs of an empty batch are not null inputs."""
    monkeypatch.setenv("SV_FAULT_INJECT", "sv_kv_plan:4")  # answers at the launch point
    none = dict(cached=None, new=None, held=None, table=None, kv=None, held_out=None, slot=None,
                pos=None)
    own = C.cast(C.create_string_buffer(1 << 16), C.c_void_p)
    args = plan_args(B=0, cap=0, cu=1 << 16, free_out=2 << 16, free_pos=3 << 16, ids=4 << 16,
                     **none)
    assert lib.sv_kv_plan(own, *args) == 4
