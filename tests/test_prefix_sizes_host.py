"""Sizes that the prefix attention has no workspace for are refused as such, whether or not
one is given."""
import pytest

from test_kv_host import h, lib  # noqa: F401  (fixtures)
from test_serving_host import prefix_args


@pytest.mark.parametrize("kw", [dict(T=1 << 27, Hq=16, H=16, groups=1 << 27, B=1 << 27),
                                dict(B=1 << 30), dict(groups=1 << 30)])
def test_sizes_without_a_workspace(lib, h, kw):  # noqa: F811
    a = dict(T=4, Hq=4, H=2, D=64, B=2, groups=1)
    a.update(kw)
    assert lib.sv_kv_prefix_work_bytes(h, *a.values()) == 0
    assert lib.sv_kv_prefix_attention(h, *prefix_args(work=None, size=0, **kw)) == 5
