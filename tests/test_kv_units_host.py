"""What the kernels of the prefix attention compute in plain arithmetic, compiled for the
host."""
import os
import subprocess

from draft_block_verification_gb300 import _build

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include "sv_kv.cuh"
int main(int n, char **a)
{
    for (int i = 1; i + 2 < n; i += 3)
        printf("%d ", (int)sv::unit_known(atoi(a[i]), atoi(a[i + 1]), atoi(a[i + 2])));
}
"""


def test_entries_of_units_that_were_never_written(tmp_path):
    """A unit's entry bounds a loop and indexes the workspace: what a kernel that gave
    up left there must pass as no CTAs."""
    src, exe = tmp_path / "units.cpp", tmp_path / "units"
    src.write_text(PROGRAM)
    cuda = os.path.join(os.path.dirname(_build._nvcc()), "..", "include")
    subprocess.run(["g++", "-std=c++17", "-I" + _build.CSRC, "-I" + cuda, str(src), "-o", str(exe)],
                   check=True)
    big = 2 ** 31 - 1
    cases = [(0, 0, 1, 1), (0, 151, 152, 1), (151, 151, 152, 1), (3, 2, 152, 0), (0, -1, 152, 0),
             (-1, 0, 152, 0), (0, 152, 152, 0), (-5, -3, 152, 0), (-big, big, 152, 0),
             (big, big, 152, 0), (0, big, 152, 0), (-1, -1, 152, 0)]
    args = [str(x) for c in cases for x in c[:3]]
    out = subprocess.run([str(exe)] + args, check=True, capture_output=True, text=True).stdout
    assert out.split() == [str(c[3]) for c in cases]
