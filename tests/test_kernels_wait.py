"""Kernels that may start while the one before them still runs wait for it before they
touch memory, and before they let the next one start."""
import os
import re

import pytest

from draft_block_verification_gb300 import _build


def kernels():
    for name in sorted(os.listdir(_build.CSRC)):
        text = open(os.path.join(_build.CSRC, name)).read()
        for m in re.finditer(r"__global__(.*?)\n\{", text, re.S):
            found = re.search(r"(\w+_kernel)\(", m.group(1))
            end = text.index("\n}\n", m.end())
            yield name, found.group(1), re.sub(r"//[^\n]*", "", text[m.end():end])


def test_there_are_kernels():
    names = {k for _, k, _ in kernels()}
    assert {"tail_kernel", "prefix_kernel", "prefix_prep_kernel", "rope_kernel", "read_kernel"} <= names


@pytest.mark.parametrize("name,kernel,body", [pytest.param(*k, id=k[0] + ":" + k[1])
                                              for k in kernels() if "pdl_" in k[2]])
def test_wait_comes_first(name, kernel, body):
    assert "pdl_wait();" in body
    first = body.index("pdl_wait();")
    for later in ("pdl_trigger();", "__ldcg(", "__ldg(", "latch("):
        if later in body:
            assert first < body.index(later), later
