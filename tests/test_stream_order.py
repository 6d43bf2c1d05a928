"""Launches that overlap the end of the one before them: what the sources of
such kernels must hold to, read from them."""
import os
import re

import pytest

from attention_forward_14_gb300.build import CSRC


def _source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def _files():
    """The translation units that launch so, with every header of this folder that they include."""
    users = [n for n in sorted(os.listdir(CSRC)) if n.endswith(".cu") and "launch_overlapped" in _source(n)]
    assert len(users) >= 4
    return users


@pytest.mark.parametrize("name", _files())
def test_every_kernel_waits_for_what_came_before(name):
    kernels = re.split(r"__global__ void", _source(name))[1:]
    assert kernels
    for k in kernels:
        assert "await_previous()" in k.split("__global__")[0], k[:120]


@pytest.mark.parametrize("name", [*_files(), "rows.cuh", "attn_kv8_common.cuh"])
def test_no_loads_of_memory_that_must_not_change(name):
    """ld.global.nc may be moved ahead of the wait, and asks for memory that
    stays as it is while the kernel lives."""
    assert not re.search(r"__ldg\s*\(|ld\.global\.nc|ld\.global(\.\w+)*\.nc", _source(name))
