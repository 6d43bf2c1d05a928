"""The checked build (the same sources with what the kernels decode and index
compared with its bounds) runs the cases of the operators around the
attention, each against its definition as in its own test file, with the
status word read after every case: no check may fire on valid inputs."""
import pytest

from attention_forward_14_gb300 import binding

import test_kv8 as K8
import test_kv_append as AP
import test_qk_norm_rope as NR

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def checked_library():
    from attention_forward_14_gb300.build import build
    build()
    saved = binding.load()
    binding._lib = binding.load(binding.CHECKED_LIB_PATH)
    binding.status_clear()
    try:
        yield
        assert binding._fast_lib is binding._lib  # the calls went to it
    finally:
        binding._lib = saved


def _clean(what):
    code = binding.status()
    assert code[0] == 0, f"{what}: status {code}"


@pytest.mark.parametrize("case", NR.CASES, ids=str)
def test_checked_norm(case):
    NR.test_forward(case)
    NR.test_backward(case)
    # (a position past the tables is one of the cases' inputs, and is recorded)
    assert binding.status()[0] in (0, 4)
    binding.status_clear()


@pytest.mark.parametrize("case", AP.CASES, ids=str)
def test_checked_append(case):
    AP.test_append(case)
    _clean(f"append {case}")


@pytest.mark.parametrize("block", [0, 16])
def test_checked_append_outside_the_pool(block):
    AP.test_pages_outside_the_pool_are_not_written(block)
    _clean("append outside the pool")


@pytest.mark.parametrize("case", K8.CASES, ids=lambda c: "_".join(map(str, c[:10])))
def test_checked_kv8(case):
    K8.test_matches_the_definition(case)
    _clean(f"e4m3 cache {case}")


def test_checked_kv8_outside_the_pool():
    K8.test_pages_outside_the_pool_read_as_zeros()
    _clean("e4m3 cache, pages outside the pool")
