"""The checked build (what the kernels decode and index compared with its
bounds) runs the cases of the operators of latent attention, each against its
definition as in its own test file, with the status word read after every
case: no check may fire on valid inputs."""
import pytest

from attention_forward_14_gb300 import binding

import test_latent_append as A
import test_latent_expanded as E
import test_latent_paged as P
import test_latent_together as T
from test_checked_ops_gpu import checked_library  # noqa: F401

pytestmark = pytest.mark.gpu


def _clean(what):
    code = binding.status()
    assert code[0] == 0, f"{what}: status {code}"


@pytest.mark.parametrize("case", A.CASES, ids=str)
def test_checked_append(case):
    A.test_append(case)
    _clean(f"append {case}")


@pytest.mark.parametrize("case", P.CASES, ids=str)
def test_checked_cache(case):
    P.test_matches_the_definition(case)
    _clean(f"cache {case}")


@pytest.mark.parametrize("case", E.CASES, ids=lambda c: str(c)[:60])
def test_checked_expanded(case):
    E.test_forward_and_gradients(case)
    _clean(f"expanded {case}")


def test_checked_server():
    T.test_a_server()
    _clean("server")


def test_checked_outside():
    P.test_pages_outside_the_pool_read_as_zeros()
    A.test_pages_outside_the_pool_are_not_written()
    E.test_sequences_outside_the_totals_are_left()
    _clean("outside")
