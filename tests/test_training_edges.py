"""Refusals of the operators of training that need no GPU."""
import pytest

from dflash2_draft_head_gb300 import binding, build_library
from test_train_abi import P, _adamw


@pytest.fixture(scope="module")
def L():
    build_library()
    return binding.lib()


@pytest.mark.parametrize("most", [1e-60, 7e-46])
def test_a_limit_of_the_norm_that_is_0_in_fp32(L, most):
    """It would count as no limit."""
    assert _adamw(L, most=most, norm=P[12]) == 1
    assert b"max_norm" in L.dflash2_last_error()
