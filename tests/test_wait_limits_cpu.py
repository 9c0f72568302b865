"""Limits of the kernels' waits that are refused, on the host."""
from __future__ import annotations

import pytest

from combine_moe_get_gb300 import binding as moe


@pytest.fixture(autouse=True)
def as_it_was():
    yield
    assert moe.LIB.moe_test_wait_limits(0, -1) == moe.MOE_OK


@pytest.mark.parametrize("ns", [1, 1000, 999_999])
def test_a_limit_that_copies_outlast_is_refused(ns):
    with pytest.raises(moe.MoeError) as e, moe.test_wait_limits(ns):
        pass
    assert e.value.code == moe.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("ns", [-1, 0, 1_000_000, 2 ** 40])
def test_other_limits_are_taken(ns):
    with moe.test_wait_limits(ns):
        pass
