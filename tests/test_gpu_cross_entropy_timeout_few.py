"""Waits that run out in the few rows' kernel with two CTAs per SM, forward (up to 32 rows) and backward: as in
test_gpu_cross_entropy_timeout, whose rows of this kind reach it in the backward only."""
import pytest

from tests import test_gpu_cross_entropy_timeout as W

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 5, 17, 32])
def test_waits_of_few_rows_that_run_out_are_reported(T):
    W.test_waits_that_run_out_are_reported(T, 16384, 20000)
