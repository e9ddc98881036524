"""Workspace sizes of the cross entropy over the range of its sizes, on the host."""
import ctypes

import pytest

import mxfp8_block_scaled_03_gb300 as mx
from tests.test_objective_abi import OK_PTR, WORKSPACE, lib  # noqa: F401  (lib: a fixture)

SIZES = (mx.linear_cross_entropy_workspace_size, mx.linear_cross_entropy_bwd_workspace_size)


@pytest.mark.parametrize("H,V", [(8, 1), (512, 1000), (4096, 128256), (1 << 20, 1 << 20)])
@pytest.mark.parametrize("T", [0, 1, 16, 17, 64, 65, 128, 1024, 1025, 40000])
def test_every_batch_has_a_size(lib, T, H, V):  # noqa: F811
    """An empty batch among them: its backward zeroes dw."""
    assert all(size(T, H, V) >= 256 for size in SIZES)


def test_an_empty_batch_s_backward_asks_for_its_workspace(lib):  # noqa: F811
    f = lib.linear_cross_entropy_bwd
    args = [OK_PTR, None, OK_PTR, OK_PTR, OK_PTR, 0, OK_PTR, 0, 512, 1000, OK_PTR, OK_PTR, OK_PTR, 100, None]
    assert f(*args) == WORKSPACE
    args[12] = ctypes.c_void_p((1 << 20) + 16)
    assert f(*args) == WORKSPACE
