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


def grid():
    sizes = [(T, H, V) for T in (65, 200, 512, 1000, 1024, 1025, 1531, 2048, 4096, 8192, 16384, 65536)
             for H in (64, 256, 1024, 2048, 4096, 8192) for V in (1000, 3600, 16384, 32000, 50257, 128256, 262144)]
    return sizes + [(8192, 4096, 64000), (4096, 4096, 256000), (100, 512, 1 << 22)]


def test_the_backward_s_workspace_over_the_range(lib):  # noqa: F811
    """With rows padded to 256: the rows that take part (2 bytes per element of x), dz of at most half the logits in bf16 (64 to
    256 MB; pieces of 2048 entries at the least, and rounded up to 256), dx or parts of it in fp32 (a quarter of the logits, 32 to
    64 MB, or 4 bytes per element of dx), parts of dw of at most 152 tiles of 64 KB."""
    size = mx.linear_cross_entropy_bwd_workspace_size
    for T, H, V in grid():
        pad = (T + 255) // 256 * 256
        logits = 2 * pad * V
        dz = max(min(max(logits // 2, 1 << 26), 1 << 28), 2 * 2048 * pad) + 2 * 256 * pad
        parts = max(min(max(logits // 4, 1 << 25), 1 << 26), 4 * T * H)
        assert size(T, H, V) <= 2 * pad * H + dz + parts + 152 * 65536 + 8 * pad + (1 << 16), (T, H, V)


@pytest.mark.parametrize("T,H,V", [(8192, 4096, 32000), (4096, 4096, 32000), (4096, 4096, 128256), (16384, 1024, 16384),
                                   (2048, 4096, 32000), (1531, 2048, 50257), (512, 4096, 128256), (1024, 4096, 128256),
                                   (65536, 4096, 128256)])
def test_the_backward_takes_less_memory_than_the_logits(lib, T, H, V):  # noqa: F811
    assert mx.linear_cross_entropy_bwd_workspace_size(T, H, V) < 0.9 * 2 * T * V
