"""Host-side argument checks and sizes of the router's and the cross entropy's calls: every bad call returns its status
before anything touches a GPU."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    from mxfp8_block_scaled_03_gb300 import build_ext
    build_ext.build()
    import mxfp8_block_scaled_03_gb300 as mx
    return mx.lib()


P = ctypes.c_void_p
OK_PTR = P(1 << 20)            # never dereferenced: every call below fails its host checks first
ODD = P((1 << 20) + 1)
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


def bad(args, **changes):
    a = list(args)
    for i, v in changes.items():
        a[int(i[1:])] = v
    return a


def test_route_forward_refusals(lib):
    f = lib.moe_route_fwd
    #        0 logits 1 dt 2 T    3 E 4 k 5 mask 6 norm 7 spread 8 experts.. 13 losses 14 workspace 15 bytes 16 stream
    args = [OK_PTR, 1, 100000, 64, 8, None, 1, 0, *[OK_PTR] * 6, OK_PTR, 1 << 40, None]
    assert f(*bad(args, a1=2)) == INVALID
    assert f(*bad(args, a2=-1)) == INVALID
    assert f(*bad(args, a2=1 << 29)) == INVALID               # T * k past 31 bits
    assert f(*bad(args, a3=0)) == INVALID
    assert f(*bad(args, a3=1025)) == INVALID
    assert f(*bad(args, a4=0)) == INVALID
    assert f(*bad(args, a4=65)) == INVALID                    # more choices than experts
    assert f(*bad(args, a4=33)) == UNSUPPORTED
    assert f(*bad(args, a6=2)) == INVALID
    assert f(*bad(args, a7=-1)) == INVALID
    assert f(*bad(args, a0=None)) == INVALID
    assert f(*bad(args, a0=P((1 << 20) + 2))) == INVALID      # float logits at half a float
    assert f(*bad(args, a0=ODD, a1=0)) == INVALID
    for i in range(8, 14):
        assert f(*bad(args, **{f"a{i}": None})) == INVALID
        assert f(*bad(args, **{f"a{i}": ODD})) == INVALID
    assert f(*bad(args, a14=None)) == INVALID
    assert f(*bad(args, a14=P((1 << 20) + 8))) == INVALID
    assert f(*bad(args, a15=1000)) == WORKSPACE
    size = lib.moe_route_workspace_size
    assert size(100000, 64, 8) > 1000 and size(-1, 64, 8) == 0 and size(4, 64, 33) == 0 and size(4, 4, 5) == 0
    assert size(0, 1, 1) > 0


def test_route_backward_refusals(lib):
    f = lib.moe_route_bwd
    #        0 logits 1 dt 2 T 3 E 4 k 5 experts 6 gates 7 lse 8 counts 9 dgates 10 rows 11 dprob 12 dlosses 13 norm 14 out
    args = [OK_PTR, 1, 100, 64, 8, *[OK_PTR] * 4, OK_PTR, OK_PTR, OK_PTR, OK_PTR, 1, OK_PTR, None]
    assert f(*bad(args, a1=-1)) == INVALID
    assert f(*bad(args, a2=-1)) == INVALID
    assert f(*bad(args, a3=1025)) == INVALID
    assert f(*bad(args, a4=65)) == INVALID
    assert f(*bad(args, a4=40)) == UNSUPPORTED
    assert f(*bad(args, a13=2)) == INVALID
    assert f(*bad(args, a9=None)) == INVALID                  # rows of gradients that are not there
    for i in (0, 5, 6, 7, 8, 14):
        assert f(*bad(args, **{f"a{i}": None})) == INVALID
        assert f(*bad(args, **{f"a{i}": ODD})) == INVALID
    for i in (9, 10, 11, 12):
        assert f(*bad(args, **{f"a{i}": ODD})) == INVALID
    assert f(*bad(args, a2=0, a0=None, a14=None)) == 0        # no tokens


def test_cross_entropy_forward_refusals(lib):
    f = lib.linear_cross_entropy_fwd
    #        0 x     1 w     2 targets 3 wide 4 T 5 H 6 V 7 loss 8 lse 9 workspace 10 bytes 11 stream
    args = [OK_PTR, OK_PTR, OK_PTR, 0, 100, 512, 1000, OK_PTR, OK_PTR, OK_PTR, 1 << 40, None]
    assert f(*bad(args, a3=2)) == INVALID
    assert f(*bad(args, a4=-1)) == INVALID
    assert f(*bad(args, a5=0)) == INVALID
    assert f(*bad(args, a6=0)) == INVALID
    assert f(*bad(args, a5=516)) == UNSUPPORTED
    assert f(*bad(args, a4=(1 << 24) + 1)) == UNSUPPORTED
    assert f(*bad(args, a5=(1 << 20) + 8)) == UNSUPPORTED
    assert f(*bad(args, a6=(1 << 28) + 1)) == UNSUPPORTED
    assert f(*bad(args, a4=1 << 24, a6=1 << 28)) == UNSUPPORTED
    for i in (0, 1, 2, 7, 8):
        assert f(*bad(args, **{f"a{i}": None})) == INVALID
        assert f(*bad(args, **{f"a{i}": ODD})) == INVALID
    for i in (0, 1):
        assert f(*bad(args, **{f"a{i}": P((1 << 20) + 8)})) == INVALID
    assert f(*bad(args, a3=1, a2=P((1 << 20) + 4))) == INVALID    # int64 targets at half of one
    assert f(*bad(args, a9=None)) == INVALID
    assert f(*bad(args, a9=P((1 << 20) + 16))) == WORKSPACE
    assert f(*bad(args, a10=1000)) == WORKSPACE
    size = lib.linear_cross_entropy_workspace_size
    assert size(100, 512, 1000) > 1000 and size(100, 516, 1000) == 0 and size(-1, 512, 1000) == 0 and size(1, 8, 0) == 0
    assert size(0, 512, 1000) > 0


def test_cross_entropy_backward_refusals(lib):
    f = lib.linear_cross_entropy_bwd
    #        0 dloss 1 dlse  2 x     3 w     4 targets 5 wide 6 lse 7 T 8 H 9 V 10 dx  11 dw   12 ws   13 bytes 14 stream
    args = [OK_PTR, OK_PTR, OK_PTR, OK_PTR, OK_PTR, 0, OK_PTR, 100, 512, 1000, OK_PTR, OK_PTR, OK_PTR, 1 << 40, None]
    assert f(*bad(args, a5=-1)) == INVALID
    assert f(*bad(args, a7=-1)) == INVALID
    assert f(*bad(args, a8=0)) == INVALID
    assert f(*bad(args, a9=-5)) == INVALID
    assert f(*bad(args, a8=1001)) == UNSUPPORTED
    assert f(*bad(args, a9=(1 << 28) + 1)) == UNSUPPORTED
    for i in (0, 2, 3, 4, 6, 10, 11):
        assert f(*bad(args, **{f"a{i}": None})) == INVALID
        assert f(*bad(args, **{f"a{i}": ODD})) == INVALID
    for i in (2, 3, 10, 11):
        assert f(*bad(args, **{f"a{i}": P((1 << 20) + 8)})) == INVALID
    assert f(*bad(args, a1=ODD)) == INVALID
    assert f(*bad(args, a12=None)) == INVALID
    assert f(*bad(args, a12=P((1 << 20) + 128))) == WORKSPACE
    assert f(*bad(args, a13=4096)) == WORKSPACE
    size = lib.linear_cross_entropy_bwd_workspace_size
    assert size(100, 512, 1000) > 4096 and size(100, 512, 0) == 0 and size(1, 12, 4) == 0


def test_the_backward_s_workspace_is_bounded_by_pieces(lib):
    """dz never has more than 2^28 entries, whatever the vocabulary; x and the parts of dx come beside it."""
    size = lib.linear_cross_entropy_bwd_workspace_size
    T, H = 8192, 4096
    rows = T * H * (2 + 4)
    assert size(T, H, 64000) <= 2 * (1 << 28) + rows + (1 << 20)
    assert size(T, H, 256000) <= 2 * (1 << 28) + rows + (1 << 20) < T * 256000 * 2
