"""Host-side argument checks and sizes of the decode-time operators and of the junction norms: every bad
call returns its status before anything touches a GPU."""
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
ODD = P((1 << 20) + 2)
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


def bad(args, **changes):
    a = list(args)
    for i, v in changes.items():
        a[int(i[1:])] = v
    return a


@pytest.mark.parametrize("nv", [False, True])
def test_moe_decode_refusals(lib, nv):
    f = lib.nvfp4_moe_decode_fwd if nv else lib.moe_decode_fwd
    w = [OK_PTR] * (6 if nv else 4)
    #        0 x     1 T 2 H  3 F  4 E 5 k 6 experts 7 gates    8.. weights   out     ws      bytes    stream
    args = [OK_PTR, 4, 256, 384, 8, 2, OK_PTR, OK_PTR, *w, OK_PTR, OK_PTR, 1 << 40, None]
    out, ws, nbytes = 8 + len(w), 9 + len(w), 10 + len(w)
    assert f(*bad(args, a1=-1)) == INVALID
    assert f(*bad(args, a4=0)) == INVALID
    assert f(*bad(args, a4=1025)) == INVALID
    assert f(*bad(args, a5=0)) == INVALID
    assert f(*bad(args, a2=0)) == INVALID
    assert f(*bad(args, a1=65)) == UNSUPPORTED
    assert f(*bad(args, a5=33)) == UNSUPPORTED
    assert f(*bad(args, a2=200)) == UNSUPPORTED
    assert f(*bad(args, a3=100)) == UNSUPPORTED
    assert f(*bad(args, a4=1024, a3=1 << 21)) == UNSUPPORTED     # E * 2F past 32 bits
    assert f(*bad(args, a0=None)) == INVALID
    assert f(*bad(args, a0=ODD)) == INVALID
    assert f(*bad(args, a6=None)) == INVALID
    assert f(*bad(args, a6=P((1 << 20) + 1))) == INVALID
    assert f(*bad(args, a7=ODD)) == INVALID
    for i in range(8, 8 + len(w)):
        assert f(*bad(args, **{f"a{i}": None})) == INVALID
    assert f(*bad(args, **{f"a{out}": None})) == INVALID
    assert f(*bad(args, **{f"a{ws}": None})) == INVALID
    assert f(*bad(args, **{f"a{ws}": P((1 << 20) + 16)})) == WORKSPACE
    assert f(*bad(args, **{f"a{nbytes}": 100})) == WORKSPACE
    need = lib.moe_decode_workspace_size(4, 2, 256, 384, 8)
    assert need > 0 and f(*bad(args, **{f"a{nbytes}": 1024})) == WORKSPACE


def test_moe_decode_workspace_size(lib):
    size = lib.moe_decode_workspace_size
    assert size(65, 2, 256, 384, 8) == 0 and size(4, 33, 256, 384, 8) == 0 and size(-1, 2, 256, 384, 8) == 0
    assert size(0, 2, 256, 384, 8) > 0
    assert size(64, 8, 2048, 1408, 64) > size(1, 8, 2048, 1408, 64)


@pytest.mark.parametrize("nv", [False, True])
def test_matvec_refusals(lib, nv):
    f = lib.nvfp4_matvec if nv else lib.mxfp8_matvec
    w = [OK_PTR] * (3 if nv else 2)
    #        0 x     1 T 2 K  3 N   4.. weight  y       ws      bytes    stream
    args = [OK_PTR, 3, 512, 256, *w, OK_PTR, OK_PTR, 1 << 40, None]
    y, ws, nbytes = 4 + len(w), 5 + len(w), 6 + len(w)
    assert f(*bad(args, a1=-1)) == INVALID
    assert f(*bad(args, a2=0)) == INVALID
    assert f(*bad(args, a3=-128)) == INVALID
    assert f(*bad(args, a1=65)) == UNSUPPORTED
    assert f(*bad(args, a2=500)) == UNSUPPORTED
    assert f(*bad(args, a3=200)) == UNSUPPORTED
    for i in [0, *range(4, 4 + len(w)), y]:
        assert f(*bad(args, **{f"a{i}": None})) == INVALID
    assert f(*bad(args, a0=ODD)) == INVALID
    assert f(*bad(args, **{f"a{ws}": None})) == INVALID
    assert f(*bad(args, **{f"a{ws}": P((1 << 20) + 64)})) == WORKSPACE
    assert f(*bad(args, **{f"a{nbytes}": 255})) == WORKSPACE
    assert lib.matvec_workspace_size(65, 512) == 0 and lib.matvec_workspace_size(64, 0) == 0
    assert lib.matvec_workspace_size(64, 16384) >= lib.matvec_workspace_size(1, 128) > 0


def test_residual_norm_refusals(lib):
    f = lib.residual_norm_fwd
    #        0 y     1 res   2 wpost 3 gate  4 wpre  5 T 6 H  7 dt 8 gk 9 pn 10 sc 11 eps 12 out 13 n    14 stats
    args = [OK_PTR, OK_PTR, OK_PTR, OK_PTR, OK_PTR, 4, 512, 0, 1, 1, 1.0, 1e-6, OK_PTR, OK_PTR, OK_PTR, None]
    assert f(*bad(args, a5=-1)) == INVALID
    assert f(*bad(args, a6=0)) == INVALID
    assert f(*bad(args, a7=2)) == INVALID
    assert f(*bad(args, a8=3)) == INVALID
    assert f(*bad(args, a9=2)) == INVALID
    assert f(*bad(args, a11=-1.0)) == INVALID
    assert f(*bad(args, a11=float("nan"))) == INVALID
    assert f(*bad(args, a3=None)) == INVALID              # a gate kind without a gate
    assert f(*bad(args, a8=0)) == INVALID                 # a gate without a kind
    assert f(*bad(args, a9=0)) == INVALID                 # a post-norm weight without the post-norm
    assert f(*bad(args, a6=516)) == UNSUPPORTED
    assert f(*bad(args, a6=8200)) == UNSUPPORTED
    for i in (0, 1, 12, 13):
        assert f(*bad(args, **{f"a{i}": None})) == INVALID
        assert f(*bad(args, **{f"a{i}": P((1 << 20) + 8)})) == INVALID
    for i in (2, 3, 4):
        assert f(*bad(args, **{f"a{i}": P((1 << 20) + 4)})) == INVALID
    assert f(*bad(args, a14=None)) == INVALID
    assert f(*bad(args, a5=0, a0=None, a1=None)) == 0     # no rows

    g = lib.residual_norm_bwd
    #        0 dn    1 dro   2 y     3 ro    4 stats 5 wpost 6 gate  7 wpre  8 T 9 H 10 dt 11 gk 12 pn 13 sc
    args = [OK_PTR] * 8 + [4, 512, 0, 1, 1, 1.0] + [OK_PTR] * 6 + [1 << 40, None]
    #        14 dy 15 dres 16 dwpost 17 dgate 18 dwpre 19 workspace 20 bytes
    assert g(*bad(args, a8=-1)) == INVALID
    assert g(*bad(args, a11=2, a6=None)) == INVALID
    assert g(*bad(args, a5=None)) == INVALID              # the gradient of a weight that is not there
    assert g(*bad(args, a7=None)) == INVALID
    assert g(*bad(args, a12=0)) == INVALID
    assert g(*bad(args, a9=8200)) == UNSUPPORTED
    for i in (0, 2, 3, 14, 15):
        assert g(*bad(args, **{f"a{i}": None})) == INVALID
    assert g(*bad(args, a1=ODD)) == INVALID
    assert g(*bad(args, a4=None)) == INVALID
    assert lib.residual_norm_bwd_workspace_size(-1, 512) == 0
    assert lib.residual_norm_bwd_workspace_size(4, 8200) == 0
    assert lib.residual_norm_bwd_workspace_size(100, 512) > 0
