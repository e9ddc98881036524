"""The bars on the decode-time operators' precision, on a CPU model of their arithmetic: the whole sum of pieces
or digits meets them, one piece or digit less does not."""
import numpy as np
import pytest

from tests import _decode_model as M

LINEAR = [(1, 512, 256), (5, 1408, 384)]
LAYERS = [(3, 128, 384), (2, 256, 1408)]
WHOLE = {"mxfp8": (2, 3), "nvfp4": (5, 5)}     # pieces of x and of h


@pytest.mark.parametrize("fmt", ["mxfp8", "nvfp4"])
@pytest.mark.parametrize("T,K,N", LINEAR)
def test_linear_bar(fmt, T, K, N):
    x, w, a, b = M.linear_case(fmt, T, K, N, seed=K)
    ref = x @ w.T
    bar = M.linear_bar(fmt, x, ref, a, b)
    assert (np.abs(M.linear_model(fmt, x, w) - ref) <= bar).all()
    for n in range(1, WHOLE[fmt][0]):
        off = np.abs(M.linear_model(fmt, x, w, pieces=n) - ref) > bar
        assert off.any(1).all(), f"{n} pieces pass in a row"


@pytest.mark.parametrize("fmt", ["mxfp8", "nvfp4"])
@pytest.mark.parametrize("E,H,F", LAYERS)
def test_layer_bar(fmt, E, H, F):
    _, _, _, w2, h, a, b = M.layer_case(fmt, E, H, F, seed=F)
    ref = np.einsum("ehf,ef->eh", w2, h)
    bar = M.layer_bar(fmt, h, ref, a, b)
    assert (np.abs(M.layer_model(fmt, h, w2) - ref) <= bar).all()
    planted = [dict(pieces=n) for n in range(1, WHOLE[fmt][1])] + ([dict(plain=True)] if fmt == "mxfp8" else [])
    for lost in planted:
        off = np.abs(M.layer_model(fmt, h, w2, **lost) - ref) > bar
        assert off.any(1).all(), f"{lost} passes for a token"


@pytest.mark.parametrize("fmt", ["mxfp8", "nvfp4"])
def test_norm_bar(fmt):
    """On ordinary random weights: the sum of pieces meets the bar on the error's norm, h in 4 bits does not."""
    rng = np.random.default_rng(1)
    h = rng.standard_normal((16, 640)) * rng.standard_normal((16, 640))
    w = 0.02 * rng.standard_normal((512, 640))
    ref = h @ w.T
    assert M.error_norm(M.bf16(M.represent(h, fmt, True) @ w.T), ref) <= M.NORM_BAR
    lost = dict(plain=True) if fmt == "mxfp8" else dict(pieces=2)
    assert M.error_norm(M.bf16(M.represent(h, fmt, True, **lost) @ w.T), ref) > 2 * M.NORM_BAR


def test_inputs_are_exact_in_both_formats():
    for fmt in ("mxfp8", "nvfp4"):
        x, _, w1, _, _, _, _ = M.layer_case(fmt, 2, 256, 128, seed=3)
        assert (M.represent(x, fmt, False) == x).all() and (M.bf16(w1) == w1).all()
        assert (np.abs(w1).reshape(-1, 16).max(1) == 6.0 / 32.0).all()
