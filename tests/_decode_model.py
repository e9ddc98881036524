"""Inputs, bars and a CPU model of the decode-time operators' arithmetic, for the tests of its precision (test code).

The inputs are made so that a result shows the bits of one activation.  A row of the (second) weight matrix holds +1
and -1, both exact in either format, at two positions whose activations are next to each other in size: the result is
their difference, and its rounding to bf16 no longer covers what the activations lose.  In the layer, x and W1 are such
that the gate and up sums are exact in 32 bits, so that all the error is h's.

Bars, per element, for a result r = a - b with block maxima A and B of a's and b's blocks:
    half a bf16 step of r (at most 2^-8 |r|; 1.01 for the step of the rounded value), and
    linear: delta (A + B), delta = 2^-17 beside MXFP8, 2^-14 beside NVFP4 weights, + 2^-20 (|a| + |b|) for 32-bit sums,
    layer:  delta (A + B), delta = 2^-12 beside MXFP8, 2^-14 beside NVFP4 weights, + 2^-19 (|a| + |b|) for those and for
            silu in 32 bits (a few roundings of 2^-24 and two functions of 2 ulp).

Bar on the norm of a whole result's error: 2^-7 / sqrt(12) = 0.00226 of the result's norm is the rounding to bf16 if all
significands were 1 (a step of 2^-7, errors even over it), its most; 2^-12 more for the activations.

The model writes activations as the operators do: MXFP8 pieces of 4 significant bits (the last rounded to nearest) in
E4M3 under a block scale, NVFP4 digits -4..4 in base 8.  `pieces` leaves the last ones out, which the bars have to
notice; `plain` is a single E4M3 (4 bits, rounded) instead.
"""
import numpy as np

NORM_BAR = 2.0 ** -7 / np.sqrt(12.0) + 2.0 ** -12
BLOCK = {"mxfp8": 32, "nvfp4": 16}


def bf16(v):
    """Nearest bf16 value, ties to even (normal range)."""
    m, e = np.frexp(np.asarray(v, dtype=np.float64))
    return np.ldexp(np.rint(m * 256.0), e - 8)


def e4m3(v):
    """Nearest E4M3 value of |v| < 464."""
    _, e = np.frexp(v)
    q = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)
    return np.rint(v / q) * q


def block_max(v, block):
    return np.repeat(np.abs(v).reshape(v.shape[:-1] + (-1, block)).max(-1), block, axis=-1)


def floor_log2(v):
    return np.frexp(np.where(v > 0, v, 1.0))[1] - 1


def represent(v, fmt, of_h, pieces=None, plain=False):
    """What the activations v [.., K] become.  All blocks here are within 2^17 of their row's largest."""
    b = block_max(v, BLOCK[fmt])
    e = floor_log2(b)
    out = np.zeros_like(v)
    if fmt == "mxfp8":
        n = 3 if of_h else 2
        r = np.ldexp(v, 7 - e)
        if plain:
            return np.ldexp(e4m3(r), e - 7)
        for i in range(n):
            m, x = np.frexp(r)
            top = r if i == n - 1 else np.ldexp(np.trunc(m * 16.0), x - 4)
            if pieces is None or i < pieces:
                out += np.ldexp(e4m3(top), e - 7 - 4 * i)
            r = (r - top) * 16.0
    else:
        r = np.ldexp(v, 1 - e)
        for i in range(5):
            d = np.rint(r)
            if pieces is None or i < pieces:
                out += np.ldexp(d, e - 1 - 3 * i)
            r = (r - d) * 8.0
    return out


def neighbours(v, n):
    """n pairs of positions of v [K] next to each other in value, spread over the range of values."""
    order = np.argsort(v, kind="stable")
    at = np.unique(np.linspace(0, len(v) - 2, n).astype(int))
    at = np.resize(at, n)
    return order[at], order[at + 1]


def pair_rows(N, K, a, b):
    w = np.zeros((N, K))
    w[np.arange(N), a] = 1.0
    w[np.arange(N), b] = -1.0
    return w


# ---- a linear ----
def linear_case(fmt, T, K, N, seed):
    """x [T, K] (bf16 values, magnitudes over ten binades), w [N, K]; the rows' powers of two differ, so that
    every row's neighbours are the first row's."""
    rng = np.random.default_rng(seed)
    x = bf16(np.exp2(rng.uniform(-10.0, 0.0, K)) * rng.choice([-1.0, 1.0], K))
    x = np.stack([np.ldexp(x, (7 * t) % 23 - 11) for t in range(T)])
    a, b = neighbours(x[0], N)
    return x, pair_rows(N, K, a, b), a, b


def linear_bar(fmt, x, ref, a, b):
    m = block_max(x, BLOCK[fmt])
    delta = 2.0 ** (-17 if fmt == "mxfp8" else -14)
    return 1.01 * 2.0 ** -8 * np.abs(ref) + delta * (m[:, a] + m[:, b]) + 2.0 ** -20 * (np.abs(x[:, a]) + np.abs(x[:, b]))


def linear_model(fmt, x, w, **lost):
    return bf16(represent(x, fmt, False, **lost) @ w.T)


# ---- a layer: token t goes to expert t % E alone, whose W2 is made for its h ----
GRID = np.array([0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def layer_case(fmt, E, H, F, seed):
    """x [E, H], gates [E], w1 [E, 2, F, H], w2 [E, H, F], h [E, F] in 64 bits, pairs a, b [E, H].  x is +-(1 + j/4) and
    w1 a 4-bit number over 2^5 with 6 in every block of 16: exact in either format, and their sums in 32 bits."""
    rng = np.random.default_rng(seed)
    x = rng.choice([-1.0, 1.0], (E, H)) * (1.0 + rng.integers(0, 4, (E, H)) / 4.0)
    w1 = rng.choice([-1.0, 1.0], (E, 2, F, H)) * rng.choice(GRID, (E, 2, F, H))
    w1[..., ::16] = 6.0 * np.sign(w1[..., ::16])
    w1 /= 32.0
    gates = 0.5 + rng.random(E, dtype=np.float32).astype(np.float64)
    g, u = (np.einsum("efh,eh->ef", w1[:, i], x) for i in range(2))
    h = gates[:, None] * g / (1.0 + np.exp(-g)) * u
    pairs = [neighbours(h[e], H) for e in range(E)]
    w2 = np.stack([pair_rows(H, F, *p) for p in pairs])
    return x, gates, w1, w2, h, np.stack([p[0] for p in pairs]), np.stack([p[1] for p in pairs])


def layer_bar(fmt, h, ref, a, b):
    m = block_max(h, BLOCK[fmt])

    def at(v, i):
        return np.take_along_axis(v, i, 1)
    delta = 2.0 ** (-12 if fmt == "mxfp8" else -14)
    return (1.01 * 2.0 ** -8 * np.abs(ref) + delta * (at(m, a) + at(m, b)) +
            2.0 ** -19 * (np.abs(at(h, a)) + np.abs(at(h, b))))


def layer_model(fmt, h, w2, **lost):
    return bf16(np.einsum("ehf,ef->eh", w2, represent(h, fmt, True, **lost)))


def error_norm(y, ref):
    return float(np.linalg.norm(y - ref) / np.linalg.norm(ref))
