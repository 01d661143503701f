"""Oracle for 4-bit microscaled values and the products on them (numpy).

TEST INFRASTRUCTURE ONLY, like the rest of this package.

The format is that of the open microscaling specification's 4-bit type: 32
values share a power-of-two scale held as a biased exponent byte, each value
is a float of one sign, two exponent and one mantissa bit.  Reading taken for
the scale: the largest magnitude's exponent less 2 (the exponent of the grid's
largest value, 6), clamped to the byte's range; values above 6 scales saturate.
"""
from __future__ import annotations

import numpy as np

from .moe import _f64, _i64, round_to, silu

#: magnitudes by the low three bits of a code
GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def mx4_encode(x):
    """(codes [rows, K], biased scale exponents [rows, K / 32]) of x [rows, K].

    Each value goes to the nearest grid point of its block's scale; a midpoint
    goes to the neighbour whose code is even.
    """
    x = _f64(x)
    rows, K = x.shape
    b = x.reshape(rows, K // 32, 32)
    finite = np.isfinite(b).all(axis=2)
    a = np.where(np.isfinite(b), np.abs(b), 0.0).max(axis=2)
    e = np.where(a > 0, np.frexp(a)[1] - 1, -1000)        # a in [2^e, 2^(e+1))
    e = np.clip(e - 2, -127, 127)
    v = np.where(np.isfinite(b), np.ldexp(np.where(np.isfinite(b), b, 0.0), -e[:, :, None]), 0.0)
    d = np.abs(np.minimum(np.abs(v), 6.0)[..., None] - GRID)  # distance to every grid point
    best = d.min(axis=-1)
    near = d == best[..., None]                            # one point, or two at a midpoint
    first = near.argmax(axis=-1)
    code = np.where(near.sum(axis=-1) == 1, first, np.where(first % 2 == 0, first, first + 1))
    code = code + 8 * np.signbit(b)
    return code.reshape(rows, K), np.where(finite, e + 127, 255)


def mx4_values(code, exponent):
    """The values (float64) of codes [rows, K] with biased exponents [rows, K / 32]."""
    c, e = _i64(code), _i64(exponent)
    v = np.where(c >= 8, -1.0, 1.0) * GRID[c % 8]
    scale = np.where(e == 255, np.nan, np.ldexp(1.0, e - 127))
    return v * np.repeat(scale, 32, axis=1)


def mx4_round(x):
    """x [rows, K] rounded to the values its 4-bit blocks stand for."""
    return mx4_values(*mx4_encode(x))


def mx4_grouped_product(a, b, expert_offsets, phys_to_expert):
    """out[q] = a[q] B_e^T for the rows of each group, e its expert; a [P, K], b [E, N, K] values."""
    a, b = _f64(a), _f64(b)
    off, pe = _i64(expert_offsets), _i64(phys_to_expert)
    out = np.zeros((a.shape[0], b.shape[1]))
    for g in range(pe.shape[0]):
        out[off[g]:off[g + 1]] = a[off[g]:off[g + 1]] @ b[pe[g]].T
    return out


def mx4_grouped_ffn(x, w13, w2, expert_offsets, phys_to_expert, dtype="bf16"):
    """SwiGLU experts on values x [P, H], w13 [E, 2I, H], w2 [E, H, I]; the activation is
    rounded to 4-bit blocks, the output stored in ``dtype``."""
    I = _f64(w2).shape[2]
    gu = mx4_grouped_product(x, w13, expert_offsets, phys_to_expert)
    h = mx4_round(silu(gu[:, :I]) * gu[:, I:])
    return round_to(mx4_grouped_product(h, w2, expert_offsets, phys_to_expert), dtype)
