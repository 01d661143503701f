"""Oracle for 4-bit weights with group scales and the products on them (numpy).

TEST INFRASTRUCTURE ONLY, like the rest of this package.

Readings taken: codes 0..15 with a scale and a zero point per group of
columns, w = (code - zero) scale; without zero points the zero is 8.  The
quantiser's divisions are fp32, so that its codes are whole numbers to compare exactly.
"""
from __future__ import annotations

import numpy as np

from .moe import _f64, _i64, bf16_round, silu


def w4_encode(x, group, zeros, scale_dtype="f32"):
    """(codes [rows, K], scales [rows, K / group], zero points or None) of x [rows, K] (fp32 values)."""
    x = np.asarray(x, dtype=np.float32)
    rows, K = x.shape
    b = x.reshape(rows, K // group, group)
    finite = np.isfinite(b).all(axis=2)
    b = np.where(finite[..., None], b, 0).astype(np.float32)
    lo, hi = np.minimum(b.min(axis=2), 0), np.maximum(b.max(axis=2), 0)
    if zeros:  # sixteenths, so that the range of the largest numbers is one
        s = (hi / np.float32(16) - lo / np.float32(16)) / np.float32(15 / 16)
    else:
        s = np.maximum(hi, -lo) / np.float32(7)
    s = s.astype(np.float32)
    if scale_dtype == "bf16":
        s = bf16_round(s).astype(np.float32)
    some = s != 0
    d = np.where(some, s, 1).astype(np.float32)
    if zeros:
        z = np.where(some & finite, np.clip(np.rint(-lo / d), 0, 15), 0)
    else:
        z = np.full(s.shape, 8.0)
    q = np.clip(np.rint(b / d[..., None]) + z[..., None], 0, 15)
    q = np.where((some & finite)[..., None], q, z[..., None]).astype(np.int64)
    return q.reshape(rows, K), np.where(finite, s, np.nan), z.astype(np.int64) if zeros else None


def w4_values(codes, scales, zeros, group):
    """The values (float64) of codes [..., K] with scales and zero points [..., K / group]."""
    z = 8 if zeros is None else np.repeat(_i64(zeros), group, axis=-1)
    return (_i64(codes) - z) * np.repeat(_f64(scales), group, axis=-1)


def w4_grouped_product(x, w, expert_offsets, phys_to_expert):
    """out[q] = x[q] W_e^T for the rows of each group, e its expert; x [P, K], w [E, N, K] values."""
    x, w = _f64(x), _f64(w)
    off, pe = _i64(expert_offsets), _i64(phys_to_expert)
    out = np.zeros((x.shape[0], w.shape[1]))
    for g in range(pe.shape[0]):
        out[off[g]:off[g + 1]] = x[off[g]:off[g + 1]] @ w[pe[g]].T
    return out


def w4_grouped_ffn(x, w13, w2, expert_offsets, phys_to_expert):
    """SwiGLU experts on values x [P, H], w13 [E, 2I, H], w2 [E, H, I]; not rounded on the way."""
    I = _f64(w2).shape[2]
    gu = w4_grouped_product(x, w13, expert_offsets, phys_to_expert)
    return w4_grouped_product(silu(gu[:, :I]) * gu[:, I:], w2, expert_offsets, phys_to_expert)
