"""Oracle for the norms around the layer (numpy).

TEST INFRASTRUCTURE ONLY, like the rest of this package.

The pages stop at the layer; the readings taken are the two norms that
models use around it: by the root mean square of a row, and about its mean
with its (biased) variance.
"""
from __future__ import annotations

import numpy as np

from .moe import _f64, _i64


def norm(x, kind, weight=None, bias=None, offset=0.0, eps=1e-6):
    """Rows of x normalised ("rms" or "layer"), times offset + weight, plus bias; "" returns x."""
    x = _f64(x)
    if kind == "":
        return x
    m = x.mean(axis=1, keepdims=True) if kind == "layer" else 0.0
    var = np.square(x - m).mean(axis=1, keepdims=True)
    y = (x - m) / np.sqrt(var + eps)
    if weight is not None:
        y = y * (offset + _f64(weight))
    return y if bias is None else y + _f64(bias)


def block_rows(y_perm, pair_to_sorted, topk_w, k_max, y_shared=None):
    """The combine's rows, not rounded: y_shared + sum of each token's weighted sorted rows."""
    y = _f64(y_perm)
    if pair_to_sorted is None:
        out = y.copy()
    else:
        q, w = _i64(pair_to_sorted).reshape(-1, k_max), _f64(topk_w)
        out = np.zeros((q.shape[0], y.shape[1]))
        for t in range(q.shape[0]):
            for j in range(k_max):
                if q[t, j] >= 0:
                    out[t] += w[t, j] * y[q[t, j]]
    return out if y_shared is None else out + _f64(y_shared)


def combine_norm(y_perm, pair_to_sorted, topk_w, k_max, y_shared=None, post="", post_weight=None, post_bias=None,
                 gate=None, block_scale=1.0, residual=None, residual_scale=1.0, next="", next_weight=None, next_bias=None,
                 offset=0.0, eps=1e-6):
    """(out, next_out): the block's rows, the norm after them, gate, residual, and the next norm of out."""
    u = norm(block_rows(y_perm, pair_to_sorted, topk_w, k_max, y_shared), post, post_weight, post_bias, offset, eps)
    if gate is not None:
        u = u * _f64(gate)
    o = block_scale * u
    if residual is not None:
        o = o + residual_scale * _f64(residual)
    return o, (norm(o, next, next_weight, next_bias, offset, eps) if next else None)
