"""Oracle for the expert choice by score (numpy, float64).

TEST INFRASTRUCTURE ONLY, like the rest of this package.
"""
from __future__ import annotations

import numpy as np

from .moe import _f64, _i64, round_to


def scores(logits, score: str) -> np.ndarray:
    """sigmoid(l), or the softmax of l over the experts."""
    l = _f64(logits)
    if score == "sigmoid":
        e = np.exp(-np.abs(l))
        return np.where(l >= 0, 1.0 / (1.0 + e), e / (1.0 + e))
    e = np.exp(l - l.max(axis=1, keepdims=True))
    return e / e.sum(axis=1, keepdims=True)


def choice_scores(logits, score: str, bias=None, n_group: int = 1, topk_group: int = 1, group_top: int = 1):
    """What experts are taken by, -inf for those that cannot be: s + bias (l without
    a bias, in the same order) within the topk_group groups whose group_top largest
    values of s + bias add up to most, the lower group first among equals."""
    l = _f64(logits)
    T, E = l.shape
    s = scores(l, score)
    c = s if bias is None else s + _f64(bias)[None, :]
    take = np.array(l if bias is None else c)
    if topk_group < n_group:
        g = np.sort(c.reshape(T, n_group, E // n_group), axis=2)[:, :, ::-1][:, :, :group_top]
        off = np.isneginf(g)
        total = np.where(off.all(axis=2), -np.inf, np.where(off, 0.0, g).sum(axis=2))
        order = np.argsort(-total, axis=1, kind="stable")[:, :topk_group]
        keep = np.zeros((T, n_group), dtype=bool)
        np.put_along_axis(keep, order, True, axis=1)
        take[~np.repeat(keep, E // n_group, axis=1)] = -np.inf
    return take


def route_select(logits, score: str, k_per_token, k_max: int, bias=None, n_group: int = 1, topk_group: int = 1,
                 group_top: int = 1, renorm: bool = True, scale: float = 1.0):
    """Experts and weights of every token.

    Slot j < k_t holds the expert of the j-th largest choice score (ties to the
    lower index); experts that cannot be taken leave padding (-1, weight 0).
    Weights: the picks' scores, over their sum if renorm, times scale (stored as fp32).
    """
    take = choice_scores(logits, score, bias, n_group, topk_group, group_top)
    k = _i64(k_per_token).reshape(take.shape[0])
    order = np.argsort(-take, axis=1, kind="stable")[:, :k_max]
    live = (np.arange(k_max)[None, :] < k[:, None]) & ~np.isneginf(np.take_along_axis(take, order, axis=1))
    w = np.where(live, np.take_along_axis(scores(logits, score), order, axis=1), 0.0)
    if renorm:
        total = w.sum(axis=1, keepdims=True)
        w = w / np.where(total > 0, total, 1.0)
    return np.where(live, order, -1), round_to(w * scale, "f32")
