"""Pins of the expert-choice and 4-bit oracles (CPU only): hand-worked examples,
brute force, and special cases that reduce to the plain router."""
import math

import numpy as np
import pytest

import oracle


def test_select_without_bias_or_groups_is_the_plain_router():
    rng = np.random.default_rng(0)
    l = rng.standard_normal((200, 16)).astype(np.float32)
    k = rng.integers(1, 6, size=200)
    idx, w = oracle.route_select(l, "softmax", k, 5)
    idx0, w0 = oracle.topk_route(l, k, 5)
    np.testing.assert_array_equal(idx, idx0)
    np.testing.assert_allclose(w, w0, rtol=1e-6)
    np.testing.assert_array_equal(oracle.route_select(l, "sigmoid", k, 5)[0], idx0)


def test_select_hand_example():
    """Sigmoid scores .5 .8 .2 .9 | .6 .6 .1 .95 in two groups, one kept by its two best."""
    s = np.array([[0.5, 0.8, 0.2, 0.9, 0.6, 0.6, 0.1, 0.95]])
    l = np.log(s / (1 - s))
    # groups: .8 + .9 = 1.7 against .6 + .95 = 1.55
    idx, w = oracle.route_select(l, "sigmoid", [3], 3, None, 2, 1, 2, True, 2.0)
    assert idx.tolist() == [[3, 1, 0]]
    np.testing.assert_allclose(w, [[1.8 / 2.2, 1.6 / 2.2, 1.0 / 2.2]], rtol=1e-6)
    # by their best alone the second group stays; its two equal experts come in index order
    assert oracle.route_select(l, "sigmoid", [3], 3, None, 2, 1, 1)[0].tolist() == [[7, 4, 5]]
    # the bias chooses but does not weigh; -inf switches off
    b = np.array([0, 0, 0.75, -np.inf, 0, 0, 0, 0])
    idx, w = oracle.route_select(l, "sigmoid", [2], 2, b, 2, 1, 2, False)
    assert idx.tolist() == [[2, 1]]
    np.testing.assert_allclose(w, [[0.2, 0.8]], rtol=1e-6)
    b = np.full(8, -np.inf)
    b[6] = 0
    idx, w = oracle.route_select(l, "sigmoid", [2], 2, b, 2, 2, 2)
    assert idx.tolist() == [[6, -1]] and w.tolist() == [[1.0, 0.0]]


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_select_brute_force(score):
    """Every rank by its definition: how many beat it."""
    rng = np.random.default_rng(5)
    E, G, keep, top = 8, 4, 2, 2
    for _ in range(60):
        l = rng.integers(-3, 4, size=E) * 0.5
        b = rng.integers(-2, 3, size=E) * 0.125
        s = [1 / (1 + math.exp(-v)) for v in l] if score == "sigmoid" else \
            [math.exp(v) / sum(math.exp(u) for u in l) for v in l]
        c = [s[e] + b[e] for e in range(E)]
        gs = [sum(sorted(c[2 * g:2 * g + 2])[-top:]) for g in range(G)]
        kept = [g for g in range(G) if sum(gs[o] > gs[g] or (gs[o] == gs[g] and o < g) for o in range(G)) < keep]
        left = [e for e in range(E) if e // 2 in kept]
        want = sorted(left, key=lambda e: (-c[e], e))[:3]
        idx, w = oracle.route_select(l[None], score, [3], 3, b, G, keep, top, True)
        near = [abs(x - y) for x in gs for y in gs if 0 < abs(x - y) < 1e-12]
        assert near or idx[0].tolist() == want
        if not near:
            np.testing.assert_allclose(w[0], [s[e] / sum(s[i] for i in want) for e in want], rtol=1e-6)


def test_mx4_hand_example():
    """A block whose largest value is 7 has scale 1: 7 saturates, midpoints go to the even code."""
    x = np.zeros((1, 32))
    x[0, :16] = [7, -6, 5, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, -0.25, 0.26, 2.49, 2.51, -5.01, 0.0, -0.0]
    code, e = oracle.mx4_encode(x)
    assert e.tolist() == [[127]]
    assert oracle.mx4_values(code, e)[0, :16].tolist() == [6, -6, 4, 4, 2, 2, 1, 1, 0, 0, 0.5, 2, 3, -6, 0, 0]
    assert code[0, :16].tolist() == [7, 15, 6, 6, 4, 4, 2, 2, 0, 8, 1, 4, 5, 15, 0, 8]


def test_mx4_scales_and_specials():
    rows = [np.zeros(32), np.full(32, 2.0 ** -149), np.full(32, np.float64(np.finfo(np.float32).max)),
            np.full(32, 4.0), np.full(32, 3.999)]
    x = np.stack(rows)
    x[0, 3] = 0.0
    code, e = oracle.mx4_encode(x)
    assert e[:, 0].tolist() == [0, 0, 252, 127, 126]
    assert (code[1] == 0).all() and (code[2] == 7).all() and (code[3] == 6).all() and (code[4] == 7).all()
    for bad in (np.nan, np.inf, -np.inf):
        x = np.ones((1, 64))
        x[0, 5] = bad
        code, e = oracle.mx4_encode(x)
        assert e[0].tolist() == [255, 125]
        v = oracle.mx4_values(code, e)
        assert np.isnan(v[0, :32]).all() and (v[0, 32:] == 1.0).all()


def test_mx4_every_grid_point_is_kept_and_error_is_bounded():
    g = np.concatenate([oracle.mx4_values(np.arange(16)[None].repeat(2, 1), np.array([[127]]))[0]])
    x = np.resize(g, (1, 32))
    x[0, 0] = 6.0
    np.testing.assert_array_equal(oracle.mx4_round(x * 2.0 ** 40), x * 2.0 ** 40)
    rng = np.random.default_rng(1)
    x = rng.standard_normal((50, 96))
    a = np.abs(x.reshape(50, 3, 32)).max(axis=2).repeat(32, 1)
    scale = 2.0 ** (np.floor(np.log2(a)) - 2)
    err = np.abs(oracle.mx4_round(x) - x)
    assert (err <= np.maximum(0.25 * scale, np.where(np.abs(x) < 6 * scale, np.abs(x) / 5 + 1e-15, np.abs(x) - 6 * scale + 1e-15))).all()


def test_mx4_grouped_ffn_is_each_rows_own_experts():
    rng = np.random.default_rng(2)
    E, H, I = 3, 64, 32
    off, pe = [0, 4, 4, 9], [2, 0, 1]
    x, w13, w2 = rng.standard_normal((9, H)), rng.standard_normal((E, 2 * I, H)), rng.standard_normal((E, H, I))
    y = oracle.mx4_grouped_ffn(x, w13, w2, off, pe, "f64")
    for q in range(9):
        e = 2 if q < 4 else 1
        g, u = w13[e, :I] @ x[q], w13[e, I:] @ x[q]
        h = oracle.mx4_round((g / (1 + np.exp(-g)) * u)[None])[0]
        np.testing.assert_allclose(y[q], w2[e] @ h, rtol=1e-12, atol=1e-12)
