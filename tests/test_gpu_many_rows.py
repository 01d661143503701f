"""More rows than fit the GPU at once: what a warp, a CTA or a ring hands on from one row, token or unit to the next.

Bounds as in test_gpu_norm (``track``) and test_gpu_w4."""
import numpy as np
import pytest
import torch

import oracle
from parity_utils import TOL, max_rel, np_
from test_gpu_norm import KIND, U, case, close, cuda, run_after, track
from test_gpu_w4 import abi, cuda as on_gpu, product, weights

pytestmark = pytest.mark.gpu
DTYPES = pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])


@DTYPES
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("H", [64, 264, 512, 1000, 1032, 2048, 4104])
def test_norm(H, kind, dtype):
    """6000 rows of different sizes: rows of a warp (one, two and four pieces a lane) and rows of a CTA."""
    T, eps = 6000, 1e-5
    if dtype == torch.float32:
        H = H // 2 + (4 if H % 16 == 8 else 0)
    rng = np.random.default_rng(H)
    x = cuda(rng.standard_normal((T, H)) * np.exp(rng.normal(0, 2, (T, 1))), dtype)
    w, b = cuda(1 + 0.3 * rng.standard_normal(H), torch.float32), cuda(rng.standard_normal(H), torch.float32)
    out = torch.full((T + 1, H), 7.0, dtype=dtype, device="cuda")
    abi().semmoe_norm(x, T, H, KIND[kind], w, b, 0.5, eps, out)
    v = np_(x).astype(np.float64)
    close(out[:T], *track(v, np.zeros_like(v), kind, w, b, 0.5, eps))
    assert bool((out[T] == 7).all())
    for lo in (0, T - 7):  # the same rows by themselves
        few = torch.empty(7, H, dtype=dtype, device="cuda")
        abi().semmoe_norm(x[lo:lo + 7], 7, H, KIND[kind], w, b, 0.5, eps, few)
        close(few, *track(v[lo:lo + 7], np.zeros((7, H)), kind, w, b, 0.5, eps))
    abi().semmoe_norm(x, T, H, KIND[kind], w, b, 0.5, eps, x)
    assert torch.equal(x, out[:T])
    assert abi().semmoe_check_errors() == 0


@DTYPES
@pytest.mark.parametrize("T,H,k,budgets,shared,post,gate,nxt", [
    (6000, 256, 8, True, False, "rms", "", "rms"), (6000, 264, 8, True, True, "rms", "channels", "rms"),
    (6000, 512, 8, True, True, "", "tokens", "layer"), (6000, 1000, 8, True, False, "layer", "tokens", ""),
    (6000, 1000, 8, False, True, "rms", "", "rms"), (5000, 2048, 8, True, False, "rms", "channels", "rms"),
    (5000, 2048, 8, True, True, "rms", "tokens", "layer"), (3000, 4104, 8, True, True, "", "tokens", "rms"),
    (6000, 264, 35, True, False, "rms", "", "rms"), (6000, 264, 1, True, False, "", "", ""),
    (6000, 264, 0, False, True, "rms", "tokens", "rms"), (6000, 2048, 0, False, False, "", "channels", "rms"),
])
def test_combine_norm(T, H, k, budgets, shared, post, gate, nxt, dtype):
    """Tokens of 0 to k slots, so that their lists of rows begin anywhere in the ring."""
    if dtype == torch.float32:
        H //= 2
    rng = np.random.default_rng(T + H + k)
    d, P = case(rng, T, H, k, dtype, budgets, shared, gate, torch.float32)
    bs, rs, eps = 0.75, 1.25, 1e-6
    out = torch.full((T + 1, H), 7.0, dtype=dtype, device="cuda")
    no = torch.full((T + 1, H), 7.0, dtype=dtype, device="cuda") if nxt else None
    run_after(d, T, H, k, P, post, nxt, 0.0, bs, rs, out, no)
    f = {key: None if t is None else np_(t).astype(np.float64) for key, t in d.items()}

    def block(y, ys):
        if not k:
            o = y.copy()
        else:
            q, w = f["q"].astype(np.int64).reshape(T, k), f["w"]
            o = np.zeros((T, H))
            for j in range(k):
                t = np.flatnonzero(q[:, j] >= 0)
                o[t] += w[t, j:j + 1] * y[q[t, j]]
        return o if ys is None else o + ys

    y = block(f["y"], f["ys"])
    size = block(np.abs(f["y"]), None if f["ys"] is None else np.abs(f["ys"]))
    u, eu = track(y, (k + 2) * U * size, post, d["pw"], d["pb"], 0.0, eps)
    if f["g"] is not None:
        u, eu = u * f["g"], (eu + U * np.abs(u)) * np.abs(f["g"])
    o = bs * u + rs * f["r"]
    eo = bs * (eu + U * np.abs(u)) + 2 * U * (np.abs(o) + np.abs(rs * f["r"]))
    close(out[:T], o, eo)
    assert bool((out[T] == 7).all())
    if nxt:
        close(no[:T], *track(o, eo, nxt, d["nw"], d["nb"], 0.0, eps))
        assert bool((no[T] == 7).all())
    again, no2 = d["r"].clone(), None if no is None else torch.empty(T, H, dtype=dtype, device="cuda")
    run_after({**d, "r": again}, T, H, k, P, post, nxt, 0.0, bs, rs, again, no2)
    assert torch.equal(again, out[:T]) and (no is None or torch.equal(no2, no[:T]))
    assert abi().semmoe_check_errors() == 0


def groups(rng, P, E):
    """Offsets of P rows in E groups of about equal size and an order of experts."""
    return np.concatenate([[0], np.cumsum(rng.multinomial(P, np.full(E, 1 / E)))]), rng.permutation(E)


@pytest.mark.parametrize("group,scale,zeros", [(128, "bf16", False), (64, "bf16", True), (32, "bf16", True), (32, "f32", False),
                                               (128, "f32", True), (96 * 4, "bf16", False)])
@pytest.mark.parametrize("per", [6, 24, 47, 64, 200])
def test_product_of_several_units_a_cta(per, group, scale, zeros):
    """64 matrices of `per` rows each, on average: units of 32, 64 and 256 rows, eleven tiles of a matrix; exact (whole numbers)."""
    E, N, K = 64, 1408, 1152 if group > 64 else 1056 if group == 32 else 1088
    rng = np.random.default_rng(per + group)
    P = E * per
    dev, w = weights(rng, E, N, K, group, scale, zeros, exact=True)
    x = rng.integers(-4, 5, (P, K)).astype(np.float64)
    off, pe = groups(rng, P, E)
    out = torch.full((P + 1, N), 7.0, dtype=torch.bfloat16, device="cuda")
    product(on_gpu(x, torch.bfloat16), dev, off, pe, P, E, N, K, group, out)
    np.testing.assert_array_equal(np_(out[:P]), oracle.bf16_round(oracle.w4_grouped_product(x, w, off, pe)))
    assert bool((out[P] == 7).all())
    assert abi().semmoe_check_errors() == 0


@pytest.mark.parametrize("group,scale,zeros", [(128, "bf16", False), (64, "bf16", True), (32, "f32", False)])
@pytest.mark.parametrize("per", [6, 47, 100])
def test_ffn_of_several_units_a_cta(per, group, scale, zeros):
    E, H, I = 64, 512, 640
    rng = np.random.default_rng(per + group)
    P = E * per
    d13, w13 = weights(rng, E, 2 * I, H, group, scale, zeros)
    d2, w2 = weights(rng, E, H, I, group, scale, zeros)
    x = on_gpu(rng.standard_normal((P, H)) * 0.5, torch.bfloat16)
    off, pe = groups(rng, P, E)
    y = torch.full((P + 1, H), 7.0, dtype=torch.bfloat16, device="cuda")
    abi().semmoe_w4_grouped_ffn(x, on_gpu(off, torch.int32), on_gpu(pe, torch.int32), *d13, *d2, P, E, H, I, group, y)
    ref = oracle.w4_grouped_ffn(np_(x), w13, w2, off, pe)
    got = np_(y[:P])
    assert max_rel(got, ref) < TOL["bf16"]
    assert np.sqrt(((got - ref) ** 2).mean()) < 5 * 2.0 ** -8 * np.sqrt((ref ** 2).mean())
    assert bool((y[P] == 7).all())
    assert abi().semmoe_check_errors() == 0
