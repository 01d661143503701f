"""The norms around the layer on the CPU: the oracle against closed forms, and what the calls refuse."""
import ctypes

import numpy as np
import pytest
import torch

import oracle


@pytest.fixture(scope="module")
def abi():
    from token_expert_routing_gb300 import build, _abi
    build.build()
    return _abi


def _err(lib):
    return lib.semmoe_last_error().decode()


P = ctypes.c_void_p(4096)
NAN, INF = float("nan"), float("inf")


def test_oracle_norms_have_their_moments():
    rng = np.random.default_rng(1)
    x = 3 + 2 * rng.standard_normal((5, 400))
    y = oracle.norm(x, "layer", eps=1e-12)
    np.testing.assert_allclose(y.mean(1), 0, atol=1e-12)
    np.testing.assert_allclose((y ** 2).mean(1), 1, rtol=1e-9)
    np.testing.assert_allclose((oracle.norm(x, "rms", eps=1e-12) ** 2).mean(1), 1, rtol=1e-9)
    # 3, 4 about 0: root mean square sqrt(12.5); weight held as its distance from 1
    np.testing.assert_allclose(oracle.norm([[3.0, 4.0]], "rms", [0.0, 1.0], [0.5, 0.0], 1.0, 0.0),
                               [[3 / 12.5 ** 0.5 + 0.5, 8 / 12.5 ** 0.5]])


def test_oracle_combine_norm_is_the_combine_and_its_steps():
    rng = np.random.default_rng(2)
    y, shared, res = rng.standard_normal((4, 8)), rng.standard_normal((2, 8)), rng.standard_normal((2, 8))
    q, w = np.array([2, -1, 0, 3]), np.array([[0.25, 0.0], [0.5, 1.5]])
    rows = np.stack([shared[0] + 0.25 * y[2], shared[1] + 0.5 * y[0] + 1.5 * y[3]])
    out, nxt = oracle.combine_norm(y, q, w, 2, shared)
    np.testing.assert_allclose(out, rows)
    assert nxt is None
    np.testing.assert_allclose(out, oracle.combine(y, q, w, np.array([1, 2]), "f32", shared), rtol=1e-6)
    gate = rng.standard_normal((1, 8))
    out, nxt = oracle.combine_norm(y, q, w, 2, shared, "rms", gate=gate, block_scale=0.5, residual=res, residual_scale=2.0,
                                   next="layer")
    np.testing.assert_allclose(out, 2 * res + 0.5 * gate * oracle.norm(rows, "rms"))
    np.testing.assert_allclose(nxt, oracle.norm(out, "layer"))


def norm(lib, x=P, dtype=1, T=4, H=64, kind=1, w=P, b=None, wd=1, off=0.0, eps=1e-6, out=P):
    return lib.semmoe_norm(x, dtype, T, H, kind, w, b, wd, off, eps, out, None)


def after(lib, y=P, q=P, w=P, ys=None, dtype=1, T=4, H=64, k=2, n=8, post=1, pw=P, pb=None, nxt=0, nw=None, nb=None, wd=1,
          off=0.0, eps=1e-6, g=None, gd=1, gr=0, bs=1.0, r=P, rs=1.0, out=P, no=None):
    return lib.semmoe_combine_norm(y, q, w, ys, dtype, T, H, k, n, post, pw, pb, nxt, nw, nb, wd, off, eps, g, gd, gr, bs, r,
                                   rs, out, no, None)


Q = ctypes.c_void_p(8192)


@pytest.mark.parametrize("call,kw,word", [
    (norm, dict(dtype=3), "dtype"), (norm, dict(T=-1), "T = -1"), (norm, dict(T=2 ** 31 - 1), "T ="),
    (norm, dict(H=0), "H = 0"), (norm, dict(H=12), "H = 12"), (norm, dict(H=-8), "H = -8"), (norm, dict(H=16392), "H = 16392"),
    (norm, dict(dtype=0, H=8196), "H = 8196"), (norm, dict(kind=0), "bad kind 0"), (norm, dict(kind=3), "bad kind 3"),
    (norm, dict(wd=2), "w_dtype 2"), (norm, dict(off=NAN), "weight_offset"), (norm, dict(eps=0.0), "eps"),
    (norm, dict(eps=-1e-6), "eps"), (norm, dict(eps=INF), "eps"), (norm, dict(eps=NAN), "eps"),
    (norm, dict(w=ctypes.c_void_p(8)), "aligned"), (norm, dict(b=ctypes.c_void_p(8)), "aligned"), (norm, dict(x=None), "null"),
    (norm, dict(out=None), "null"), (norm, dict(x=ctypes.c_void_p(8)), "aligned"), (norm, dict(out=ctypes.c_void_p(8)), "aligned"),
    (after, dict(dtype=2), "dtype"), (after, dict(T=-1), "T = -1"), (after, dict(H=20), "H = 20"), (after, dict(k=0), "k_max=0"),
    (after, dict(n=-1), "P=-1"), (after, dict(T=1 << 30, k=2), "too large"), (after, dict(post=4), "post_kind 4"),
    (after, dict(nxt=-1, no=Q), "next_kind -1"), (after, dict(wd=9), "w_dtype 9"), (after, dict(eps=0.0), "eps"),
    (after, dict(post=0, nxt=1, eps=0.0, no=Q), "eps"), (after, dict(g=P, gd=5, gr=1), "gate_dtype 5"),
    (after, dict(g=P, gr=2), "gate_rows = 2"), (after, dict(g=P, gr=0), "gate_rows = 0"), (after, dict(bs=INF), "scales"),
    (after, dict(rs=NAN), "scales"), (after, dict(out=None), "null"), (after, dict(w=None), "null"), (after, dict(y=None), "null y_perm"),
    (after, dict(y=None, q=None), "null y_perm"), (after, dict(nxt=1), "next_out"), (after, dict(no=Q), "next_out"),
    (after, dict(nxt=1, no=P), "of its own"), (after, dict(ys=ctypes.c_void_p(8)), "aligned"),
    (after, dict(r=ctypes.c_void_p(4)), "aligned"), (after, dict(g=ctypes.c_void_p(8), gr=1), "aligned"),
    (after, dict(q=ctypes.c_void_p(2)), "misaligned"), (after, dict(pw=ctypes.c_void_p(8)), "aligned"),
    (after, dict(), "out is neither"), (after, dict(q=None, g=P, gr=1), "out is neither"),
    (after, dict(y=Q, g=ctypes.c_void_p(16384), gr=4, nxt=1, no=ctypes.c_void_p(16384)), "next_out no gate"),
])
def test_refusals(abi, call, kw, word):
    lib = abi.lib()
    assert call(lib, **kw) == 1, kw
    assert word in _err(lib), (kw, _err(lib))


def test_no_rows_are_no_work(abi):
    assert norm(abi.lib(), T=0, x=None, out=None) == 0
    assert after(abi.lib(), T=0, y=None, out=None, n=0) == 0


T, H, N, K = 3, 64, 5, 2
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def entry(name):
    """The call and its buffers: argument name -> (type, elements, what the refusal names)."""
    if name == "norm":
        return (dict(x=(BF16, T * H, "x"), weight=(F32, H, "weight"), bias=(F32, H, "bias"), out=(BF16, T * H, "out")),
                lambda a, b: a.semmoe_norm(b["x"], T, H, 1, b["weight"], b["bias"], 0.0, 1e-6, b["out"]))
    if name == "norm_bias":
        return (dict(x=(F32, T * H, "x"), bias=(BF16, H, "bias"), out=(F32, T * H, "out")),
                lambda a, b: a.semmoe_norm(b["x"], T, H, 1, None, b["bias"], 0.0, 1e-6, b["out"]))
    maps = {} if name == "dense" else dict(q=(I32, T * K, "pair_to_sorted"), w=(F32, T * K, "topk_w"))
    rows = T if name == "dense" else N
    return (dict(y=(BF16, rows * H, "y_perm"), **maps, ys=(BF16, T * H, "y_shared"), pw=(F32, H, "post_weight"),
                 pb=(F32, H, "post_bias"), nw=(F32, H, "next_weight"), nb=(F32, H, "next_bias"), g=(BF16, T * H, "gate"),
                 r=(BF16, T * H, "residual"), out=(BF16, T * H, "out"), no=(BF16, T * H, "next_out")),
            lambda a, b: a.semmoe_combine_norm(b["y"], b.get("q"), b.get("w"), b["ys"], T, H, K, N, 1, b["pw"], b["pb"], 2, b["nw"],
                                               b["nb"], 0.0, 1e-6, b["g"], T, 1.0, b["r"], 1.0, b["out"], b["no"]))


@pytest.mark.parametrize("name", ["norm", "norm_bias", "combine", "dense"])
def test_every_buffer_is_checked(abi, name):
    spec, call = entry(name)
    good = {k: torch.zeros(n, dtype=t) for k, (t, n, _) in spec.items()}
    with pytest.raises(ValueError, match="expected a CUDA tensor"):
        call(abi, good)
    for key, (t, n, what) in spec.items():
        with pytest.raises(ValueError, match=f"^{what}: expected at least {n} "):
            call(abi, {**good, key: good[key][:n - 1]})
        with pytest.raises(ValueError, match=f"^{what}: expected|unsupported dtype"):
            call(abi, {**good, key: torch.zeros(n, dtype=torch.int64)})


def test_the_norms_of_one_call_share_a_weight_type(abi):
    spec, call = entry("dense")
    good = {k: torch.zeros(n, dtype=t) for k, (t, n, _) in spec.items()}
    good["nw"], good["nb"] = good["nw"].bfloat16(), good["nb"].bfloat16()
    with pytest.raises(ValueError, match="one type"):
        call(abi, good)
