"""The norms around the layer on the GPU against the oracle in 64 bits.

Tolerances follow the arithmetic: ``track`` carries a bound of the fp32 error of every value
through the same steps (u = 2^-24 a rounding, SUMS roundings on the longest way through a sum,
2 steps of rsqrt), and an output adds half a step of its type."""
import numpy as np
import pytest
import torch

import oracle
from parity_utils import np_

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
SUMS = 64          # a thread adds at most 4 x 8 values, then ten levels of lanes and warps
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
KIND = {"": 0, "rms": 1, "layer": 2}


def abi():
    from token_expert_routing_gb300 import _abi
    return _abi


def cuda(a, dtype):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(dtype).cuda()


def track(v, ev, kind, w, b, offset, eps):
    """(normalised rows, bound of their error) of rows v known within ev."""
    if kind == "":
        return v, ev
    m, em = 0.0, 0.0
    if kind == "layer":
        m = v.mean(1, keepdims=True)
        em = ev.mean(1, keepdims=True) + SUMS * U * np.abs(v).mean(1, keepdims=True)
    d = v - m
    ed = ev + em + U * np.abs(d)
    var = np.square(d).mean(1, keepdims=True)
    evar = 2 * (np.abs(d) * ed).mean(1, keepdims=True) + np.square(ed).mean(1, keepdims=True) + SUMS * U * var
    rstd = 1 / np.sqrt(var + eps)
    rho = evar / (var + eps) + 6 * U  # half of the variance's relative error, with room for its square
    y, ey = d * rstd, ed * rstd + np.abs(d * rstd) * (rho + 3 * U)
    if w is not None:
        g = offset + np_(w).astype(np.float64)
        y, ey = y * g, ey * np.abs(g) + 3 * U * np.abs(y * g)
    if b is not None:
        y = y + np_(b).astype(np.float64)
        ey = ey + U * np.abs(y)
    return y, ey


def close(got, ref, err):
    half = HALF[got.dtype]
    g = np_(got).astype(np.float64)
    bad = ~(np.abs(g - ref) <= err + half * (np.abs(ref) + err))
    assert not bad.any(), (int(bad.sum()), np.abs(g - ref)[bad].max(), np.argwhere(bad)[:4])


SHAPES = [(1, 8), (3, 24), (5, 256), (130, 264), (1, 512), (33, 520), (7, 1024), (2, 1032), (64, 1056), (9, 2048), (1, 2048),
          (300, 2056), (3, 4096), (5, 4104), (2, 8192), (3, 16384)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("T,H", SHAPES)
def test_norm(T, H, kind, dtype):
    if dtype == torch.float32:
        H = H // 2 + (4 if H % 16 == 8 else 0)
    rng = np.random.default_rng(T * 31 + H)
    wd = dtype if H % 3 else torch.float32 if dtype == torch.bfloat16 else torch.bfloat16
    offset = float(H % 2 == 0 and T % 2)
    x = cuda(rng.standard_normal((T, H)) * np.exp(rng.normal(0, 2, (T, 1))) + rng.normal(0, 1, (T, 1)), dtype)
    w = None if T == 3 else cuda(1 - offset + 0.3 * rng.standard_normal(H), wd)
    b = cuda(rng.standard_normal(H), wd) if T % 2 else None
    out = torch.full((T + 1, H), 7.0, dtype=dtype, device="cuda")
    eps = 1e-5
    abi().semmoe_norm(x, T, H, KIND[kind], w, b, offset, eps, out)
    v = np_(x).astype(np.float64)
    ref, err = track(v, np.zeros_like(v), kind, w, b, offset, eps)
    np.testing.assert_allclose(ref, oracle.norm(v, kind, None if w is None else np_(w), None if b is None else np_(b), offset, eps),
                               rtol=1e-10, atol=1e-12)
    close(out[:T], ref, err)
    assert bool((out[T] == 7).all())  # the row behind the last one
    inplace = x.clone()
    abi().semmoe_norm(inplace, T, H, KIND[kind], w, b, offset, eps, inplace)
    assert torch.equal(inplace, out[:T])
    assert abi().semmoe_check_errors() == 0


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("H", [64, 1000, 4096])
def test_rows_at_the_ends_of_the_range(H, kind):
    """Rows of zeros, huge and tiny values, constants; rows that hold NaN or infinities stay to themselves."""
    rng = np.random.default_rng(H)
    x = rng.standard_normal((12, H))
    x[1] = 0
    x[2] *= 1e30
    x[3] *= 3e37
    x[4] *= 1e-30
    x[5] = 2.5
    x[6] = 3e38 * np.sign(x[6])
    x[7] *= 1e-18
    x = x.astype(np.float32).astype(np.float64)
    for eps in (1e-6, 1e-30):
        ref, err = track(x, np.zeros_like(x), kind, None, None, 0.0, eps)
        xt = cuda(x, torch.float32)
        xt[9, H // 2], xt[10, H - 1], xt[11, 0] = float("nan"), float("inf"), -float("inf")
        out = torch.empty_like(xt)
        abi().semmoe_norm(xt, 12, H, KIND[kind], None, None, 0.0, eps, out)
        rows = [0, 1, 2, 3, 4, 5, 6, 7, 8]
        # values below the smallest normal number are held with that much error
        close(out[rows], ref[rows], err[rows] + 2.0 ** -126 * 1e3)
        assert bool(torch.isnan(out[9]).all())
        assert bool(torch.isnan(out[10, H - 1])) and bool(torch.isnan(out[11, 0]))
        if kind == "rms":
            assert bool((out[10, :H - 1] == 0).all()) and bool((out[11, 1:] == 0).all())
    assert abi().semmoe_check_errors() == 0


def case(rng, T, H, k, dtype, budgets, shared, gate, wd):
    P = 0
    q = w = None
    if k:
        live = np.ones((T, k), bool)
        if budgets:
            live = np.arange(k)[None] < rng.integers(0, k + 1, (T, 1))  # some tokens have no pair at all
        P = int(live.sum())
        q = np.full(T * k, -1, np.int32)
        q[live.reshape(-1)] = rng.permutation(P)
        w = np.where(live, rng.uniform(0.05, 1, (T, k)), 0)
    d = dict(y=cuda(rng.standard_normal((P if k else T, H)), dtype), q=None if q is None else torch.from_numpy(q).cuda(),
             w=cuda(w, torch.float32), ys=cuda(rng.standard_normal((T, H)), dtype) if shared else None,
             r=cuda(2 * rng.standard_normal((T, H)), dtype))
    d["g"] = {"": None, "channels": cuda(rng.standard_normal((1, H)), wd),
              "tokens": cuda(rng.standard_normal((T, H)), dtype)}[gate]
    for key in ("pw", "pb", "nw", "nb"):
        d[key] = cuda(1 + 0.3 * rng.standard_normal(H), wd)
    return d, P


def run_after(d, T, H, k, P, post, nxt, offset, bs, rs, out, no, stream=None):
    eps = 1e-6
    abi().semmoe_combine_norm(d["y"], d["q"], d["w"], d["ys"], T, H, k, P, KIND[post], d["pw"], d["pb"], KIND[nxt], d["nw"], d["nb"],
                              offset, eps, d["g"], 0 if d["g"] is None else len(d["g"]), bs, d["r"], rs, out, no, stream)


CASES = [  # T, H, k, budgets, shared, post, gate, next
    (1, 2048, 8, False, False, "rms", "", "rms"), (1, 64, 1, False, True, "", "", ""), (64, 2048, 6, True, True, "rms", "channels", "rms"),
    (33, 1056, 3, True, False, "layer", "tokens", "layer"), (130, 256, 4, True, True, "", "tokens", "rms"), (17, 512, 40, True, False, "rms", "", "layer"),
    (9, 4096, 2, False, True, "layer", "channels", ""), (5, 8200, 5, True, True, "rms", "tokens", "rms"), (3, 16384, 8, False, False, "rms", "", "rms"),
    (40, 2048, 0, False, False, "", "tokens", "layer"), (7, 264, 0, False, True, "rms", "channels", "rms"), (2, 1040, 0, False, False, "layer", "", ""),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,H,k,budgets,shared,post,gate,nxt", CASES)
def test_combine_norm(T, H, k, budgets, shared, post, gate, nxt, dtype):
    if dtype == torch.float32:
        H //= 2
    rng = np.random.default_rng(T * 7 + H + k)
    wd = torch.float32 if H % 3 == 0 else torch.bfloat16
    d, P = case(rng, T, H, k, dtype, budgets, shared, gate, wd)
    offset, bs, rs = float(T % 2), 0.75, 1.0 if T % 2 else 0.7
    out = torch.full((T + 1, H), 7.0, dtype=dtype, device="cuda")
    no = torch.full((T + 1, H), 7.0, dtype=dtype, device="cuda") if nxt else None
    run_after(d, T, H, k, P, post, nxt, offset, bs, rs, out, no)
    f = {key: None if t is None else np_(t).astype(np.float64) for key, t in d.items()}
    y = oracle.block_rows(f["y"], f["q"], f["w"], k, f["ys"])
    size = oracle.block_rows(np.abs(f["y"]), f["q"], f["w"], k, None if f["ys"] is None else np.abs(f["ys"]))
    u, eu = track(y, (k + 2) * U * size, post, d["pw"], d["pb"], offset, 1e-6)
    if f["g"] is not None:
        u, eu = u * f["g"], (eu + U * np.abs(u)) * np.abs(f["g"])
    b32, r32 = float(np.float32(bs)), float(np.float32(rs))
    o = b32 * u + r32 * f["r"]
    eo = b32 * (eu + U * np.abs(u)) + 2 * U * (np.abs(o) + np.abs(r32 * f["r"]))
    ref, ref_next = oracle.combine_norm(f["y"], f["q"], f["w"], k, f["ys"], post, f["pw"], f["pb"], f["g"], b32, f["r"], r32, nxt,
                                        f["nw"], f["nb"], offset, 1e-6)
    np.testing.assert_allclose(o, ref, rtol=1e-10, atol=1e-12)
    close(out[:T], o, eo)
    assert bool((out[T] == 7).all())
    if nxt:
        z, ez = track(o, eo, nxt, d["nw"], d["nb"], offset, 1e-6)
        np.testing.assert_allclose(z, ref_next, rtol=1e-9, atol=1e-10)
        close(no[:T], z, ez)
        assert bool((no[T] == 7).all())
    # the residual's own buffer as the output, on another stream than the current one
    again, no2 = d["r"].clone(), None if no is None else torch.empty_like(no)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    run_after({**d, "r": again}, T, H, k, P, post, nxt, offset, bs, rs, again, no2, side)
    side.synchronize()
    assert torch.equal(again, out[:T]) and (no is None or torch.equal(no2[:T], no[:T]))
    assert abi().semmoe_check_errors() == 0


def test_combine_norm_without_norms_is_the_combine():
    rng = np.random.default_rng(5)
    T, H, k = 77, 1024, 6
    d, P = case(rng, T, H, k, torch.bfloat16, True, True, "", torch.float32)
    out, plain = torch.empty(T, H, dtype=torch.bfloat16, device="cuda"), torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    run_after({**d, "r": None}, T, H, k, P, "", "", 0.0, 1.0, 1.0, out, None)
    abi().semmoe_combine(d["y"], d["q"], d["w"], d["ys"], T, H, k, P, plain)
    assert torch.equal(out, plain)
    assert abi().semmoe_check_errors() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,H", [(2, 264), (2500, 136), (2500, 264), (2500, 1032), (2100, 2056), (1300, 4104), (700, 16384 // 2)])
def test_dense_rows_are_one_slot_of_weight_one(T, H, dtype):
    """A dense block's rows, the residual's buffer written over, against the same sums by way of the maps: equal bit for bit."""
    rng = np.random.default_rng(T + H)
    y, shared, residual, gates = (cuda(rng.standard_normal((T, H)), dtype) for _ in range(4))
    post, nxt, bias, row = (cuda(rng.standard_normal(H), torch.float32) for _ in range(4))
    ident = torch.arange(T, dtype=torch.int32, device="cuda")
    ones = torch.ones(T, device="cuda")
    other = gates.to(torch.float32 if dtype == torch.bfloat16 else torch.bfloat16)
    for s, g, pk, nk in ((None, gates, 1, 2), (shared, other, 0, 1), (shared, row, 2, 0), (None, None, 0, 2)):
        got = []
        for maps in (False, True):
            out, z = residual.clone(), torch.zeros_like(residual)
            stream = torch.cuda.Stream()
            stream.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(stream):
                abi().semmoe_combine_norm(y, ident if maps else None, ones if maps else None, s, T, H, 1 if maps else 0, T,
                                          pk, post if pk else None, None, nk, nxt if nk else None, bias if nk == 2 else None, 0.5, 1e-6,
                                          g, 0 if g is None else 1 if g is row else T, 0.75, out, 1.25, out, z if nk else None)
            torch.cuda.current_stream().wait_stream(stream)
            got.append((out, z))
        assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
        assert not torch.equal(got[0][0], residual)
    assert abi().semmoe_check_errors() == 0


def test_a_bad_sorted_row_is_flagged_and_skipped():
    rng = np.random.default_rng(6)
    T, H, k = 5, 256, 2
    for k, at in ((2, 3), (40, 5 * 40 - 1)):
        d, P = case(rng, T, H, k, torch.bfloat16, False, False, "", torch.float32)
        out, want = torch.empty(T, H, dtype=torch.bfloat16, device="cuda"), torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
        gone = d["q"].clone()
        gone[at] = -1
        run_after({**d, "q": gone}, T, H, k, P, "rms", "", 0.0, 1.0, 1.0, want, None)
        d["q"][at] = P
        run_after(d, T, H, k, P, "rms", "", 0.0, 1.0, 1.0, out, None)
        with pytest.raises(abi().SemMoEError) as e:
            abi().semmoe_check_errors()
        assert e.value.bits == abi().SEMMOE_DEVERR_PAIRS
        assert torch.equal(out, want)


def test_norms_in_a_graph():
    rng = np.random.default_rng(7)
    T, H, k = 50, 2048, 4
    d, P = case(rng, T, H, k, torch.bfloat16, True, False, "channels", torch.float32)
    z, out, no = (torch.empty(T, H, dtype=torch.bfloat16, device="cuda") for _ in range(3))

    def step():
        abi().semmoe_norm(d["r"], T, H, 1, d["pw"], None, 0.0, 1e-6, z)
        run_after({**d, "ys": z}, T, H, k, P, "rms", "layer", 1.0, 1.0, 1.0, out, no)

    step()
    want = [t.clone() for t in (z, out, no)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for t in (z, out, no):
        t.zero_()
    for _ in range(2):
        g.replay()
    assert all(torch.equal(a, b) for a, b in zip((z, out, no), want))
    d["r"].neg_()
    g.replay()
    step_out = out.clone()
    step()
    assert torch.equal(out, step_out)
    assert abi().semmoe_check_errors() == 0
