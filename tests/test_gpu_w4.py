"""4-bit weights with group scales on the GPU against the oracle: conversions exact, products exact where every
number is, and within the bound of their roundings where not.

Bound of a product: every weight may be rounded to bf16 (2^-8 of it), the sum of K fp32 products adds at most
K 2^-22 of the products' magnitudes, and the output half a step.  Over many outputs the roundings are independent of
the products' signs, so the root mean square of the error stays below a half step (2^-8 of the outputs') a rounding."""
import numpy as np
import pytest
import torch

import oracle
from parity_utils import TOL, max_rel, np_

pytestmark = pytest.mark.gpu

U8 = dict(dtype=torch.uint8, device="cuda")
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def abi():
    from token_expert_routing_gb300 import _abi
    return _abi


def cuda(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dtype).cuda()


def pack(code):
    return (code[..., 0::2] | (code[..., 1::2] << 4)).astype(np.uint8)


def unpack(codes):
    c = np_(codes)
    return np.stack([c & 15, c >> 4], axis=-1).reshape(*c.shape[:-1], -1)


@pytest.mark.parametrize("zeros", [True, False], ids=["zeros", "symmetric"])
@pytest.mark.parametrize("scale", ["bf16", "f32"])
@pytest.mark.parametrize("rows,K,group", [(1, 32, 32), (3, 352, 32), (130, 320, 64), (77, 1024, 128), (5, 1536, 512)])
def test_quantize_and_dequantize(rows, K, group, scale, zeros):
    rng = np.random.default_rng(rows + K)
    x = rng.standard_normal((rows, K)) * np.exp(rng.normal(0, 4, (rows, 1)))
    x.reshape(-1)[::group // 2 + 1] = 0
    if rows > 2:
        x[1, :group] = 0
        x[1, -group:] = 2.5
        x[2] = np.abs(x[2])
    for dtype in ("f32", "bf16"):
        xt = cuda(x, DT[dtype])
        if rows > 100:
            xt[3, 1], xt[4, K - 1] = float("nan"), float("-inf")
            xt[5] *= 3e38 / float(xt[5].abs().max())
        codes = torch.full((rows + 1, K // 2), 0x5a, **U8)
        scales = torch.full((rows + 1, K // group), 3.0, dtype=DT[scale], device="cuda")
        zp = torch.full((rows + 1, K // group), 99, **U8) if zeros else None
        abi().semmoe_w4_quantize(xt, rows, K, group, codes, scales, zp)
        code, s, z = oracle.w4_encode(np_(xt), group, zeros, scale)
        np.testing.assert_array_equal(np_(scales[:rows]), s)
        np.testing.assert_array_equal(unpack(codes[:rows]), code)
        if zeros:
            np.testing.assert_array_equal(np_(zp[:rows]), z)
            assert bool((zp[rows] == 99).all())
        assert bool((codes[rows] == 0x5a).all()) and bool((scales[rows] == 3).all())
        for t in ("f32", "bf16"):
            out = torch.empty(rows, K, dtype=DT[t], device="cuda")
            abi().semmoe_w4_dequantize(codes, scales, zp, rows, K, group, out)
            np.testing.assert_array_equal(np_(out), oracle.round_to(oracle.w4_values(code, s, z, group), t))
    assert abi().semmoe_check_errors() == 0


def weights(rng, E, rows, K, group, scale, zeros, exact=False):
    """(device tuple, values [E, rows, K]); exact: scales are powers of two, so that w is exact in bf16."""
    code = rng.integers(0, 16, (E, rows, K))
    s = np.exp2(rng.integers(-3, 2, (E, rows, K // group))) if exact else rng.uniform(0.2, 1.0, (E, rows, K // group)) / 8
    s = oracle.round_to(s, scale)
    z = rng.integers(0, 16, (E, rows, K // group)) if zeros else None
    dev = (cuda(pack(code), torch.uint8), cuda(s, DT[scale]), None if z is None else cuda(z, torch.uint8))
    return dev, oracle.w4_values(code, s, z, group)


def split(rng, P, E, empty=()):
    """Offsets of P rows in E uneven groups and an order of experts."""
    p = rng.dirichlet(np.full(E, 0.6))
    p[list(empty)] = 0
    p = p / p.sum() if p.sum() else np.eye(E)[0]
    count = rng.multinomial(P, p)
    return np.concatenate([[0], np.cumsum(count)]), rng.permutation(E)


def product(x, dev, off, pe, P, E, N, K, group, out, stream=None):
    abi().semmoe_w4_grouped_gemm(x, cuda(off, torch.int32), cuda(pe, torch.int32), *dev, P, E, N, K, group, out, stream)


CASES = [  # P, E, N, K, group, scale, zeros
    (1, 1, 8, 32, 32, "bf16", False), (1, 1, 2048, 2048, 128, "bf16", False), (1, 1, 40, 1408, 128, "f32", True),
    (2, 4, 96, 96, 32, "f32", True), (7, 3, 72, 352, 32, "bf16", True), (9, 8, 200, 640, 64, "bf16", True),
    (48, 5, 264, 768, 256, "f32", False), (100, 128, 64, 512, 64, "bf16", False), (130, 3, 120, 160, 32, "bf16", True),
    (333, 7, 136, 1056, 32, "f32", True), (600, 2, 1000, 384, 128, "bf16", True), (1500, 4, 304, 2080, 32, "bf16", False),
    (3000, 9, 520, 576, 64, "f32", True), (257, 256, 16, 64, 64, "bf16", True), (4096, 1, 256, 1024, 1024, "bf16", False),
]


@pytest.mark.parametrize("P,E,N,K,group,scale,zeros", CASES)
def test_product_of_whole_numbers_is_exact(P, E, N, K, group, scale, zeros):
    """Whole rows and scales that are powers of two: every partial sum is exact in fp32, so only the output rounds."""
    rng = np.random.default_rng(P + N + K)
    dev, w = weights(rng, E, N, K, group, scale, zeros, exact=True)
    x = rng.integers(-4, 5, (P, K)).astype(np.float64)
    off, pe = split(rng, P, E)
    out = torch.full((P + 1, N), 7.0, dtype=torch.bfloat16, device="cuda")
    product(cuda(x, torch.bfloat16), dev, off, pe, P, E, N, K, group, out)
    np.testing.assert_array_equal(np_(out[:P]), oracle.bf16_round(oracle.w4_grouped_product(x, w, off, pe)))
    assert bool((out[P] == 7).all())
    assert abi().semmoe_check_errors() == 0


@pytest.mark.parametrize("P,E,N,K,group,scale,zeros", CASES)
def test_product(P, E, N, K, group, scale, zeros):
    rng = np.random.default_rng(P * 3 + N + K)
    dev, w = weights(rng, E, N, K, group, scale, zeros)
    x = cuda(rng.standard_normal((P, K)), torch.bfloat16)
    off, pe = split(rng, P, E, empty=(0,) if E > 2 else ())
    out = torch.empty(P, N, dtype=torch.bfloat16, device="cuda")
    product(x, dev, off, pe, P, E, N, K, group, out)
    ref = oracle.w4_grouped_product(np_(x), w, off, pe)
    size = oracle.w4_grouped_product(np.abs(np_(x)), np.abs(w), off, pe)
    err = np.abs(np_(out) - ref)
    assert (err <= (2.0 ** -8 + K * 2.0 ** -22) * size + 2.0 ** -8 * np.abs(ref)).all()
    if P * N > 1000:
        assert np.sqrt((err ** 2).mean()) < 2 * 2.0 ** -8 * np.sqrt((ref ** 2).mean())
    again = torch.empty_like(out)
    product(x, dev, off, pe, P, E, N, K, group, again)
    assert torch.equal(again, out)
    assert abi().semmoe_check_errors() == 0


FFN = [  # P, E, H, I, group, scale, zeros
    (1, 1, 32, 32, 32, "bf16", False), (8, 128, 256, 96, 32, "f32", True), (24, 6, 352, 160, 32, "bf16", True),
    (40, 64, 512, 256, 128, "bf16", False), (300, 5, 384, 192, 64, "bf16", True), (900, 3, 256, 352, 32, "f32", False),
    (2500, 16, 1024, 768, 256, "bf16", False), (2048, 1, 320, 1408, 64, "f32", True),
]


@pytest.mark.parametrize("P,E,H,I,group,scale,zeros", FFN)
def test_ffn(P, E, H, I, group, scale, zeros):
    rng = np.random.default_rng(P + H + I)
    d13, w13 = weights(rng, E, 2 * I, H, group, scale, zeros)
    d2, w2 = weights(rng, E, H, I, group, scale, zeros)
    x = cuda(rng.standard_normal((P, H)) * 0.5, torch.bfloat16)
    off, pe = split(rng, P, E)
    tabs = cuda(off, torch.int32), cuda(pe, torch.int32)
    y = torch.full((P + 1, H), 7.0, dtype=torch.bfloat16, device="cuda")
    abi().semmoe_w4_grouped_ffn(x, *tabs, *d13, *d2, P, E, H, I, group, y)
    ref = oracle.w4_grouped_ffn(np_(x), w13, w2, off, pe)
    got = np_(y[:P])
    assert max_rel(got, ref) < TOL["bf16"]
    # four roundings: both weights, h (carried through the gate and up products' curvature: counted twice), the output
    assert np.sqrt(((got - ref) ** 2).mean()) < 5 * 2.0 ** -8 * np.sqrt((ref ** 2).mean())
    assert bool((y[P] == 7).all())
    # a workspace of the caller's on another stream
    ws = torch.empty(abi().semmoe_w4_grouped_ffn_workspace_size(P, I), **U8)
    y2 = torch.empty(P, H, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    abi().semmoe_w4_grouped_ffn(x, *tabs, *d13, *d2, P, E, H, I, group, y2, ws, side)
    side.synchronize()
    assert torch.equal(y2, y[:P])
    assert abi().semmoe_check_errors() == 0


@pytest.mark.parametrize("P", [6, 60, 900])
def test_rows_that_are_not_finite_stay_to_themselves(P):
    rng = np.random.default_rng(P)
    E, N, K, group = 3, 136, 320, 64
    dev, w = weights(rng, E, N, K, group, "bf16", True)
    x = cuda(rng.standard_normal((P, K)), torch.bfloat16)
    off, pe = split(rng, P, E)
    clean, out = (torch.empty(P, N, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    product(x, dev, off, pe, P, E, N, K, group, clean)
    x[1, 5], x[P // 2, 0], x[P - 1, K - 1] = float("nan"), float("inf"), -float("inf")
    product(x, dev, off, pe, P, E, N, K, group, out)
    rows = [1, P // 2, P - 1]
    keep = np.setdiff1d(np.arange(P), rows)
    assert torch.equal(out[keep], clean[keep])
    assert bool(torch.isnan(out[1]).all()) and not bool(torch.isfinite(out[rows]).any())
    assert abi().semmoe_check_errors() == 0


@pytest.mark.parametrize("P", [9, 700])
def test_bad_groups_are_flagged_and_leave_their_rows(P):
    rng = np.random.default_rng(P)
    E, N, K, group = 4, 72, 128, 128
    dev, w = weights(rng, E, N, K, group, "f32", False, exact=True)
    x = rng.integers(-4, 5, (P, K)).astype(np.float64)
    a, b = P // 3, 2 * P // 3
    for off, pe, live, bits in (
            ([0, a, b, P, P], [1, 9, 2, 0], [(0, a, 1), (b, P, 2)], abi().SEMMOE_DEVERR_EXPERT),
            ([0, a, b, P, P], [1, -1, 2, 0], [(0, a, 1), (b, P, 2)], abi().SEMMOE_DEVERR_EXPERT),
            ([0, a, P + 1, P, P], [1, 0, 2, 3], [(0, a, 1)], abi().SEMMOE_DEVERR_PAIRS),
            ([-1, a, b, P, P], [1, 0, 2, 3], [(a, b, 0), (b, P, 2)], abi().SEMMOE_DEVERR_PAIRS)):
        out = torch.full((P, N), 7.0, dtype=torch.bfloat16, device="cuda")
        product(cuda(x, torch.bfloat16), dev, np.array(off), np.array(pe), P, E, N, K, group, out)
        with pytest.raises(abi().SemMoEError) as e:
            abi().semmoe_check_errors()
        assert e.value.bits == bits
        ref = np.full((P, N), 7.0)
        for lo, hi, ex in live:
            ref[lo:hi] = oracle.bf16_round(x[lo:hi] @ w[ex].T)
        np.testing.assert_array_equal(np_(out), ref)
    # ranges that overlap into more blocks than P rows have: nothing runs
    off = np.array([0, P, 0, P, 0, P])
    dev5, _ = weights(rng, 5, N, K, group, "f32", False, exact=True)
    out = torch.full((P, N), 7.0, dtype=torch.bfloat16, device="cuda")
    product(cuda(x, torch.bfloat16), dev5, off, np.arange(5), P, 5, N, K, group, out)
    with pytest.raises(abi().SemMoEError) as e:
        abi().semmoe_check_errors()
    assert e.value.bits == abi().SEMMOE_DEVERR_PAIRS


def test_rows_outside_every_group_are_left():
    rng = np.random.default_rng(4)
    E, N, K, P = 3, 64, 64, 50
    dev, w = weights(rng, E, N, K, 32, "bf16", True, exact=True)
    x = rng.integers(-4, 5, (P, K)).astype(np.float64)
    off, pe = np.array([5, 5, 20, 41]), np.array([2, 1, 0])
    out = torch.full((P, N), 7.0, dtype=torch.bfloat16, device="cuda")
    product(cuda(x, torch.bfloat16), dev, off, pe, P, E, N, K, 32, out)
    ref = np.full((P, N), 7.0)
    ref[5:20], ref[20:41] = oracle.bf16_round(x[5:20] @ w[1].T), oracle.bf16_round(x[20:41] @ w[0].T)
    np.testing.assert_array_equal(np_(out), ref)
    assert abi().semmoe_check_errors() == 0


@pytest.mark.parametrize("P", [3, 400])
def test_matrices_past_32_bits(P):
    """The last expert's codes start 4 GB into the tensor."""
    rng = np.random.default_rng(8)
    E, N, K, group = 256, 4096, 8320, 128
    codes = torch.empty(E, N, K // 2, **U8)
    assert (E - 1) * N * (K // 2) > 2 ** 32
    scales = torch.ones(E, N, K // group, dtype=torch.bfloat16, device="cuda")
    last = torch.randint(0, 256, (N, K // 2), **U8)
    codes[E - 1] = last
    x = torch.randint(-2, 3, (P, K), device="cuda").to(torch.bfloat16)
    off = torch.tensor([0] * E + [P], dtype=torch.int32, device="cuda")
    pe = torch.arange(E, dtype=torch.int32, device="cuda")
    out = torch.empty(P, N, dtype=torch.bfloat16, device="cuda")
    abi().semmoe_w4_grouped_gemm(x, off, pe, codes, scales, None, P, E, N, K, group, out)
    w = torch.stack([last & 15, last >> 4], -1).flatten(1).double() - 8
    assert torch.equal(out, (x.double() @ w.T).to(torch.bfloat16))
    assert abi().semmoe_check_errors() == 0


@pytest.mark.parametrize("P", [4, 500])
def test_ffn_in_graphs_that_run_at_once(P):
    """Two captured calls with workspaces of their own, replayed beside one another and after eager calls."""
    rng = np.random.default_rng(P)
    E, H, I, group = 6, 256, 128, 64
    d13, _ = weights(rng, E, 2 * I, H, group, "bf16", True)
    d2, _ = weights(rng, E, H, I, group, "bf16", True)
    off, pe = split(rng, P, E)
    tabs = cuda(off, torch.int32), cuda(pe, torch.int32)
    xs = [cuda(rng.standard_normal((P, H)), torch.bfloat16) for _ in range(2)]
    ys = [torch.empty(P, H, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    want = []
    for x in xs:
        y = torch.empty_like(ys[0])
        abi().semmoe_w4_grouped_ffn(x, *tabs, *d13, *d2, P, E, H, I, group, y)
        want.append(y)
    graphs, streams = [], [torch.cuda.Stream() for _ in range(2)]
    for x, y in zip(xs, ys):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            abi().semmoe_w4_grouped_ffn(x, *tabs, *d13, *d2, P, E, H, I, group, y)
        graphs.append(g)
    for y in ys:
        y.zero_()
    torch.cuda.synchronize()
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ys, want))
    assert abi().semmoe_check_errors() == 0


def test_product_whose_wait_runs_out_ends_and_the_next_is_right():
    """Every CTA's issuer waits for a barrier that only it could complete, for its 2 s; all other roles then stop."""
    import time
    a = abi()
    rng = np.random.default_rng(17)
    E, N, K, group = 3, 264, 1408, 128
    for P in (40, 700):  # k-blocks of 128 and of 64 columns
        dev, w = weights(rng, E, N, K, group, "bf16", False, exact=True)
        x = rng.integers(-4, 5, (P, K)).astype(np.float64)
        off, pe = split(rng, P, E)
        out = torch.full((P, N), 7.0, dtype=torch.bfloat16, device="cuda")
        xt, ot, pt = cuda(x, torch.bfloat16), cuda(off, torch.int32), cuda(pe, torch.int32)
        t0 = time.perf_counter()
        a.semmoe_selftest_w4_wait(xt, ot, pt, *dev, P, E, N, K, group, out)
        with pytest.raises(a.SemMoEError) as ei:
            a.semmoe_check_errors()
        assert ei.value.code == a.SEMMOE_ERR_DEVICE_TIMEOUT and ei.value.bits & a.SEMMOE_DEVERR_TIMEOUT
        assert 0.1 < time.perf_counter() - t0 < 60
        assert bool((out == 7).all())
        assert a.semmoe_check_errors() == 0
        a.semmoe_w4_grouped_gemm(xt, ot, pt, *dev, P, E, N, K, group, out)
        np.testing.assert_array_equal(np_(out), oracle.bf16_round(oracle.w4_grouped_product(x, w, off, pe)))
        assert a.semmoe_check_errors() == 0
