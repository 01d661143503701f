"""GPU parity of the 4-bit microscaled operators against the oracle: codes and
scales bit-exact, dequantised values exact, products within the bound of their
fp32 sums, the FFN within the bf16 layer tolerance."""
import numpy as np
import pytest
import torch

import oracle
from parity_utils import TOL, max_rel, np_

pytestmark = pytest.mark.gpu

i32 = dict(dtype=torch.int32, device="cuda")
u8 = dict(dtype=torch.uint8, device="cuda")


def abi():
    from token_expert_routing_gb300 import _abi
    return _abi


def cuda(a, dtype=torch.float32):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dtype).cuda()


def pack(code):
    code = np.asarray(code)
    return (code[..., 0::2] | (code[..., 1::2] << 4)).astype(np.uint8)


def unpack(codes):
    c = np_(codes)
    return np.stack([c & 15, c >> 4], axis=-1).reshape(*c.shape[:-1], -1)


def scale_at(first_tile, r, blk, K):
    """Byte of block ``blk`` of row r of a group whose scales start at row tile ``first_tile``."""
    kc = -(-K // 128)
    return ((first_tile + r // 128) * kc + blk // 4) * 512 + 16 * (r % 32) + 4 * ((r % 128) // 32) + blk % 4


def scales_of(tiles, counts, K):
    """[rows, K / 32] from the tiled layout of groups of ``counts`` rows."""
    t = np_(tiles)
    out, first = [], 0
    for n in counts:
        r, b = np.arange(n)[:, None], np.arange(K // 32)[None, :]
        out.append(t[scale_at(first, r, b, K)])
        first += -(-n // 128)
    return np.concatenate(out)


def tile_scales(e, counts, K, size, fill=0):
    t = np.full(size, fill, dtype=np.uint8)
    first = row = 0
    for n in counts:
        r, b = np.arange(n)[:, None], np.arange(K // 32)[None, :]
        t[scale_at(first, r, b, K)] = e[row:row + n]
        first, row = first + -(-n // 128), row + n
    kb = K // 32
    if kb % 4:  # column blocks past K of the last tile hold 0
        tt = t.reshape(-1, -(-K // 128), 512)
        tt[:, -1].reshape(-1, 32, 4, 4)[..., kb % 4:] = 0
    return t


def hard_rows(rng, rows, K):
    """Rows over the whole exponent range, with midpoints, saturating values, zeros and denormals."""
    x = rng.standard_normal((rows, K)) * np.exp(rng.normal(0, 3, (rows, 1)))
    b = x.reshape(rows, -1, 32)
    pick = rng.integers(0, 6, b.shape[:2])
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.9, 6.0, 0.0])
    b[pick == 1] = rng.choice(mids, (int((pick == 1).sum()), 32)) * rng.choice([-1, 1], (int((pick == 1).sum()), 32))
    b[pick == 1, 0] = 7.0
    b[pick == 2] = 0.0
    b[pick == 3] *= 2.0 ** -130
    b[pick == 4] *= 2.0 ** 110
    return x


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("groups,rows,K", [(1, 1, 32), (1, 130, 96), (3, 77, 352), (2, 256, 2080), (5, 128, 128)])
def test_quantize_and_dequantize_are_exact(groups, rows, K, dtype):
    rng = np.random.default_rng(groups * 1000 + rows + K)
    x = cuda(hard_rows(rng, groups * rows, K), torch.bfloat16 if dtype == "bf16" else torch.float32)
    if rows > 1:
        x[1, 3], x[rows - 1, K - 1], x[rows // 2, 0] = float("nan"), float("inf"), -float("inf")
    codes = torch.full((groups * rows, K // 2), 0x5a, **u8)
    scales = torch.full((abi().semmoe_mx4_scales_size(groups * rows, K, groups),), 0x5a, **u8)
    abi().semmoe_mx4_quantize(x, groups, rows, K, codes, scales)
    ref_code, ref_e = oracle.mx4_encode(np_(x))
    e = scales_of(scales, [rows] * groups, K)
    np.testing.assert_array_equal(e, ref_e)
    live = np.repeat(ref_e != 255, 32, axis=1)
    np.testing.assert_array_equal(unpack(codes)[live], ref_code[live])
    kb = K // 32
    if kb % 4:  # column blocks past K
        used = groups * (-(-rows // 128)) * (-(-K // 128)) * 512
        last = np_(scales)[:used].reshape(-1, -(-K // 128), 32, 4, 4)[:, -1, :, :, kb % 4:]
        assert (last == 0).all()
    for t in (torch.float32, torch.bfloat16):
        out = torch.empty(groups * rows, K, dtype=t, device="cuda")
        abi().semmoe_mx4_dequantize(codes, scales, groups, rows, K, out)
        np.testing.assert_array_equal(np_(out), oracle.mx4_values(ref_code, ref_e))
    assert abi().semmoe_check_errors() == 0


def routing(rng, T, k_max, E, budgets=False, empty=()):
    """Pairs of a batch, sorted stably by expert: maps and offsets as semmoe_permute writes them."""
    p = rng.dirichlet(np.full(E, 0.7))
    p[list(empty)] = 0
    noise = np.log(np.maximum(p, 1e-30))[None] - np.log(-np.log(rng.uniform(1e-9, 1, (T, E))))
    idx = np.argsort(-noise, axis=1)[:, :k_max]
    k = rng.integers(1, k_max + 1, T) if budgets else np.full(T, k_max)
    live = (np.arange(k_max)[None] < k[:, None]).reshape(-1)
    flat = np.where(live, idx.reshape(-1), E)
    order = np.argsort(flat, kind="stable")[:live.sum()]
    back = np.full(T * k_max, -1)
    back[order] = np.arange(len(order))
    count = np.bincount(flat[live], minlength=E)[:E]
    return order, back, np.concatenate([[0], np.cumsum(count)]), count


@pytest.mark.parametrize("T,k_max,E,K,budgets", [(1, 1, 1, 32, False), (1, 8, 128, 2048, False), (300, 3, 7, 352, True),
                                                 (64, 40, 64, 160, True), (515, 6, 256, 4160, False)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_quantize_rows_is_quantise_then_permute(T, k_max, E, K, budgets, dtype):
    rng = np.random.default_rng(T + K)
    order, back, off, count = routing(rng, T, k_max, E, budgets, empty=(0,) if E > k_max else ())
    P = len(order)
    x = cuda(hard_rows(rng, T, K), torch.bfloat16 if dtype == "bf16" else torch.float32)
    codes = torch.zeros(P, K // 2, **u8)
    scales = torch.zeros(abi().semmoe_mx4_scales_size(P, K, E), **u8)
    abi().semmoe_mx4_quantize_rows(x, T, K, cuda(back, torch.int32), k_max, P, cuda(off, torch.int32), E, codes, scales)
    assert abi().semmoe_check_errors() == 0
    ref_code, ref_e = oracle.mx4_encode(np_(x))
    np.testing.assert_array_equal(unpack(codes), ref_code[order // k_max])
    np.testing.assert_array_equal(scales_of(scales, count, K), ref_e[order // k_max])


def test_quantize_rows_flags_what_does_not_fit():
    """A sorted row past P or outside every group is skipped and flagged, and so are offsets that step back."""
    from token_expert_routing_gb300 import SemMoEError
    x = torch.ones(2, 64, device="cuda")
    codes, scales = torch.full((3, 32), 0x77, **u8), torch.full((abi().semmoe_mx4_scales_size(3, 64, 2),), 0x77, **u8)
    for back, off in (([0, 5, 1, 2], [0, 1, 3]), ([0, 2, 1, -1], [0, 1, 2]), ([0, 1, 2, -1], [2, 1, 3])):
        codes.fill_(0x77)
        abi().semmoe_mx4_quantize_rows(x, 2, 64, cuda(np.array(back), torch.int32), 2, 3, cuda(np.array(off), torch.int32),
                                       2, codes, scales)
        with pytest.raises(SemMoEError) as e:
            abi().semmoe_check_errors()
        assert e.value.bits == abi().SEMMOE_DEVERR_PAIRS
    assert (np_(codes)[0] == 0x77).all()


def operands(rng, P, E, N, K, count, zero_fill=0):
    """Random 4-bit rows and matrices: packed device tensors and their values."""
    code = rng.integers(0, 16, (P, K))
    e = rng.integers(117, 130, (P, K // 32))
    wcode, we = rng.integers(0, 16, (E * N, K)), rng.integers(120, 126, (E * N, K // 32))
    # the scales of unused rows stand for NaN: they may not reach any result
    a_sc = tile_scales(e, count, K, abi().semmoe_mx4_scales_size(P, K, E), fill=255)
    b_sc = tile_scales(we, [N] * E, K, abi().semmoe_mx4_scales_size(E * N, K, E), fill=255)
    dev = (torch.from_numpy(pack(code)).cuda(), torch.from_numpy(a_sc).cuda(),
           torch.from_numpy(pack(wcode)).cuda(), torch.from_numpy(b_sc).cuda())
    return dev, oracle.mx4_values(code, e), oracle.mx4_values(wcode, we).reshape(E, N, K)


SHAPES = [  # counts per group, N, K
    ([1], 8, 32), ([5, 0, 3], 128, 256), ([127, 128, 129, 1], 264, 96), ([0, 0, 300], 520, 352),
    ([256, 257, 0, 40], 256, 1056), ([1, 0, 2, 0, 1, 700], 1000, 768),
    # groups long enough on average for pairs of CTAs: one row, one past a row tile, one past a pair
    ([600, 1, 129], 72, 32), ([1000], 264, 544), ([385, 257, 0, 513], 520, 352), ([2000, 128, 0, 0, 256], 128, 800),
]


@pytest.mark.parametrize("count,N,K", SHAPES)
def test_grouped_gemm_matches_oracle(count, N, K):
    rng = np.random.default_rng(N + K)
    E, P = len(count), sum(count)
    (a, a_sc, b, b_sc), av, bv = operands(rng, P, E, N, K, count)
    pe = rng.permutation(E)
    off = np.concatenate([[0], np.cumsum(count)])
    y = torch.full((P + 1, N), 77.0, device="cuda")
    args = (a, a_sc, cuda(off, torch.int32), cuda(pe, torch.int32), b, b_sc, P, E, N, K)
    abi().semmoe_mx4_grouped_gemm(*args, y[:P])
    assert abi().semmoe_check_errors() == 0
    ref = oracle.mx4_grouped_product(av, bv, off, pe)
    # K exact products summed in fp32: each add is off by at most one unit in the last place of a
    # partial sum, at most 2^-23 of the sum of magnitudes
    size = oracle.mx4_grouped_product(np.abs(av), np.abs(bv), off, pe)
    assert (np.abs(np_(y[:P]) - ref) <= K * 2.0 ** -23 * size).all()
    assert (np_(y[P]) == 77.0).all()
    # the bf16 output is the same sum, rounded to nearest
    z = torch.full((P + 1, N), 77.0, dtype=torch.bfloat16, device="cuda")
    abi().semmoe_mx4_grouped_gemm(*args, z[:P])
    assert torch.equal(z, y.to(torch.bfloat16))


def test_grouped_gemm_block_of_nan_reaches_its_row_only():
    rng = np.random.default_rng(3)
    count, N, K = [130, 4], 136, 192
    (a, a_sc, b, b_sc), av, bv = operands(rng, 134, 2, N, K, count)
    a_sc[scale_at(0, 129, 2, K)] = 255
    off = np.array([0, 130, 134])
    y = torch.empty(134, N, device="cuda")
    abi().semmoe_mx4_grouped_gemm(a, a_sc, cuda(off, torch.int32), cuda(np.arange(2), torch.int32), b, b_sc, 134, 2, N, K, y)
    bad = np.isnan(np_(y))
    assert bad[129].all() and not np.delete(bad, 129, axis=0).any()


def test_grouped_gemm_flags_bad_tables_and_skips_their_groups():
    from token_expert_routing_gb300 import SemMoEError
    rng = np.random.default_rng(4)
    count, N, K = [3, 2], 64, 64
    (a, a_sc, b, b_sc), av, bv = operands(rng, 5, 2, N, K, count)
    for off, pe, bit in (([0, 3, 5], [0, 2], abi().SEMMOE_DEVERR_EXPERT), ([0, 3, 9], [0, 1], abi().SEMMOE_DEVERR_PAIRS)):
        y = torch.full((5, N), 7.0, device="cuda")
        abi().semmoe_mx4_grouped_gemm(a, a_sc, cuda(np.array(off), torch.int32), cuda(np.array(pe), torch.int32), b, b_sc,
                                      5, 2, N, K, y)
        with pytest.raises(SemMoEError) as e:
            abi().semmoe_check_errors()
        assert e.value.bits == bit
        assert (np_(y[3:]) == 7.0).all()
        assert max_rel(np_(y[:3]), av[:3] @ bv[0].T) < 1e-5


@pytest.mark.parametrize("T,k_max,E,H,I,budgets", [(1, 1, 1, 32, 32, False), (1, 8, 128, 256, 96, False),
                                                   (200, 3, 7, 544, 352, True), (260, 4, 5, 1056, 160, False),
                                                   (64, 6, 64, 256, 1408, True), (1500, 2, 4, 320, 256, False),
                                                   (900, 3, 3, 1056, 480, False)])
def test_grouped_ffn_matches_oracle(T, k_max, E, H, I, budgets):
    rng = np.random.default_rng(T + H + I)
    order, back, off, count = routing(rng, T, k_max, E, budgets)
    P = len(order)
    x = cuda(rng.standard_normal((T, H)), torch.bfloat16)
    w13 = cuda(rng.standard_normal((E, 2 * I, H)) / np.sqrt(H), torch.bfloat16)
    w2 = cuda(rng.standard_normal((E, H, I)) / np.sqrt(I), torch.bfloat16)
    size = abi().semmoe_mx4_scales_size
    q13, s13 = torch.empty(E, 2 * I, H // 2, **u8), torch.empty(size(2 * E * I, H, 2 * E), **u8)
    q2, s2 = torch.empty(E, H, I // 2, **u8), torch.empty(size(E * H, I, E), **u8)
    abi().semmoe_mx4_quantize(w13, 2 * E, I, H, q13, s13)
    abi().semmoe_mx4_quantize(w2, E, H, I, q2, s2)
    xq, xs = torch.empty(P, H // 2, **u8), torch.empty(size(P, H, E), **u8)
    offd, pe = cuda(off, torch.int32), cuda(rng.permutation(E), torch.int32)
    abi().semmoe_mx4_quantize_rows(x, T, H, cuda(back, torch.int32), k_max, P, offd, E, xq, xs)
    y = torch.full((P + 1, H), 77.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.full((abi().semmoe_mx4_grouped_ffn_workspace_size(P, E, I),), 255, **u8)
    abi().semmoe_mx4_grouped_ffn(xq, xs, offd, pe, q13, s13, q2, s2, P, E, H, I, y[:P], ws)
    assert abi().semmoe_check_errors() == 0
    ref = oracle.mx4_grouped_ffn(oracle.mx4_round(np_(x))[order // k_max], oracle.mx4_round(np_(w13).reshape(-1, H)).reshape(E, 2 * I, H),
                                 oracle.mx4_round(np_(w2).reshape(-1, I)).reshape(E, H, I), off, np_(pe))
    assert max_rel(np_(y[:P]), ref) < TOL["bf16"]
    assert (np_(y[P]) == 77.0).all()
    y2 = torch.empty(P, H, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    abi().semmoe_mx4_grouped_ffn(xq, xs, offd, pe, q13, s13, q2, s2, P, E, H, I, y2, ws, side)
    side.synchronize()
    assert torch.equal(y[:P], y2)  # the same bits on every call and stream


def test_empty_inputs_enqueue_nothing():
    n0 = abi().semmoe_kernel_launches()
    e8, e32 = torch.empty(0, **u8), torch.empty(0, device="cuda")
    abi().semmoe_mx4_quantize(e32, 3, 0, 64, e8, e8)
    abi().semmoe_mx4_dequantize(e8, e8, 3, 0, 64, e32)
    assert abi().semmoe_kernel_launches() == n0


def test_quantize_past_2_31_elements():
    """Element offsets pass 32 bits: the last rows of 70000 x 32768 values."""
    rows, K = 70000, 32768
    x = torch.zeros(rows, K, dtype=torch.bfloat16, device="cuda")
    x[-130:] = torch.randn(130, K, device="cuda").to(torch.bfloat16)
    codes = torch.empty(rows, K // 2, **u8)
    scales = torch.empty(abi().semmoe_mx4_scales_size(rows, K, 1), **u8)
    abi().semmoe_mx4_quantize(x, 1, rows, K, codes, scales)
    ref_code, ref_e = oracle.mx4_encode(np_(x[-130:]))
    np.testing.assert_array_equal(unpack(codes[-130:]), ref_code)
    r, b = np.arange(rows - 130, rows)[:, None], np.arange(K // 32)[None, :]
    at = torch.from_numpy(scale_at(0, r, b, K)).cuda()
    np.testing.assert_array_equal(np_(scales[at]), ref_e)
    assert not codes[:-130].any()
    abi().semmoe_mx4_dequantize(codes, scales, 1, rows, K, x)
    np.testing.assert_array_equal(np_(x[-130:]), oracle.mx4_values(ref_code, ref_e))


def test_refuses_what_is_not_dense():
    x = torch.zeros(8, 128, device="cuda")
    codes, scales = torch.empty(8, 32, **u8), torch.empty(1024, **u8)
    with pytest.raises(ValueError, match="contiguous"):
        abi().semmoe_mx4_quantize(x[:, :64], 1, 8, 64, codes, scales)
    with pytest.raises(ValueError, match="CUDA"):
        abi().semmoe_mx4_quantize(x.cpu(), 1, 8, 64, codes, scales)


@pytest.mark.parametrize("seed", range(10))
def test_grouped_gemm_random_groups(seed):
    """Random tables: skewed, empty and one-row groups, experts in any order, ragged N and K."""
    rng = np.random.default_rng(900 + seed)
    E = int(rng.integers(1, 40))
    count = np.maximum(rng.geometric(rng.uniform(0.005, 0.3), E) - 1, 0)
    count[rng.random(E) < 0.3] = 0
    count[rng.integers(E)] += 1
    count = count.tolist()
    N, K, P = 8 * int(rng.integers(1, 70)), 32 * int(rng.integers(1, 40)), sum(count)
    (a, a_sc, b, b_sc), av, bv = operands(rng, P, E, N, K, count)
    pe, off = rng.permutation(E), np.concatenate([[0], np.cumsum(count)])
    y = torch.full((P + 1, N), 77.0, device="cuda")
    abi().semmoe_mx4_grouped_gemm(a, a_sc, cuda(off, torch.int32), cuda(pe, torch.int32), b, b_sc, P, E, N, K, y[:P])
    assert abi().semmoe_check_errors() == 0
    size = oracle.mx4_grouped_product(np.abs(av), np.abs(bv), off, pe)
    assert (np.abs(np_(y[:P]) - oracle.mx4_grouped_product(av, bv, off, pe)) <= K * 2.0 ** -23 * size).all()
    assert (np_(y[P]) == 77.0).all()


def test_rows_past_the_last_group_are_left_alone():
    """P may be more than the groups hold: the rows past them are not written, here and by the quantisation."""
    rng = np.random.default_rng(6)
    count, N, K, P = [70, 0, 60], 136, 96, 150
    (a, a_sc, b, b_sc), av, bv = operands(rng, P, 3, N, K, count + [20])
    off = np.array([0, 70, 70, 130])
    for dtype in (torch.float32, torch.bfloat16):
        y = torch.full((P, N), 77.0, dtype=dtype, device="cuda")
        abi().semmoe_mx4_grouped_gemm(a, a_sc, cuda(off, torch.int32), cuda(np.arange(3), torch.int32), b, b_sc, P, 3, N, K, y)
        assert (np_(y[130:]) == 77.0).all()
        assert max_rel(np_(y[:130]), oracle.mx4_grouped_product(av[:130], bv, off, np.arange(3))) < 1e-2
    x = torch.randn(P, 64, device="cuda")
    codes, scales = torch.full((P, 32), 0x77, **u8), torch.empty(abi().semmoe_mx4_scales_size(P, 64, 3), **u8)
    back = np.where(np.arange(P) < 130, np.arange(P), -1)
    abi().semmoe_mx4_quantize_rows(x, P, 64, cuda(back, torch.int32), 1, P, cuda(off, torch.int32), 3, codes, scales)
    assert abi().semmoe_check_errors() == 0
    assert (np_(codes[130:]) == 0x77).all()
    np.testing.assert_array_equal(unpack(codes[:130]), oracle.mx4_encode(np_(x[:130]))[0])


def test_grouped_ffn_with_a_non_finite_row():
    """A NaN or an infinity in a token's row makes that row's output NaN and no other's."""
    rng = np.random.default_rng(12)
    T, H, I, E = 140, 256, 96, 2
    x = torch.randn(T, H, device="cuda").to(torch.bfloat16)
    x[3, 7], x[139, 200] = float("nan"), float("inf")
    w13, w2 = torch.randn(E, 2 * I, H, device="cuda").to(torch.bfloat16), torch.randn(E, H, I, device="cuda").to(torch.bfloat16)
    size = abi().semmoe_mx4_scales_size
    q13, s13, q2, s2 = (torch.empty(E * 2 * I * H // 2, **u8), torch.empty(size(2 * E * I, H, 2 * E), **u8),
                        torch.empty(E * H * I // 2, **u8), torch.empty(size(E * H, I, E), **u8))
    abi().semmoe_mx4_quantize(w13, 2 * E, I, H, q13, s13)
    abi().semmoe_mx4_quantize(w2, E, H, I, q2, s2)
    off = cuda(np.array([0, 130, 140]), torch.int32)
    xq, xs, y = torch.empty(T, H // 2, **u8), torch.empty(size(T, H, E), **u8), torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(abi().semmoe_mx4_grouped_ffn_workspace_size(T, E, I), **u8)
    abi().semmoe_mx4_quantize_rows(x, T, H, cuda(np.arange(T), torch.int32), 1, T, off, E, xq, xs)
    abi().semmoe_mx4_grouped_ffn(xq, xs, off, cuda(np.arange(E), torch.int32), q13, s13, q2, s2, T, E, H, I, y, ws)
    bad = np.isnan(np_(y))
    assert bad[[3, 139]].all() and not np.delete(bad, [3, 139], axis=0).any()
