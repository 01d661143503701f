"""4-bit products at the ends of a row's groups: what lies beside the scales and zero points takes no part.

Whole rows and scales that are powers of two, so that every sum is exact in fp32 and only the output rounds."""
import numpy as np
import pytest
import torch

import oracle
from parity_utils import np_
from test_gpu_w4 import DT, U8, abi, cuda, pack, product, split

pytestmark = pytest.mark.gpu

# (group, K): rows of fewer groups than 128 columns have, rows that end inside 128 columns, whole ones
ENDS = [(32, 32), (32, 64), (32, 96), (32, 128), (32, 160), (32, 352), (32, 576), (64, 64), (64, 128), (64, 192), (64, 704),
        (128, 128), (128, 640), (256, 256)]
# P, E, N: a few rows; more rows than the form of a few rows takes
SIZES = [(2, 1, 40), (5, 3, 72), (100, 2, 136), (600, 2, 136)]


def inside(t, fill):
    """t's values in a buffer that begins 16 bytes into a larger one, whose other elements are `fill`."""
    n = 16 // t.element_size()
    big = torch.full((t.numel() + 64 * n,), fill, dtype=t.dtype, device="cuda")
    view = big[n:n + t.numel()].reshape(t.shape)
    view.copy_(t)
    return view


def matrices(rng, E, rows, K, group, scale, zeros, bad=None):
    """(device tuple, values [E, rows, K]); bad: (matrix, row) whose scales are NaN.  The scales lie between NaN, the zero points
    between 255."""
    code = rng.integers(0, 16, (E, rows, K))
    s = np.exp2(rng.integers(-3, 2, (E, rows, K // group)))
    z = rng.integers(0, 16, (E, rows, K // group)) if zeros else None
    w = oracle.w4_values(code, s, z, group)
    if bad is not None:
        s[bad] = np.nan
    return (cuda(pack(code), torch.uint8), inside(cuda(s, DT[scale]), float("nan")),
            None if z is None else inside(cuda(z, torch.uint8), 255)), w


@pytest.mark.parametrize("zeros", [True, False], ids=["zeros", "symmetric"])
@pytest.mark.parametrize("scale", ["bf16", "f32"])
@pytest.mark.parametrize("P,E,N", SIZES)
@pytest.mark.parametrize("group,K", ENDS)
def test_a_row_reads_its_own_scales(group, K, P, E, N, scale, zeros):
    rng = np.random.default_rng(K + P + group)
    off, pe = split(rng, P, E)
    x = rng.integers(-4, 5, (P, K)).astype(np.float64)
    dev, w = matrices(rng, E, N, K, group, scale, zeros, bad=(E - 1, 3))
    out = torch.full((P + 1, N), 7.0, dtype=torch.bfloat16, device="cuda")
    product(cuda(x, torch.bfloat16), dev, off, pe, P, E, N, K, group, out)
    ref = oracle.bf16_round(oracle.w4_grouped_product(x, w, off, pe))
    b = int(np.argwhere(pe == E - 1)[0, 0])
    ref[off[b]:off[b + 1], 3] = np.nan
    np.testing.assert_array_equal(np_(out[:P]), ref)
    assert bool((out[P] == 7).all())
    assert abi().semmoe_check_errors() == 0


@pytest.mark.parametrize("P,E", [(1, 1), (6, 3), (120, 2)])
@pytest.mark.parametrize("zeros", [True, False], ids=["zeros", "symmetric"])
@pytest.mark.parametrize("H,I,group", [(32, 32, 32), (96, 64, 32), (64, 96, 32), (160, 96, 32), (64, 64, 64), (192, 64, 64)])
def test_ffn_reads_its_own_scales(H, I, group, zeros, P, E):
    """Equal bit for bit with the same matrices in buffers whose neighbours are finite."""
    rng = np.random.default_rng(H + I + P)
    off, pe = split(rng, P, E)
    tabs = cuda(off, torch.int32), cuda(pe, torch.int32)
    x = cuda(rng.standard_normal((P, H)), torch.bfloat16)
    d13, _ = matrices(rng, E, 2 * I, H, group, "bf16", zeros)
    d2, _ = matrices(rng, E, H, I, group, "bf16", zeros)
    got = []
    for move in (lambda t, fill: t, inside):
        args = [None if t is None else move(t.clone(), f) for d in (d13, d2) for t, f in zip(d, (0, 1.0, 8))]
        y = torch.empty(P, H, dtype=torch.bfloat16, device="cuda")
        ws = torch.empty(abi().semmoe_w4_grouped_ffn_workspace_size(P, I), **U8)
        abi().semmoe_w4_grouped_ffn(x, *tabs, *args, P, E, H, I, group, y, ws)
        got.append(y)
    y = torch.empty_like(got[0])
    abi().semmoe_w4_grouped_ffn(x, *tabs, *d13, *d2, P, E, H, I, group, y)
    assert bool(torch.isfinite(y).all())
    assert torch.equal(y, got[0]) and torch.equal(y, got[1])
    assert abi().semmoe_check_errors() == 0


@pytest.mark.parametrize("zeros", [True, False], ids=["zeros", "symmetric"])
@pytest.mark.parametrize("P,E,N", SIZES)
@pytest.mark.parametrize("group,K", [(32, 96), (32, 160), (32, 512), (64, 704), (128, 640), (128, 1024), (256, 256)])
def test_an_infinite_scale_of_the_last_group(group, K, P, E, N, zeros):
    """Codes above the zero point and rows of one sign: the sums are infinite, of the row's sign, wherever the columns end."""
    rng = np.random.default_rng(K + P)
    off, pe = split(rng, P, E)
    code = rng.integers(9, 16, (E, N, K))
    s = np.exp2(rng.integers(-3, 2, (E, N, K // group)))
    z = rng.integers(0, 8, (E, N, K // group)) if zeros else None
    w = oracle.w4_values(code, s, z, group)
    s[:, 5, -1] = np.inf
    dev = cuda(pack(code), torch.uint8), cuda(s, torch.float32), None if z is None else cuda(z, torch.uint8)
    sign = np.where(np.arange(P) % 2, -1, 1)
    x = rng.integers(1, 3, (P, K)) * sign[:, None].astype(np.float64)
    out = torch.empty(P, N, dtype=torch.bfloat16, device="cuda")
    product(cuda(x, torch.bfloat16), dev, off, pe, P, E, N, K, group, out)
    ref = oracle.bf16_round(oracle.w4_grouped_product(x, w, off, pe))
    ref[:, 5] = np.inf * sign
    np.testing.assert_array_equal(np_(out), ref)
    assert abi().semmoe_check_errors() == 0


@pytest.mark.parametrize("zeros", [True, False], ids=["zeros", "symmetric"])
@pytest.mark.parametrize("scale", ["bf16", "f32"])
@pytest.mark.parametrize("P,E,N", SIZES)
@pytest.mark.parametrize("group,K", [(32, 96), (32, 352), (64, 704), (128, 640), (128, 2048), (256, 1024)])
def test_large_values_on_weights_of_zero(group, K, P, E, N, scale, zeros):
    """Rows with values of 2^22 in columns whose codes are the zero point: weights of 0, whatever the value, so the sums stay
    those of the other columns, whole numbers below 2^24."""
    rng = np.random.default_rng(K + P)
    off, pe = split(rng, P, E)
    code = rng.integers(0, 16, (E, N, K))
    z = rng.integers(0, 16, (E, N, K // group)) if zeros else None
    s = np.ones((E, N, K // group))
    large = [1, K // 2, K - 3]
    for c in large:
        code[:, :, c] = 8 if z is None else z[:, :, c // group]
    w = oracle.w4_values(code, s, z, group)
    x = rng.integers(-4, 5, (P, K)).astype(np.float64)
    x[:, large] = 2.0 ** 22 * rng.choice([-1, 1, 0.75], (P, len(large)))
    dev = cuda(pack(code), torch.uint8), cuda(s, DT[scale]), None if z is None else cuda(z, torch.uint8)
    out = torch.empty(P, N, dtype=torch.bfloat16, device="cuda")
    product(cuda(x, torch.bfloat16), dev, off, pe, P, E, N, K, group, out)
    np.testing.assert_array_equal(np_(out), oracle.bf16_round(oracle.w4_grouped_product(x, w, off, pe)))
    assert abi().semmoe_check_errors() == 0
