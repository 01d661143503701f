"""Norms about the mean of rows whose mean is much larger than what their values differ by, against 64 bits.

Bound, with u = 2^-24 and SUMS roundings on the longest way through a sum: the mean m' that a sum in fp32 has is off by at most
em = SUMS u mean|v|.  A difference d = v - m' rounds once (u |d|), their sum has SUMS u mean|d|, and taken off them it leaves
v - m within eu = u |d| + (SUMS + 1) u mean|d|, |d| <= |v - m| + em: whatever the mean is off by, it is not in it.  The variance is
off by 2 mean(|v - m| eu) + mean(eu^2), and by twice SUMS u mean(d^2), the squares' sum and the square that is taken off it."""
import numpy as np
import pytest
import torch

from parity_utils import np_
from test_gpu_norm import SUMS, U, abi, close, cuda

pytestmark = pytest.mark.gpu
LAYER = 2


def about_mean(v, eps):
    m = v.mean(1, keepdims=True)
    em = SUMS * U * np.abs(v).mean(1, keepdims=True)
    d = np.abs(v - m) + em
    eu = U * d + (SUMS + 1) * U * d.mean(1, keepdims=True)
    var = np.square(v - m).mean(1, keepdims=True)
    evar = 2 * (np.abs(v - m) * eu).mean(1, keepdims=True) + np.square(eu).mean(1, keepdims=True) + \
        2 * SUMS * U * np.square(d).mean(1, keepdims=True)
    rho = evar / (var + eps) + 6 * U
    assert rho.max() < 0.1
    y = (v - m) / np.sqrt(var + eps)
    return y, (1 + rho) * eu / np.sqrt(var + eps) + (rho + 3 * U) * np.abs(y)


def rows(T, H, dtype, seed):
    """Constants, and values beside means of 10 to 10000."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((T, H)) + np.resize([10.0, 1e3, -1e4, 0.0], (T, 1))
    const = [100.0, 1234.5, 1e4, -12345.678, 30001.0, 0.1]
    x[::3] = np.resize(const, (len(x[::3]), 1))
    return cuda(x, dtype)


SHAPES = [(7, 64), (9, 1000), (6, 1060), (12, 2048), (5, 8192), (1300, 136), (1300, 520), (2500, 1000), (1300, 2056)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,H", SHAPES)
def test_norm_of_rows_far_from_zero(T, H, dtype):
    if dtype == torch.bfloat16:
        H -= H % 8
    x = rows(T, H, dtype, T + H)
    out = torch.empty_like(x)
    eps = 1e-6
    abi().semmoe_norm(x, T, H, LAYER, None, None, 0.0, eps, out)
    ref, err = about_mean(np_(x).astype(np.float64), float(np.float32(eps)))
    close(out, ref, err)
    assert abi().semmoe_check_errors() == 0


@pytest.mark.parametrize("maps", [False, True], ids=["dense", "slots"])
@pytest.mark.parametrize("T,H", SHAPES)
def test_norms_of_a_combine_far_from_zero(T, H, maps):
    """The row itself normalised after the block; and the residual alone, the block's rows times 0, before the next."""
    x = rows(T, H, torch.float32, T * H)
    ident = torch.arange(T, dtype=torch.int32, device="cuda") if maps else None
    ones = torch.ones(T, 1, device="cuda") if maps else None
    eps = 1e-6
    ref, err = about_mean(np_(x).astype(np.float64), float(np.float32(eps)))
    out, nxt = torch.empty_like(x), torch.empty_like(x)
    abi().semmoe_combine_norm(x, ident, ones, None, T, H, int(maps), T, LAYER, None, None, 0, None, None, 0.0, eps, None, 0, 1.0,
                              None, 1.0, out)
    close(out, ref, err)
    abi().semmoe_combine_norm(x.clone(), ident, ones, None, T, H, int(maps), T, 0, None, None, LAYER, None, None, 0.0, eps, None, 0,
                              0.0, x, 1.0, out, nxt)
    assert torch.equal(out, x)
    close(nxt, ref, err)
    assert abi().semmoe_check_errors() == 0


CONSTANTS = [1e-40, 1e-20, 0.1, 100.0, 1234.5, -123456.7, 1e19, -3.3e25, 1e30, 3e38]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,H", SHAPES + [(20, 16384 // 2)])
def test_constant_rows_are_zeros(T, H, dtype):
    """The differences from the mean that fp32 has are equal and at most SUMS steps of the value, so their sum (below 2^24 such
    steps) and its quotient by H are exact, and what is left is 0: the output is the bias."""
    if dtype == torch.bfloat16:
        H -= H % 8
    x = cuda(np.resize(CONSTANTS, (T, 1)) * np.ones((1, H)), dtype)
    bias = cuda(np.random.default_rng(H).standard_normal(H), dtype)
    out, nxt = torch.empty_like(x), torch.empty_like(x)
    abi().semmoe_norm(x, T, H, LAYER, None, bias, 0.0, 1e-6, out)
    assert torch.equal(out, bias.expand(T, H))
    abi().semmoe_combine_norm(x, None, None, None, T, H, 0, T, LAYER, None, bias, 0, None, None, 0.0, 1e-6, None, 0, 1.0, None, 1.0,
                              out)
    assert torch.equal(out, bias.expand(T, H))
    zero = torch.zeros_like(x)
    abi().semmoe_combine_norm(zero, None, None, None, T, H, 0, T, 0, None, None, LAYER, None, bias, 0.0, 1e-6, None, 0, 1.0, x, 1.0,
                              out, nxt)
    assert torch.equal(out, x) and torch.equal(nxt, bias.expand(T, H))
    assert abi().semmoe_check_errors() == 0


@pytest.mark.parametrize("value", [1e4, 1e19, 1e30, 3e38])
@pytest.mark.parametrize("H", [64, 136, 520])
def test_one_value_a_step_beside_the_others(H, value):
    """Differences are k and k + 1 steps, |k| <= SUMS: sums exact, the variance (1 - 1 / H) / H of a step's square but for three
    roundings of k^2, and the mean's rest off by one rounding of k."""
    T, eps = 9, 1e-30
    x = np.full((T, H), np.float32(value))
    at = np.arange(T) * (H // T)
    x[np.arange(T), at] = np.nextafter(np.float32(value), np.float32(np.inf))
    out = torch.empty(T, H, device="cuda")
    abi().semmoe_norm(cuda(x, torch.float32), T, H, LAYER, None, None, 0.0, eps, out)
    ref = np.full((T, H), -1 / np.sqrt(H - 1))
    ref[np.arange(T), at] = np.sqrt(H - 1)
    rho = 3 * U * SUMS ** 2 * H
    assert rho < 0.5
    assert (np.abs(np_(out) - ref) <= rho * np.abs(ref) + SUMS * U * np.sqrt(H)).all()
    assert abi().semmoe_check_errors() == 0
