"""Which buffers the 4-bit products' outputs may share with their rows."""
import ctypes

import numpy as np
import pytest
import torch

from test_w4_cpu import _err, abi, ffn, gemm  # noqa: F401  (abi: the fixture)

X, Y, W = (ctypes.c_void_p(n << 20) for n in (1, 2, 3))  # buffers far from one another


def at(p, n):
    return ctypes.c_void_p(p.value + n)


@pytest.mark.parametrize("out,N", [(X, 256), (X, 64), (at(X, 7 * 512), 64), (at(X, -1024), 256)])
def test_a_product_lies_apart_from_its_rows(abi, out, N):  # noqa: F811
    """Rows of 256 columns (512 bytes), 8 of them: every column of a row is read for each column of out."""
    assert gemm(abi.lib(), x=X, out=out, N=N) == 1
    assert "out overlaps x" in _err(abi.lib())


@pytest.mark.parametrize("kw", [dict(ws=X), dict(ws=Y), dict(ws=at(Y, 4096 - 256)), dict(ws=at(X, -1024))])
def test_a_workspace_lies_apart_from_the_rows(abi, kw):  # noqa: F811
    assert ffn(abi.lib(), **{**dict(x=X, y=Y, ws=W), **kw}) == 1
    assert "workspace overlaps" in _err(abi.lib())


@pytest.mark.gpu
@pytest.mark.parametrize("P", [1, 6, 60, 900])
@pytest.mark.parametrize("zeros", [True, False], ids=["zeros", "symmetric"])
def test_an_ffn_over_its_own_rows(P, zeros):
    """y_perm in x's buffer: x has been read when the first row of y_perm is stored."""
    from test_gpu_w4 import abi as lib, cuda, split, weights
    rng = np.random.default_rng(P)
    E, H, I, group = 3, 640, 1408, 64
    d13, _ = weights(rng, E, 2 * I, H, group, "bf16", zeros)
    d2, _ = weights(rng, E, H, I, group, "bf16", zeros)
    off, pe = split(rng, P, E)
    tabs = cuda(off, torch.int32), cuda(pe, torch.int32)
    x = cuda(rng.standard_normal((P, H)), torch.bfloat16)
    y = torch.empty_like(x)
    lib().semmoe_w4_grouped_ffn(x, *tabs, *d13, *d2, P, E, H, I, group, y)
    for _ in range(5):
        again = x.clone()
        lib().semmoe_w4_grouped_ffn(again, *tabs, *d13, *d2, P, E, H, I, group, again)
        assert torch.equal(again, y)
    assert lib().semmoe_check_errors() == 0
