"""Groups that the 4-bit products skip: an expert id out of range, first, in the
middle or last, changes nothing in the groups around it, whose scales stay where the
offsets put them."""
import numpy as np
import pytest
import torch

import oracle
from parity_utils import TOL, max_rel, np_
from test_gpu_mx4 import abi, cuda, operands, u8

pytestmark = pytest.mark.gpu

COUNT = [130, 5, 0, 257, 64]  # 2, 1, 0, 3 and 1 row tiles


def good_rows(bad):
    off = np.concatenate([[0], np.cumsum(COUNT)])
    ok = np.ones(off[-1], dtype=bool)
    for g in bad:
        ok[off[g]:off[g + 1]] = False
    return off, ok


def flagged():
    from token_expert_routing_gb300 import SemMoEError
    with pytest.raises(SemMoEError) as e:
        abi().semmoe_check_errors()
    assert e.value.bits == abi().SEMMOE_DEVERR_EXPERT


@pytest.mark.parametrize("bad", [[0], [1], [3], [4], [0, 3], [2], [0, 1, 3, 4]])
@pytest.mark.parametrize("value", [-1, 5, 2 ** 31 - 1])
def test_grouped_gemm_skips_groups_of_bad_experts_alone(bad, value):
    rng = np.random.default_rng(31)
    E, N, K = len(COUNT), 264, 352
    off, ok = good_rows(bad)
    P = len(ok)
    (a, a_sc, b, b_sc), av, bv = operands(rng, P, E, N, K, COUNT)
    pe = rng.permutation(E)
    table = pe.copy()
    table[bad] = value
    y = torch.full((P, N), 77.0, device="cuda")
    abi().semmoe_mx4_grouped_gemm(a, a_sc, cuda(off, torch.int32), cuda(table, torch.int32), b, b_sc, P, E, N, K, y)
    flagged()
    assert (np_(y)[~ok] == 77.0).all()
    # K exact products summed in fp32: at most 2^-23 of the sum of magnitudes a step
    ref = oracle.mx4_grouped_product(av, bv, off, pe)
    size = oracle.mx4_grouped_product(np.abs(av), np.abs(bv), off, pe)
    assert (np.abs(np_(y) - ref) <= K * 2.0 ** -23 * size)[ok].all()


@pytest.mark.parametrize("bad", [[0], [3], [4], [0, 3]])
def test_grouped_ffn_skips_groups_of_bad_experts_alone(bad):
    rng = np.random.default_rng(32)
    E, H, I = len(COUNT), 544, 352
    off, ok = good_rows(bad)
    P = len(ok)
    x = cuda(rng.standard_normal((P, H)) * np.exp(rng.normal(0, 2, (P, 1))), torch.bfloat16)
    w13 = cuda(rng.standard_normal((E, 2 * I, H)) / np.sqrt(H), torch.bfloat16)
    w2 = cuda(rng.standard_normal((E, H, I)) / np.sqrt(I), torch.bfloat16)
    size = abi().semmoe_mx4_scales_size
    q13, s13 = torch.empty(E, 2 * I, H // 2, **u8), torch.empty(size(2 * E * I, H, 2 * E), **u8)
    q2, s2 = torch.empty(E, H, I // 2, **u8), torch.empty(size(E * H, I, E), **u8)
    abi().semmoe_mx4_quantize(w13, 2 * E, I, H, q13, s13)
    abi().semmoe_mx4_quantize(w2, E, H, I, q2, s2)
    offd = cuda(off, torch.int32)
    xq, xs = torch.empty(P, H // 2, **u8), torch.empty(size(P, H, E), **u8)
    abi().semmoe_mx4_quantize_rows(x, P, H, cuda(np.arange(P), torch.int32), 1, P, offd, E, xq, xs)
    pe = rng.permutation(E)
    out = []
    for skip in ([], bad):
        table = pe.copy()
        table[skip] = E
        y = torch.full((P, H), 77.0, dtype=torch.bfloat16, device="cuda")
        ws = torch.full((abi().semmoe_mx4_grouped_ffn_workspace_size(P, E, I),), 255, **u8)
        abi().semmoe_mx4_grouped_ffn(xq, xs, offd, cuda(table, torch.int32), q13, s13, q2, s2, P, E, H, I, y, ws)
        if skip:
            flagged()
        else:
            assert abi().semmoe_check_errors() == 0
        out.append(np_(y))
    assert (out[1][~ok] == 77.0).all()
    np.testing.assert_array_equal(out[1][ok], out[0][ok])  # the same bits as beside groups that are all good
    ref = oracle.mx4_grouped_ffn(oracle.mx4_round(np_(x)), oracle.mx4_round(np_(w13).reshape(-1, H)).reshape(E, 2 * I, H),
                                 oracle.mx4_round(np_(w2).reshape(-1, I)).reshape(E, H, I), off, pe)
    assert max_rel(out[1][ok], ref[ok]) < TOL["bf16"]
