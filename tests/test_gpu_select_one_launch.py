"""The choice by score in the launch that makes its logits (up to 1024 tokens and two passes of
experts): one CTA and several a token tile, a ragged second pass, both scores, budgets, more than
32 picks, and what is not finite or out of range, against the oracle on the same logits."""
import numpy as np
import pytest
import torch

import oracle
from parity_utils import LOGIT_TOL, max_rel, np_
from test_gpu_select import W_RTOL, abi, decided, i32

pytestmark = pytest.mark.gpu


def inputs(rng, T, H, E, wd):
    x = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).to(torch.bfloat16).cuda()
    w = torch.from_numpy((rng.standard_normal((E, H)) / np.sqrt(H)).astype(np.float32))
    return x, w.to(torch.bfloat16 if wd == "bf16" else torch.float32).cuda()


def run(x, w, score, k, k_max, bias=None, G=1, keep=1, top=1, renorm=True, scale=1.0):
    """Picks, weights, logits and the count table; k: a budget for all, or one a token."""
    T, H = x.shape
    E = w.shape[0]
    idx, gw = torch.full((T, k_max), -7, **i32), torch.full((T, k_max), 7.0, device="cuda")
    logits = torch.full((T, E), 7.0, device="cuda")
    pc = torch.full((E, abi().semmoe_pair_counts_stride(T)), -3, **i32)
    kpt = None if np.isscalar(k) else torch.from_numpy(np.asarray(k, dtype=np.int32)).cuda()
    b = None if bias is None else torch.from_numpy(np.asarray(bias, dtype=np.float32)).cuda()
    code = abi().SEMMOE_SCORE_SIGMOID if score == "sigmoid" else abi().SEMMOE_SCORE_SOFTMAX
    n0 = abi().semmoe_kernel_launches()
    abi().semmoe_route_select(x, w, None, logits, code, b, G, keep, top, renorm, scale, kpt, k if kpt is None else 0, T, H,
                              E, k_max, idx, gw, pair_counts=pc)
    # one launch, behind the one that splits an fp32 weight
    assert abi().semmoe_kernel_launches() - n0 == (1 if w.dtype == torch.bfloat16 else 2)
    return np_(idx), np_(gw), np_(logits), np_(pc)


def check(idx, w, logits, pc, x, wr, score, k, k_max, bias=None, G=1, keep=1, top=1, renorm=True, scale=1.0, rows=None):
    T, E = logits.shape
    rows = np.ones(T, dtype=bool) if rows is None else rows
    assert max_rel(logits[rows], oracle.router_logits(x, wr)[rows]) < LOGIT_TOL
    kt = np.full(T, k) if np.isscalar(k) else np.clip(k, 1, k_max)
    l = np.where(rows[:, None], logits, 0.0)
    ref_idx, ref_w = oracle.route_select(l, score, kt, k_max, bias, G, keep, top, renorm, scale)
    ok = decided(l, score, k_max, bias, G, keep, top) & rows
    assert ok.sum() >= 0.9 * rows.sum()
    np.testing.assert_array_equal(idx[ok], ref_idx[ok])
    np.testing.assert_allclose(w[ok], ref_w[ok], rtol=W_RTOL)
    table = np.zeros(pc.shape, dtype=np.int64)
    t, j = np.nonzero(idx >= 0)
    np.add.at(table, (idx[t, j], t // 128), 1)
    np.testing.assert_array_equal(pc, table)
    # rows that hang on the last bits too: as many distinct experts as the oracle takes, of kept groups
    for r in np.nonzero(rows & ~ok)[0]:
        live = idx[r][idx[r] >= 0]
        assert len(set(live)) == len(live) == (ref_idx[r] >= 0).sum()
        assert len(set(live // (E // G))) <= keep


CASES = [  # T, H, E, weight, k_max, groups, kept, group_top, bias
    (1, 8, 1, "bf16", 1, 1, 1, 1, False), (1, 64, 100, "bf16", 8, 4, 2, 2, True), (129, 192, 128, "bf16", 8, 8, 4, 2, True),
    (1000, 8, 128, "bf16", 6, 1, 1, 1, True), (1000, 192, 100, "f32", 40, 1, 1, 1, False), (129, 64, 1, "f32", 1, 1, 1, 1, True),
    (1000, 64, 64, "f32", 6, 8, 3, 1, False), (1, 2048, 128, "f32", 8, 4, 3, 2, True), (130, 2048, 100, "f32", 12, 25, 9, 1, True),
    (1, 2048, 255, "bf16", 8, 5, 2, 2, True), (1024, 512, 129, "bf16", 6, 3, 2, 2, False), (777, 264, 200, "bf16", 24, 100, 50, 2, True),
    (129, 2048, 255, "bf16", 70, 1, 1, 1, True), (1000, 1000, 144, "bf16", 33, 12, 8, 1, False), (64, 136, 256, "bf16", 200, 1, 1, 1, False),
    (1024, 256, 16, "bf16", 4, 16, 7, 1, True),
]


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("budgets,renorm,scale", [(False, True, 1.0), (True, True, 2.5), (True, False, 1.0)])
@pytest.mark.parametrize("T,H,E,wd,k_max,G,keep,top,with_bias", CASES)
def test_choice_in_one_launch(T, H, E, wd, k_max, G, keep, top, with_bias, score, budgets, renorm, scale):
    rng = np.random.default_rng(T + 3 * H + 7 * E)
    x, w = inputs(rng, T, H, E, wd)
    b = (rng.standard_normal(E) * 0.1).astype(np.float32) if with_bias else None
    k = rng.integers(1, k_max + 1, T) if budgets else k_max
    out = run(x, w, score, k, k_max, b, G, keep, top, renorm, scale)
    assert abi().semmoe_check_errors() == 0
    check(*out, x, w, score, k, k_max, b, G, keep, top, renorm, scale)


@pytest.mark.parametrize("H", [64, 2048])
@pytest.mark.parametrize("E,wd", [(100, "f32"), (200, "bf16")])
def test_experts_switched_off(E, wd, H):
    """-inf biases: a group that is off, and tokens with fewer experts left than their budget."""
    rng = np.random.default_rng(E + H)
    T, G = 300, 10
    x, w = inputs(rng, T, H, E, wd)
    b = (rng.standard_normal(E) * 0.1).astype(np.float32)
    b[:E // G] = -np.inf
    b[E // G:E // 2:2] = -np.inf
    out = run(x, w, "sigmoid", 8, 8, b, G, 4, 2)
    assert abi().semmoe_check_errors() == 0
    check(*out, x, w, "sigmoid", 8, 8, b, G, 4, 2)
    b[:] = -np.inf
    b[[3, E - 1, E // 2]] = 0.25
    out = run(x, w, "softmax", 8, 8, b)
    assert abi().semmoe_check_errors() == 0
    assert (out[0][:, 3:] == -1).all() and (out[0][:, :3] >= 0).all()
    check(*out, x, w, "softmax", 8, 8, b)


@pytest.mark.parametrize("H", [64, 2048])
@pytest.mark.parametrize("E,wd", [(64, "f32"), (200, "bf16")])
def test_flags_rows_that_are_not_finite(E, wd, H):
    """A NaN or an infinity in a token's row: its picks are padding or finite, the flag is set, other rows stay."""
    from token_expert_routing_gb300 import SemMoEError
    rng = np.random.default_rng(E)
    T = 140
    x, w = inputs(rng, T, H, E, wd)
    x[5, 3] = float("nan")
    x[129, H - 1] = float("nan")
    idx, gw, logits, pc = run(x, w, "sigmoid", 4, 4)
    with pytest.raises(SemMoEError) as e:
        abi().semmoe_check_errors()
    assert e.value.bits == abi().SEMMOE_DEVERR_NONFINITE
    rows = np.ones(T, dtype=bool)
    rows[[5, 129]] = False
    assert np.isnan(logits[~rows]).all() and (idx[~rows] == -1).all() and (gw[~rows] == 0).all()
    check(idx, gw, logits, pc, x, w, "sigmoid", 4, 4, rows=rows)


@pytest.mark.parametrize("H", [64, 2048])
def test_flags_budgets_out_of_range(H):
    """Budgets of 0 and past k_max are flagged and taken as 1 and k_max."""
    from token_expert_routing_gb300 import SemMoEError
    rng = np.random.default_rng(H)
    T, E, k_max = 200, 128, 6
    x, w = inputs(rng, T, H, E, "bf16")
    k = rng.integers(1, k_max + 1, T)
    k[[0, 130]], k[[7, 199]] = 0, k_max + 1
    out = run(x, w, "softmax", k, k_max, renorm=False)
    with pytest.raises(SemMoEError) as e:
        abi().semmoe_check_errors()
    assert e.value.bits == abi().SEMMOE_DEVERR_K
    check(*out, x, w, "softmax", k, k_max, renorm=False)


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_flags_biases_that_are_not_finite(value):
    from token_expert_routing_gb300 import SemMoEError
    rng = np.random.default_rng(17)
    T, E = 130, 96
    x, w = inputs(rng, T, 512, E, "bf16")
    b = (rng.standard_normal(E) * 0.1).astype(np.float32)
    b[40] = value
    out = run(x, w, "sigmoid", 5, 5, b)
    with pytest.raises(SemMoEError) as e:
        abi().semmoe_check_errors()
    assert e.value.bits == abi().SEMMOE_DEVERR_NONFINITE
    off = b.copy()
    off[40] = -np.inf
    check(*out, x, w, "sigmoid", 5, 5, off)


@pytest.mark.parametrize("case", range(4))
def test_layer_rows_differ_only_where_they_hang_on_the_last_bits(case):
    """The layer's picks, row by row: equal to the oracle's wherever no decision is within the scores' error of a tie."""
    import workloads as wl
    from test_gpu_layer_select_mx4 import CASES as LAYERS, api, layer_of
    name, over, sel = LAYERS[case]
    d = wl.make_inputs(wl.scaled(name, **over))
    s = d["spec"]
    bias = (0.1 * np.random.default_rng(9).standard_normal(s.E)).astype(np.float32)
    select = api().RouteSelect(bias=torch.from_numpy(bias), **sel)
    layer = layer_of(d, select=select, fused_gather=False)
    k = d["k_per_token"].numpy()
    res = layer.forward(d["x"].cuda(), d["token_ids"].cuda(), d["k_per_token"].cuda() if s.k_choices else None,
                        None if s.k_choices else s.k, int(k.sum()), keep_logits=True)
    api()._abi.semmoe_check_errors()
    l = np_(res.logits)
    G, keep, top = select.n_group, select.topk_group, select.group_top
    ref_idx, ref_w = oracle.route_select(l, select.score, k, s.k_max, bias, G, keep, top, select.renorm, select.scale)
    ok = decided(l, select.score, s.k_max, bias, G, keep, top)
    assert ok.mean() > 0.9
    np.testing.assert_array_equal(np_(res.topk_idx)[ok], ref_idx[ok])
    np.testing.assert_allclose(np_(res.topk_w)[ok], ref_w[ok], rtol=W_RTOL)
