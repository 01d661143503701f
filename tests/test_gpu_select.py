"""GPU parity of the expert choice by score (semmoe_route_select): picks equal
to the oracle's wherever the choice does not hang on the last bits of fp32
scores, ties exact, weights within the bound of their fp32 arithmetic."""
import numpy as np
import pytest
import torch

import oracle
from parity_utils import LOGIT_TOL, max_rel, np_

pytestmark = pytest.mark.gpu

i32 = dict(dtype=torch.int32, device="cuda")

#: scores: an exponential (2 ulp), a sum, a division and the bias's addition, each half an ulp of at most 1
SCORE_ERR = 2.0 ** -21
#: weights: differences of logs of magnitude <= 16 rounded thrice (3 * 16 * 2^-24), the exponentials, k <= 40
#: terms of the sum, a division and the scale: under 1e-5 of the weight
W_RTOL = 1e-5


def abi():
    from token_expert_routing_gb300 import _abi
    return _abi


def run(logits, score, k, k_max, bias=None, G=1, keep=1, top=1, renorm=True, scale=1.0, per_token=True, counts=False):
    T, E = logits.shape
    idx = torch.full((T, k_max), -7, **i32)
    w = torch.full((T, k_max), 7.0, device="cuda")
    pc = torch.full((E, abi().semmoe_pair_counts_stride(T)), -3, **i32) if counts else None
    kpt = torch.from_numpy(np.asarray(k, dtype=np.int32)).cuda() if per_token else None
    b = None if bias is None else torch.from_numpy(np.asarray(bias, dtype=np.float32)).cuda()
    code = abi().SEMMOE_SCORE_SIGMOID if score == "sigmoid" else abi().SEMMOE_SCORE_SOFTMAX
    abi().semmoe_route_select(None, None, torch.from_numpy(logits).cuda(), None, code, b, G, keep, top, renorm, scale,
                              kpt, 0 if per_token else int(k[0]), T, 0, E, k_max, idx, w, pair_counts=pc)
    return np_(idx), np_(w), None if pc is None else np_(pc)


def decided(logits, score, k_max, bias, G, keep, top):
    """Tokens none of whose decisions (group, pick, order of picks) is within the scores' error of a tie."""
    T, E = logits.shape
    ok = np.ones(T, dtype=bool)
    s = oracle.scores(logits, score)
    c = s if bias is None else s + np.asarray(bias, dtype=np.float64)
    if keep < G:
        g = np.sort(c.reshape(T, G, -1), axis=2)[:, :, ::-1][:, :, :top]
        g = np.sort(np.where(np.isneginf(g), 0, g).sum(axis=2), axis=1)[:, ::-1]
        ok &= g[:, keep - 1] - g[:, keep] > 2 * top * SCORE_ERR
    if bias is not None:
        t = -np.sort(-oracle.choice_scores(logits, score, bias, G, keep, top), axis=1)[:, :k_max + 1]
        with np.errstate(invalid="ignore"):
            gap = t[:, :-1] - t[:, 1:]
        ok &= ((gap > 2 * SCORE_ERR) | np.isneginf(t[:, 1:])).all(axis=1)
    return ok


CASES = [  # E, k_max, groups, kept, group_top, bias
    (8, 2, 1, 1, 1, False), (16, 4, 4, 2, 2, True), (64, 6, 8, 3, 1, False), (256, 8, 8, 4, 2, True),
    (128, 8, 1, 1, 1, True), (36, 5, 12, 5, 2, True), (250, 12, 25, 9, 1, True), (256, 40, 64, 32, 2, False),
    (1, 1, 1, 1, 2, True), (6, 3, 6, 3, 2, True), (200, 24, 100, 50, 2, True),
]


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm,scale", [(True, 2.5), (False, 1.0)])
@pytest.mark.parametrize("E,k_max,G,keep,top,bias", CASES)
def test_select_from_logits(E, k_max, G, keep, top, bias, score, renorm, scale):
    rng = np.random.default_rng(E * 10 + k_max)
    T = 700
    l = (rng.standard_normal((T, E)) * 2).astype(np.float32)
    b = (rng.standard_normal(E) * 0.1).astype(np.float32) if bias else None
    k = rng.integers(1, k_max + 1, T)
    idx, w, pc = run(l, score, k, k_max, b, G, keep, top, renorm, scale, counts=True)
    assert abi().semmoe_check_errors() == 0
    ref_idx, ref_w = oracle.route_select(l, score, k, k_max, b, G, keep, top, renorm, scale)
    ok = decided(l, score, k_max, b, G, keep, top)
    assert ok.mean() > 0.95
    np.testing.assert_array_equal(idx[ok], ref_idx[ok])
    np.testing.assert_allclose(w[ok], ref_w[ok], rtol=W_RTOL)
    # every token: distinct experts of kept groups, descending, and the count table of the picks
    table = np.zeros_like(pc)
    for t in range(T):
        live = idx[t, :k[t]]
        assert (live >= 0).all() and len(set(live)) == k[t] and (idx[t, k[t]:] == -1).all() and (w[t, k[t]:] == 0).all()
        assert len(set(live // (E // G))) <= keep
        np.add.at(table, (live, t // 128), 1)
    np.testing.assert_array_equal(pc, table)


def test_select_ties_keep_the_lower_group_and_expert():
    """Equal logits and biases give equal scores bit for bit."""
    rng = np.random.default_rng(7)
    T, E, G = 1000, 32, 8
    l = rng.integers(-2, 3, (T, E)).astype(np.float32)
    l[:, 3] = -0.0
    for score in ("sigmoid", "softmax"):
        # without a bias the order is the logits', ties and all; groups score their single best
        k = np.full(T, 6)
        idx, w, _ = run(l, score, k, 6, None, G, 4, 1, per_token=False)
        best = l.reshape(T, G, 4).max(axis=2)
        order = np.argsort(-best, axis=1, kind="stable")[:, :4]
        kept = np.zeros((T, G), dtype=bool)
        np.put_along_axis(kept, order, True, axis=1)
        left = np.where(np.repeat(kept, 4, axis=1), l, -np.inf)
        np.testing.assert_array_equal(idx, np.argsort(-left, axis=1, kind="stable")[:, :6])


def test_select_experts_switched_off():
    """-inf biases: never taken, nothing to their group, and padding where too few are left."""
    rng = np.random.default_rng(8)
    T, E, G = 300, 16, 4
    l = rng.standard_normal((T, E)).astype(np.float32)
    b = np.zeros(E, dtype=np.float32)
    b[[0, 1, 2, 3, 5, 6, 7, 9, 13]] = -np.inf       # group 0 off, group 1 down to expert 4
    idx, w, _ = run(l, "sigmoid", np.full(T, 6), 6, b, G, 3, 2)
    assert abi().semmoe_check_errors() == 0
    ref_idx, ref_w = oracle.route_select(l, "sigmoid", np.full(T, 6), 6, b, G, 3, 2)
    ok = decided(l, "sigmoid", 6, b, G, 3, 2)
    assert ok.mean() > 0.95
    np.testing.assert_array_equal(idx[ok], ref_idx[ok])
    np.testing.assert_allclose(w[ok], ref_w[ok], rtol=W_RTOL)
    b[:] = -np.inf
    idx, w, pc = run(l, "softmax", np.full(T, 6), 6, b, G, 3, 2, counts=True)
    assert (idx == -1).all() and (w == 0).all() and (pc == 0).all()
    b[10] = 0
    idx, w, _ = run(l, "sigmoid", np.full(T, 3), 3, b, G, 2, 2, True, 1.5)
    assert (idx[:, 0] == 10).all() and (idx[:, 1:] == -1).all() and (w[:, 0] == 1.5).all() and (w[:, 1:] == 0).all()
    assert abi().semmoe_check_errors() == 0


@pytest.mark.parametrize("where", ["logit", "bias nan", "bias inf"])
def test_select_flags_what_is_not_finite(where):
    from token_expert_routing_gb300 import SemMoEError
    l = np.tile(np.linspace(-1, 1, 8, dtype=np.float32), (3, 1))
    b = np.zeros(8, dtype=np.float32)
    if where == "logit":
        l[1, 7] = np.nan
    else:
        b[7] = np.nan if "nan" in where else np.inf
    idx, w, _ = run(l, "sigmoid", np.full(3, 2), 2, b)
    with pytest.raises(SemMoEError) as e:
        abi().semmoe_check_errors()
    assert e.value.bits == abi().SEMMOE_DEVERR_NONFINITE
    assert idx.tolist() == ([[7, 6], [6, 5], [7, 6]] if where == "logit" else [[6, 5]] * 3)
    assert np.isfinite(w).all()


def test_select_weights_of_scores_that_underflow():
    """Sigmoid scores of -200 and -201 are 0 in fp32; their renormalised weights are not."""
    l = np.full((1, 8), -300.0, dtype=np.float32)
    l[0, 2], l[0, 5] = -200.0, -201.0
    idx, w, _ = run(l, "sigmoid", [2], 2)
    assert idx.tolist() == [[2, 5]]
    np.testing.assert_allclose(w[0], [1 / (1 + np.exp(-1)), 1 / (1 + np.exp(1))], rtol=W_RTOL)


@pytest.mark.parametrize("T,H,E,xd,wd", [(1, 2048, 256, "bf16", "bf16"), (129, 264, 64, "bf16", "f32"),
                                         (1000, 512, 128, "bf16", "f32"), (40, 100, 24, "f32", "f32"),
                                         (33, 100, 24, "bf16", "bf16"), (12000, 64, 48, "bf16", "f32"),
                                         (11000, 128, 128, "bf16", "bf16")])
def test_select_with_its_router_product(T, H, E, xd, wd):
    rng = np.random.default_rng(T + E)
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}
    x = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).to(dt[xd]).cuda()
    wr = torch.from_numpy((rng.standard_normal((E, H)) / np.sqrt(H)).astype(np.float32)).to(dt[wd]).cuda()
    b = torch.from_numpy((rng.standard_normal(E) * 0.1).astype(np.float32)).cuda()
    k_max = 4
    idx, w = torch.empty(T, k_max, **i32), torch.empty(T, k_max, device="cuda")
    logits = torch.empty(T, E, device="cuda")
    pc = torch.full((E, abi().semmoe_pair_counts_stride(T)), -3, **i32)
    abi().semmoe_route_select(x, wr, None, logits, abi().SEMMOE_SCORE_SIGMOID, b, 4, 2, 2, True, 1.0, None, k_max, T, H, E,
                              k_max, idx, w, pair_counts=pc)
    assert abi().semmoe_check_errors() == 0
    l = np_(logits)
    assert max_rel(l, oracle.router_logits(x, wr)) < LOGIT_TOL
    ref_idx, ref_w = oracle.route_select(l, "sigmoid", np.full(T, k_max), k_max, np_(b), 4, 2, 2)
    ok = decided(l, "sigmoid", k_max, np_(b), 4, 2, 2)
    assert ok.mean() > 0.95
    np.testing.assert_array_equal(np_(idx)[ok], ref_idx[ok])
    np.testing.assert_allclose(np_(w)[ok], ref_w[ok], rtol=W_RTOL)
    table = np.zeros(pc.shape, dtype=np.int64)
    np.add.at(table, (np_(idx), np.repeat(np.arange(T)[:, None] // 128, k_max, axis=1)), 1)
    np.testing.assert_array_equal(np_(pc), table)
    # the same picks without the logits written
    idx2, w2 = torch.empty_like(idx), torch.empty_like(w)
    abi().semmoe_route_select(x, wr, None, None, abi().SEMMOE_SCORE_SIGMOID, b, 4, 2, 2, True, 1.0, None, k_max, T, H, E,
                              k_max, idx2, w2)
    assert torch.equal(idx, idx2) and torch.equal(w, w2)


@pytest.mark.parametrize("T,H,E,wd", [(1300, 512, 256, torch.float32), (1025, 264, 200, torch.float32),
                                      (2100, 1024, 100, torch.bfloat16)])
def test_select_count_table_of_calls_in_a_row(T, H, E, wd):
    rng = np.random.default_rng(T)
    xs = [torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).to(torch.bfloat16).cuda() for _ in range(4)]
    wr = torch.from_numpy((rng.standard_normal((E, H)) / np.sqrt(H)).astype(np.float32)).to(wd).cuda()
    k_max = 5
    pc = torch.full((E, abi().semmoe_pair_counts_stride(T)), -3, **i32)  # one table and one workspace for all
    ws = torch.empty(abi().semmoe_route_select_workspace_size(T, H, E, abi().SEMMOE_BF16, abi().dtype_code(wr)),
                     dtype=torch.uint8, device="cuda")
    out = []
    for x in xs:
        idx, w = torch.empty(T, k_max, **i32), torch.empty(T, k_max, device="cuda")
        abi().semmoe_route_select(x, wr, None, None, abi().SEMMOE_SCORE_SOFTMAX, None, 1, 1, 1, True, 1.0, None, k_max,
                                  T, H, E, k_max, idx, w, ws=ws, pair_counts=pc)
        out.append((idx, pc.clone()))
    assert abi().semmoe_check_errors() == 0
    for x, (idx, counts) in zip(xs, out):
        table = np.zeros(counts.shape, dtype=np.int64)
        np.add.at(table, (np_(idx), np.repeat(np.arange(T)[:, None] // 128, k_max, axis=1)), 1)
        np.testing.assert_array_equal(np_(counts), table)


def test_select_on_another_stream_and_in_place_logits():
    """The calls run on the stream they are given; logits routed as given may be written onto themselves."""
    rng = np.random.default_rng(21)
    T, E, k = 2000, 64, 4
    l = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)).cuda()
    idx, w = torch.empty(T, k, **i32), torch.empty(T, k, device="cuda")
    want = oracle.route_select(np_(l), "softmax", np.full(T, k), k)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    before = l.clone()
    abi().semmoe_route_select(None, None, l, l, abi().SEMMOE_SCORE_SOFTMAX, None, 1, 1, 1, True, 1.0, None, k, T, 0, E, k,
                              idx, w, stream=side)
    side.synchronize()
    assert torch.equal(l, before)
    np.testing.assert_array_equal(np_(idx), want[0])
    np.testing.assert_allclose(np_(w), want[1], rtol=W_RTOL)


def test_select_flags_a_budget_out_of_range():
    from token_expert_routing_gb300 import SemMoEError
    l = np.tile(np.arange(8, dtype=np.float32), (4, 1))
    idx, _, _ = run(l, "sigmoid", [1, 0, 9, 2], 3)
    with pytest.raises(SemMoEError) as e:
        abi().semmoe_check_errors()
    assert e.value.bits == abi().SEMMOE_DEVERR_K
    assert idx.tolist() == [[7, -1, -1], [7, -1, -1], [7, 6, 5], [7, 6, -1]]


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_select_biases_of_the_lowest_float(score):
    """The type's lowest value as a bias puts an expert last without switching it off: it is taken
    when nothing else is left, before a group that is off, ties by index."""
    l = np.tile(np.linspace(-2, 2, 16, dtype=np.float32), (3, 1))
    low = np.finfo(np.float32).min
    b = np.full(16, low, dtype=np.float32)
    b[:4] = -np.inf                       # group 0 off; groups 1 to 3 at the lowest value
    idx, w, _ = run(l, score, [6] * 3, 6, b, 4, 2, 2)
    assert (idx == np.arange(4, 10)).all() and np.isfinite(w).all() and (w > 0).all()
    b[13] = 0.0                           # one ordinary expert: its group's sum is the lowest value's alone
    idx, _, _ = run(l, score, [6] * 3, 6, b, 4, 2, 1)
    assert (idx == [13, 4, 5, 6, 7, 12]).all()
    b[4:] = -np.inf
    b[13] = low
    idx, w, _ = run(l, score, [2] * 3, 2, b, 4, 1, 2)
    assert (idx == [13, -1]).all() and (w == [1.0, 0.0]).all()
    assert abi().semmoe_check_errors() == 0
