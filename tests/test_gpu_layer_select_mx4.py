"""The layer with the expert choice by score and 4-bit experts, together and
alone, against the composition of the oracle's steps."""
import numpy as np
import pytest
import torch

import oracle
import workloads as wl
from parity_utils import LOGIT_TOL, TOL, max_rel, np_

pytestmark = pytest.mark.gpu


def api():
    import token_expert_routing_gb300 as m
    return m


def layer_of(d, **kw):
    s = d["spec"]
    return api().MoELayer(d["w_router"], d["w13"], d["w2"], d["expert_rank"], d["lut"], s.R, s.k_max, d["ws13"], d["ws2"], **kw)


def check(d, res, mx4, select=None):
    """Every output, with the selection taken from the GPU (its own tests pin it to the oracle's)."""
    s = d["spec"]
    k = d["k_per_token"].numpy()
    assert max_rel(np_(res.logits), oracle.router_logits(d["x"], d["w_router"])) < LOGIT_TOL
    idx, w = np_(res.topk_idx), np_(res.topk_w)
    if select is None:
        ref_idx, ref_w = oracle.topk_route(np_(res.logits), k, s.k_max)
        np.testing.assert_array_equal(idx, ref_idx)
    else:
        ref_idx, ref_w = oracle.route_select(np_(res.logits), select.score, k, s.k_max,
                                             None if select.bias is None else np_(select.bias), select.n_group,
                                             select.topk_group, select.group_top, select.renorm, select.scale)
        assert (idx == ref_idx).all(axis=1).mean() > 0.98  # scores a bit apart may change places
    same = (idx == ref_idx).all(axis=1)
    np.testing.assert_allclose(w[same], ref_w[same], rtol=1e-5)
    live = (idx >= 0).sum(axis=1)
    perm = oracle.permute(idx, live, d["expert_rank"], s.R)
    n = int(live.sum())
    for key in ("expert_offsets", "rank_offsets", "phys_to_expert", "expert_counts", "pair_to_sorted"):
        np.testing.assert_array_equal(np_(getattr(res, key)), perm[key], err_msg=key)
    np.testing.assert_array_equal(np_(res.sorted_to_pair)[:n], perm["sorted_to_pair"])
    tok = perm["sorted_to_pair"] // s.k_max
    off, pe = perm["expert_offsets"], perm["phys_to_expert"]
    E, I, H = s.E, s.I, s.H
    if mx4:
        rows = oracle.mx4_round(np_(d["x"]))[tok]
        y = oracle.mx4_grouped_ffn(rows, oracle.mx4_round(np_(d["w13"]).reshape(-1, H)).reshape(E, 2 * I, H),
                                   oracle.mx4_round(np_(d["w2"]).reshape(-1, I)).reshape(E, H, I), off, pe)
    else:
        y = oracle.grouped_ffn(np_(d["x"])[tok], off, pe, d["w13"], d["w2"], s.dtype)
    assert max_rel(np_(res.y_perm)[:n], y) < TOL["bf16"]
    ys = None if d["ws13"] is None else oracle.shared_ffn(d["x"], d["ws13"], d["ws2"], s.dtype)
    out = oracle.combine(y, perm["pair_to_sorted"], w, live, s.dtype, ys)
    assert max_rel(np_(res.out), out) < TOL["bf16"]


CASES = [
    ("dsv2lite_prefill_T4096", dict(T=300, H=256, I=160, I_shared=320, V=3000), dict(score="softmax", n_group=8, topk_group=3, group_top=1, renorm=False)),
    ("dsv2lite_decode_T64", dict(T=1, H=256, I=160, I_shared=320, V=3000), dict(n_group=8, topk_group=4, scale=2.5)),
    ("qwen3_30b_a3b_T16384", dict(T=1515, H=256, I=96, V=3000), dict(n_group=4, topk_group=2, scale=1.5)),
    ("prism_subexpert_T8192", dict(T=512, H=256, I=32, V=3000, tokens_per_request=64), dict()),
]


@pytest.mark.parametrize("mx4", [True, False], ids=["mx4", "bf16"])
@pytest.mark.parametrize("name,over,sel", CASES, ids=[c[0] for c in CASES])
def test_layer_with_choice_by_score(name, over, sel, mx4):
    d = wl.make_inputs(wl.scaled(name, **over))
    s = d["spec"]
    rng = np.random.default_rng(9)
    select = api().RouteSelect(bias=torch.from_numpy((0.1 * rng.standard_normal(s.E)).astype(np.float32)), **sel)
    layer = layer_of(d, select=select, mx4=mx4, **({} if mx4 else dict(fused_gather=False)))
    kpt = d["k_per_token"].cuda() if s.k_choices else None
    res = layer.forward(d["x"].cuda(), d["token_ids"].cuda(), kpt, None if s.k_choices else s.k,
                        int(d["k_per_token"].sum()), keep_logits=True)
    api()._abi.semmoe_check_errors()
    assert (res.x_perm is None) == mx4
    check(d, res, mx4, select)


def test_layer_mx4_with_the_plain_router_and_captured():
    """4-bit experts behind the plain router, and the same bits from a captured graph."""
    d = wl.make_inputs(wl.scaled("qwen3_30b_a3b_T16384", T=700, H=512, I=224, V=3000))
    layer = layer_of(d, mx4=True)
    res = layer.forward(d["x"].cuda(), d["token_ids"].cuda(), k=d["spec"].k, keep_logits=True)
    api()._abi.semmoe_check_errors()
    check(d, res, True)
    cap = api().CapturedLayer(layer, 700, k=d["spec"].k)
    for _ in range(2):
        cap.x.copy_(d["x"])
        cap.token_ids.copy_(d["token_ids"])
        assert torch.equal(cap.replay().out, res.out)
    api()._abi.semmoe_check_errors()


@pytest.mark.parametrize("mx4", [True, False], ids=["mx4", "bf16"])
def test_layer_with_experts_switched_off(mx4):
    """A rank's experts switched off by the bias: no row reaches them, tokens keep the rest,
    and with one expert fewer than k left every token has k - 1 pairs (given as P)."""
    d = wl.make_inputs(wl.scaled("dsv2lite_decode_T64", T=200, H=256, I=160, I_shared=320, V=3000))
    s = d["spec"]
    bias = torch.zeros(s.E)
    bias[np_(d["expert_rank"]) != 2] = -float("inf")
    bias[np_(d["expert_rank"]) == 3] = 0.5
    bias[torch.nonzero(torch.isfinite(bias)).flatten()[5:]] = -float("inf")  # 5 experts left for k = 6
    select = api().RouteSelect(bias=bias)
    layer = layer_of(d, select=select, mx4=mx4, **({} if mx4 else dict(fused_gather=False)))
    res = layer.forward(d["x"].cuda(), d["token_ids"].cuda(), d["k_per_token"].cuda(), P=5 * s.T, keep_logits=True)
    api()._abi.semmoe_check_errors()
    assert ((np_(res.topk_idx) >= 0).sum(axis=1) == 5).all()
    check(d, res, mx4, select)


def test_layer_refuses_what_mx4_cannot_do():
    d = wl.make_inputs(wl.scaled("qwen3_30b_a3b_T16384", T=8, H=256, I=96, V=3000))
    for kw in (dict(fused_gather=True), dict(fused_combine=True), dict(sub_logw=torch.zeros(128), select=api().RouteSelect())):
        with pytest.raises(ValueError):
            layer_of(d, mx4=True, **kw)
    d["w13"], d["w2"] = d["w13"].float(), d["w2"].float()
    with pytest.raises(ValueError, match="bf16"):
        layer_of(d, mx4=True)
    d["w13"], d["w2"] = d["w13"].bfloat16()[:, :80].contiguous(), d["w2"].bfloat16()[:, :, :40].contiguous()
    with pytest.raises(ValueError, match="blocks of 32"):
        layer_of(d, mx4=True)
    with pytest.raises(ValueError, match="score"):
        api().RouteSelect(score="relu")
