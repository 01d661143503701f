"""The layer with norms around it and experts in 4-bit group-scaled weights, together and alone, against the composition
of the oracle's steps."""
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


def block_norm(rng, H, before, after, nxt, gate, wd=torch.float32, offset=0.0, bs=0.75, rs=1.0):
    def vec(on):
        return torch.from_numpy((1 - offset + 0.2 * rng.standard_normal(H)).astype(np.float32)).to(wd) if on else None
    return api().BlockNorm(before, vec(before), vec(before == "layer"), after, vec(after), vec(after == "layer"), nxt, vec(nxt),
                           vec(nxt == "layer"), offset, 1e-6, vec(gate), bs, rs)


def norm_of(x, nm, which):
    w, b = getattr(nm, f"{which}_weight"), getattr(nm, f"{which}_bias")
    return oracle.norm(x, getattr(nm, which), None if w is None else np_(w), None if b is None else np_(b), nm.weight_offset, nm.eps)


def check(d, res, w4, nm, gate=None, group=32):
    """Every output, step by step: each step's inputs are those that the GPU's earlier steps wrote."""
    s, x = d["spec"], np_(d["x"])
    k = d["k_per_token"].numpy()
    z = x
    if nm is not None and nm.before:
        assert max_rel(np_(res.x_norm), norm_of(x, nm, "before")) < 2.0 ** -8
        z = np_(res.x_norm)
    assert max_rel(np_(res.logits), oracle.router_logits(z, d["w_router"])) < LOGIT_TOL
    idx, w = oracle.topk_route(np_(res.logits), k, s.k_max)
    np.testing.assert_array_equal(np_(res.topk_idx), idx)
    perm = oracle.permute(idx, k, d["expert_rank"], s.R)
    for key in ("expert_offsets", "phys_to_expert", "pair_to_sorted", "sorted_to_pair"):
        np.testing.assert_array_equal(np_(getattr(res, key)), perm[key], err_msg=key)
    rows = z[perm["sorted_to_pair"] // s.k_max]
    off, pe = perm["expert_offsets"], perm["phys_to_expert"]
    if w4 is not None:
        def values(codes, scales, zeros):
            c = np_(codes)
            c = np.stack([c & 15, c >> 4], -1).reshape(*c.shape[:-1], -1)
            return oracle.w4_values(c, np_(scales), None if zeros is None else np_(zeros), w4.group)
        y = oracle.w4_grouped_ffn(rows, values(w4.w13, w4.w13_scales, w4.w13_zeros), values(w4.w2, w4.w2_scales, w4.w2_zeros), off, pe)
    else:
        y = oracle.grouped_ffn(rows, off, pe, d["w13"], d["w2"], s.dtype)
    assert max_rel(np_(res.y_perm), y) < TOL[s.dtype]
    ys = None if res.y_shared is None else np_(res.y_shared)
    if ys is not None:
        assert max_rel(ys, oracle.shared_ffn(z, d["ws13"], d["ws2"], s.dtype)) < TOL[s.dtype]
    y = np_(res.y_perm)
    half = 2.0 ** -8 if s.dtype == "bf16" else 2.0 ** -18
    if nm is None:
        assert max_rel(np_(res.out), oracle.combine(y, perm["pair_to_sorted"], w, k, s.dtype, ys)) < half
        return
    g = gate if gate is not None else nm.gate
    w_of = lambda t: None if t is None else np_(t)  # noqa: E731
    out, nxt = oracle.combine_norm(y, perm["pair_to_sorted"], np_(res.topk_w), s.k_max, ys, nm.after, w_of(nm.after_weight),
                                   w_of(nm.after_bias), w_of(g), nm.block_scale, x, nm.residual_scale, nm.next,
                                   w_of(nm.next_weight), w_of(nm.next_bias), nm.weight_offset, nm.eps)
    assert max_rel(np_(res.out), out) < half
    assert (res.next_out is None) == (nxt is None)
    if nxt is not None:
        assert max_rel(np_(res.next_out), nxt) < half


CASES = [  # workload, sizes, group, zeros, norms (before, after, next), gate
    ("dsv2lite_prefill_T4096", dict(T=300, H=256, I=160, I_shared=320, V=3000), 32, True, ("rms", "rms", "rms"), True),
    ("dsv2lite_decode_T64", dict(T=1, H=256, I=192, I_shared=320, V=3000), 64, False, ("rms", "", "rms"), False),
    ("qwen3_30b_a3b_T16384", dict(T=1515, H=512, I=128, V=3000), 128, False, ("layer", "", ""), False),
    ("prism_subexpert_T8192", dict(T=512, H=256, I=32, V=3000, tokens_per_request=64), 32, True, ("", "layer", "layer"), True),
]


@pytest.mark.parametrize("parts", ["w4+norm", "w4", "norm"])
@pytest.mark.parametrize("name,over,group,zeros,norms,gate", CASES, ids=[c[0] for c in CASES])
def test_layer(name, over, group, zeros, norms, gate, parts):
    d = wl.make_inputs(wl.scaled(name, **over))
    s = d["spec"]
    rng = np.random.default_rng(17)
    nm = block_norm(rng, s.H, *norms, gate) if "norm" in parts else None
    w4 = api().W4Experts.quantize(d["w13"], d["w2"], group, zeros) if "w4" in parts else None
    kw = dict(fused_gather=False) if w4 is None else {}
    layer = api().MoELayer(d["w_router"], None if w4 else d["w13"], None if w4 else d["w2"], d["expert_rank"], d["lut"], s.R, s.k_max,
                           d["ws13"], d["ws2"], w4=w4, norm=nm, **kw)
    kpt = d["k_per_token"].cuda() if s.k_choices else None
    call = dict(k_per_token=kpt, k=None if s.k_choices else s.k, P=int(d["k_per_token"].sum()), keep_logits=True)
    res = layer.forward(d["x"].cuda(), d["token_ids"].cuda(), **call)
    api()._abi.semmoe_check_errors()
    check(d, res, w4, nm, group=group)
    if nm is not None:  # a gate per token, on another stream
        gate_t = torch.from_numpy(rng.standard_normal((s.T, s.H)).astype(np.float32)).cuda()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        res = layer.forward(d["x"].cuda(), d["token_ids"].cuda(), stream=side, gate=gate_t, **call)
        side.synchronize()
        api()._abi.semmoe_check_errors()
        check(d, res, w4, nm, gate_t, group=group)


def test_fp32_layer_with_norms():
    d = wl.make_inputs(wl.scaled("tiny_fp32_T256_E8", T=77))
    s = d["spec"]
    nm = block_norm(np.random.default_rng(3), s.H, "rms", "layer", "rms", True, offset=1.0, rs=0.5)
    layer = api().MoELayer(d["w_router"], d["w13"], d["w2"], d["expert_rank"], d["lut"], s.R, s.k_max, d["ws13"], d["ws2"], norm=nm)
    res = layer.forward(d["x"].cuda(), d["token_ids"].cuda(), k=s.k, keep_logits=True)
    api()._abi.semmoe_check_errors()
    check(d, res, None, nm)


def test_two_layers_in_a_row_captured():
    """Layer after layer as a model runs them -- the second one's norm comes with the first one's output -- from a graph,
    for a decode batch and a larger one, with the same bits as the eager calls."""
    d = wl.make_inputs(wl.scaled("dsv2lite_decode_T64", T=200, H=512, I=256, I_shared=512, V=3000))
    s = d["spec"]
    rng = np.random.default_rng(5)
    w4 = api().W4Experts.quantize(d["w13"], d["w2"], 128)

    def layer(before, nxt):
        nm = block_norm(rng, s.H, before, "", nxt, False, torch.bfloat16, bs=1.0)
        return api().MoELayer(d["w_router"], None, None, d["expert_rank"], d["lut"], s.R, s.k_max, d["ws13"], d["ws2"], w4=w4, norm=nm)

    first, second = layer("rms", "rms"), layer("rms", "")

    def run(x, ids):
        a = first.forward(x, ids, k=s.k)
        return a, second.forward(a.out, ids, k=s.k)

    for T in (3, 200):
        x, ids = d["x"][:T].cuda().contiguous(), d["token_ids"][:T].cuda().contiguous()
        a, b = run(x, ids)
        want = [t.clone() for t in (a.out, a.next_out, b.out)]
        caps = [api().CapturedLayer(first, T, k=s.k), api().CapturedLayer(second, T, k=s.k)]
        for _ in range(2):
            caps[0].x.copy_(x), caps[0].token_ids.copy_(ids), caps[1].token_ids.copy_(ids)
            r0 = caps[0].replay()
            caps[1].x.copy_(r0.out)
            r1 = caps[1].replay()
            assert all(torch.equal(p, q) for p, q in zip((r0.out, r0.next_out, r1.out), want))
        # the graphs' workspaces stay theirs when a larger call replaces the layer's
        first.forward(d["x"].cuda(), d["token_ids"].cuda(), k=s.k)
        assert torch.equal(caps[0].replay().out, want[0])
    api()._abi.semmoe_check_errors()
