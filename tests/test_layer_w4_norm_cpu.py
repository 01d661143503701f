"""What a layer with norms around it or experts in 4-bit group-scaled weights takes and refuses (no device: the library
is a stand-in that records its calls)."""
import pytest
import torch

from test_streams import FakeLibrary, Recorder

U8, BF16 = torch.uint8, torch.bfloat16


def api():
    import token_expert_routing_gb300 as m
    return m


def experts(E=4, I=64, H=64, group=32, zeros=False, scale=BF16, **over):
    z = dict(w13_zeros=torch.zeros(E, 2 * I, H // group, dtype=U8), w2_zeros=torch.zeros(E, H, I // group, dtype=U8)) if zeros else {}
    d = dict(w13=torch.zeros(E, 2 * I, H // 2, dtype=U8), w13_scales=torch.zeros(E, 2 * I, H // group, dtype=scale),
             w2=torch.zeros(E, H, I // 2, dtype=U8), w2_scales=torch.zeros(E, H, I // group, dtype=scale), group=group, **z)
    return api().W4Experts(**{**d, **over})


def layer(w13=None, w2=None, **kw):
    return api().MoELayer(torch.zeros(4, 64, dtype=BF16), w13, w2, torch.zeros(4, dtype=torch.int32), torch.zeros(10, 1), 1, 2,
                          overlap=False, overlap_shared=False, device="cpu", **kw)


@pytest.fixture
def calls(monkeypatch):
    from token_expert_routing_gb300 import _abi
    names = []

    class Library(FakeLibrary):
        def __getattr__(self, name):
            f = super().__getattr__(name)
            if name.endswith("_size"):
                return f
            return lambda *a: (names.append((name.removeprefix("semmoe_"), a)), f(*a))[1]

    lib = Library()
    Recorder(monkeypatch)
    monkeypatch.setattr(_abi, "fast", lambda: lib)
    monkeypatch.setattr(_abi, "_stream", lambda s: 0)
    return names


def test_shapes_of_experts():
    e = experts(zeros=True)
    assert len(e.args) == 6 and e.args[2] is e.w13_zeros and e.args[5] is e.w2_zeros
    for kw, word in ((dict(group=48), "group"), (dict(w2=torch.zeros(4, 64, 16, dtype=U8)), "whole groups"), (dict(H=96, group=64), "whole groups"),
                     (dict(w13_scales=torch.zeros(4, 128, 1)), "w13_scales"), (dict(w2_zeros=torch.zeros(4, 64, 2, dtype=U8)), "both"),
                     (dict(zeros=True, w2_zeros=torch.zeros(4, 64, 4, dtype=U8)), "w2_zeros")):
        with pytest.raises(ValueError, match=word):
            experts(**kw)


def test_quantize_needs_whole_groups(calls):
    with pytest.raises(ValueError, match="96 columns"):
        api().W4Experts.quantize(torch.zeros(2, 128, 96), torch.zeros(2, 96, 64), group=64, device="cpu")
    e = api().W4Experts.quantize(torch.zeros(2, 128, 96), torch.zeros(2, 96, 64), group=32, zeros=True, device="cpu")
    assert e.w13.shape == (2, 128, 48) and e.w2_zeros.shape == (2, 96, 2) and [n for n, _ in calls] == ["w4_quantize"] * 2


def test_a_layer_refuses_what_does_not_go_together(calls):
    w13, w2 = torch.zeros(4, 128, 64, dtype=BF16), torch.zeros(4, 64, 64, dtype=BF16)
    norm = api().BlockNorm()
    for kw, word in ((dict(w13=w13, w2=w2, w4=experts()), "w4 holds"), (dict(w4=experts(), mx4=True), "no mx4"),
                     (dict(w4=experts(), fused_gather=True), "fused"), (dict(w4=experts(), fused_combine=True), "fused"),
                     (dict(w4=experts(), ws13=torch.zeros(64, 64), ws2=torch.zeros(64, 32)), "bf16 shared"),
                     (dict(), "or w4"), (dict(w13=w13, w2=w2, norm=norm, fused_combine=True), "fused_combine"),
                     (dict(w13=w13, w2=w2, norm=api().BlockNorm(before_weight=torch.ones(63))), "before_weight"),
                     (dict(w13=w13, w2=w2, norm=api().BlockNorm(gate=torch.ones(2, 64))), "gate")):
        with pytest.raises(ValueError, match=word):
            layer(**kw)
    with pytest.raises(ValueError, match="after"):
        api().BlockNorm(after="batch")
    x, ids = torch.zeros(3, 64, dtype=BF16), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="gate"):
        layer(w13=w13, w2=w2).forward(x, ids, k=2, gate=torch.zeros(3, 64))
    with pytest.raises(ValueError, match="gate"):
        layer(w13=w13, w2=w2, norm=norm).forward(x, ids, k=2, gate=torch.zeros(1, 64))


def test_the_steps_of_a_layer_with_norms_and_4_bit_experts(calls):
    norm = api().BlockNorm(before_weight=torch.ones(64), after="layer", next="rms", gate=torch.ones(64))
    moe = layer(w4=experts(), norm=norm)
    calls.clear()
    x = torch.zeros(3, 64, dtype=BF16)
    res = moe.forward(x, torch.zeros(3, dtype=torch.int32), k=2)
    names = [n for n, _ in calls]
    assert names[0] == "norm" and names[-1] == "combine_norm" and "w4_grouped_ffn" in names
    assert not {"combine", "grouped_ffn", "mx4_grouped_ffn"} & set(names)
    by = dict(calls)
    assert by["norm"][0] is x and by["route"][0] is res.x_norm
    # y_perm, ..., gate, gate_rows, block_scale, residual, residual_scale, out, next_out, stream
    a = by["combine_norm"]
    assert a[0] is res.y_perm and a[17] == 1 and a[19] is x and a[21] is res.out and a[22] is res.next_out
    per_token = torch.zeros(3, 64)
    moe.forward(x, torch.zeros(3, dtype=torch.int32), k=2, gate=per_token)
    assert dict(calls)["combine_norm"][16] is per_token and dict(calls)["combine_norm"][17] == 3
