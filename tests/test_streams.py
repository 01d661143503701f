"""Memory that a call takes for itself belongs to the stream that the call runs on."""
import contextlib
import gc
import weakref

import numpy as np
import pytest
import torch


class FakeStream:
    def __init__(self, handle):
        self.cuda_stream = handle

    def __eq__(self, other):
        return self.cuda_stream == other.cuda_stream

    def __hash__(self):
        return hash(self.cuda_stream)


class Recorder:
    """Torch's stream context and allocation, recorded: which stream was current at each torch.empty."""

    def __init__(self, monkeypatch):
        self.current, self.allocated = None, []
        real = torch.empty

        @contextlib.contextmanager
        def use(stream):
            before, self.current = self.current, stream
            yield
            self.current = before

        def empty(*a, **kw):
            kw.pop("device", None)
            self.allocated.append(None if self.current is None else self.current.cuda_stream)
            return real(*a, **kw)

        monkeypatch.setattr(torch.cuda, "Stream", FakeStream)
        monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: FakeStream(handle))
        monkeypatch.setattr(torch.cuda, "stream", use)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: self.current or FakeStream(0))
        monkeypatch.setattr(torch, "empty", empty)


class FakeLibrary:
    """The compiled entries: sizes are 1 MB unless set, calls return success and keep the stream they were given."""

    def __init__(self):
        self.streams, self.size = [], 1 << 20

    def __getattr__(self, name):
        if name.endswith("_size"):
            return lambda *a: self.size

        def call(*a):
            self.streams.append(a[-1])
            return 0
        return call


def small_layer(**kw):
    from token_expert_routing_gb300 import MoELayer
    bf16 = dict(dtype=torch.bfloat16)
    return MoELayer(torch.zeros(4, 32, **bf16), torch.zeros(4, 64, 32, **bf16), torch.zeros(4, 32, 32, **bf16),
                    torch.zeros(4, dtype=torch.int32), torch.zeros(10, 1), 1, 2, overlap=False, overlap_shared=False,
                    device="cpu", **kw)


ROUTE, HIER, SELECT = "semmoe_route", "semmoe_route_hier", "semmoe_route_select"


@pytest.mark.parametrize("name,kind", [(n, k) for n in (ROUTE, HIER, SELECT) for k in ("none", "stream")]
                         + [(SELECT, "address"), (SELECT, "object")])
def test_a_call_takes_its_workspace_on_its_own_stream(monkeypatch, name, kind):
    from token_expert_routing_gb300 import _abi
    lib = FakeLibrary()
    x, w = torch.zeros(2, 8, dtype=torch.bfloat16), torch.zeros(4, 8)
    idx, gw, sub = torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, 1), torch.zeros(8)
    rec = Recorder(monkeypatch)
    monkeypatch.setattr(_abi, "fast", lambda: lib)
    monkeypatch.setattr(_abi, "_stream", lambda s: 0 if s is None else s.cuda_stream)
    stream = {"none": None, "stream": FakeStream(77), "address": 77, "object": type("S", (), {"cuda_stream": 77})()}[kind]
    if name == ROUTE:
        _abi.semmoe_route(x, w, None, None, None, 1, 2, 8, 4, 1, idx, gw, stream=stream)
    elif name == HIER:
        _abi.semmoe_route_hier(x, w, None, None, sub, 2, None, 1, 2, 8, 4, 1, idx, gw, stream=stream)
    else:
        _abi.semmoe_route_select(x, w, None, None, 0, None, 1, 1, 1, True, 1.0, None, 1, 2, 8, 4, 1, idx, gw, stream=stream)
    assert rec.allocated == [None if kind == "none" else 77]
    assert len(lib.streams) == 1


@pytest.mark.parametrize("mx4", [False, True])
@pytest.mark.parametrize("handle", [None, 0, 77])
def test_a_forward_takes_its_memory_on_its_own_stream(monkeypatch, mx4, handle):
    """Tables that a forward drops when it returns (the count table, workspaces), and its outputs."""
    from token_expert_routing_gb300 import _abi
    lib = FakeLibrary()
    rec = Recorder(monkeypatch)
    monkeypatch.setattr(_abi, "fast", lambda: lib)
    monkeypatch.setattr(_abi, "_stream", lambda s: rec.current.cuda_stream if s is None and rec.current else 0 if s is None else s.cuda_stream)
    bf16 = dict(dtype=torch.bfloat16)
    layer = small_layer(mx4=mx4, fused_gather=None if mx4 else False)
    rec.allocated.clear()
    lib.streams.clear()
    layer.forward(torch.zeros(3, 32, **bf16), torch.zeros(3, dtype=torch.int32), k=2,
                  stream=None if handle is None else FakeStream(handle))
    assert len(rec.allocated) > 10 and {h or 0 for h in rec.allocated} == {handle or 0}
    assert len(lib.streams) >= 5


@pytest.mark.parametrize("mx4", [False, True])
def test_a_captured_layer_keeps_the_workspaces_of_its_graph(monkeypatch, mx4):
    """A forward of a larger batch replaces the layer's workspaces; a graph captured before still writes its own."""
    from token_expert_routing_gb300 import CapturedLayer, _abi

    class Graph:
        pass

    lib = FakeLibrary()
    Recorder(monkeypatch)
    monkeypatch.setattr(_abi, "fast", lambda: lib)
    monkeypatch.setattr(_abi, "_stream", lambda s: 0)
    monkeypatch.setattr(FakeStream, "wait_stream", lambda self, other: None, raising=False)
    monkeypatch.setattr(torch.cuda, "Stream", lambda device=None: FakeStream(5))
    monkeypatch.setattr(torch.cuda, "CUDAGraph", Graph)
    monkeypatch.setattr(torch.cuda, "graph", lambda g: torch.cuda.stream(FakeStream(9)))
    layer = small_layer(mx4=mx4, fused_gather=None if mx4 else False)
    cap = CapturedLayer(layer, 3, k=2)
    used = {k: weakref.ref(b) for k, b in layer._ws.items()}
    assert {"route", "permute", "ffn"} <= set(used) and ("mx4_rows" in used) == mx4
    lib.size = 1 << 21
    layer.forward(torch.zeros(300, 32, dtype=torch.bfloat16), torch.zeros(300, dtype=torch.int32), k=2)
    gc.collect()
    assert all(layer._ws[k] is not ref() for k, ref in used.items())
    assert all(ref() is not None for ref in used.values())
    del cap
    gc.collect()
    assert all(ref() is None for ref in used.values())


@pytest.mark.gpu
@pytest.mark.parametrize("name", [ROUTE, HIER, SELECT])
def test_workspace_on_a_side_stream_is_not_handed_on_early(name):
    """A product with partial logits in its workspace, behind work on its own stream, and allocations of the
    same size written on the current stream right after the call."""
    from token_expert_routing_gb300 import _abi
    rng = np.random.default_rng(3)
    T, H, E, k = 3000, 512, 256, 6
    x = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).to(torch.bfloat16).cuda()
    wr = torch.from_numpy((rng.standard_normal((E, H)) / np.sqrt(H)).astype(np.float32)).cuda()
    Ep = 64
    sub = torch.zeros(E, device="cuda")

    def call(stream):
        idx, w = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
        if name == ROUTE:
            _abi.semmoe_route(x, wr, None, None, None, k, T, H, E, k, idx, w, stream=stream)
        elif name == HIER:
            _abi.semmoe_route_hier(x, wr[:Ep], None, None, sub, E // Ep, None, k, T, H, Ep, k, idx, w, stream=stream)
        else:
            _abi.semmoe_route_select(x, wr, None, None, _abi.SEMMOE_SCORE_SOFTMAX, None, 1, 1, 1, True, 1.0, None, k, T, H,
                                     E, k, idx, w, stream=stream)
        return idx, w

    want = [t.clone() for t in call(None)]
    n = max(_abi.semmoe_route_workspace_size(T, H, E, _abi.SEMMOE_BF16, _abi.SEMMOE_F32),
            _abi.semmoe_route_select_workspace_size(T, H, E, _abi.SEMMOE_BF16, _abi.SEMMOE_F32))
    busy = torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    for form in ("stream", "address") if name == SELECT else ("stream",):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for _ in range(4):
                busy @ busy  # the call waits behind these
        got = call(side if form == "stream" else side.cuda_stream)
        spoilers = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
        side.synchronize()
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        del spoilers
    assert _abi.semmoe_check_errors() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("mx4", [False, True])
def test_a_captured_layer_after_a_larger_forward_and_a_second_graph(mx4):
    """Replays of a graph captured for a small batch, with the memory that larger forwards freed filled by others."""
    import workloads as wl
    from token_expert_routing_gb300 import CapturedLayer, MoELayer, _abi
    d = wl.make_inputs(wl.scaled("qwen3_30b_a3b_T16384", T=900, H=256, I=96, V=3000))
    s = d["spec"]
    layer = MoELayer(d["w_router"], d["w13"], d["w2"], d["expert_rank"], d["lut"], s.R, s.k_max, mx4=mx4)
    x, ids = d["x"].cuda(), d["token_ids"].cuda()
    small = CapturedLayer(layer, 50, k=s.k)
    larger = CapturedLayer(layer, 300, k=s.k)
    want = [layer.forward(x[:n].clone(), ids[:n].clone(), k=s.k).out.clone() for n in (50, 300)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    whole = layer.forward(x, ids, k=s.k, stream=side).out  # replaces every workspace
    side.synchronize()
    spoilers = [torch.full((1 << n,), 255, dtype=torch.uint8, device="cuda") for n in range(8, 25) for _ in range(4)]
    for cap, n, ref in ((small, 50, want[0]), (larger, 300, want[1])):
        cap.x.copy_(x[:n])
        cap.token_ids.copy_(ids[:n])
        assert torch.equal(cap.replay().out, ref)
    torch.cuda.synchronize()
    assert all(bool((t == 255).all()) for t in spoilers)
    assert torch.equal(layer.forward(x, ids, k=s.k).out, whole)
    assert _abi.semmoe_check_errors() == 0
