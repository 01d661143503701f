"""Refusals of the expert-choice router and the 4-bit operators: bad arguments
are rejected on the host before any CUDA call (CPU only)."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def lib():
    from token_expert_routing_gb300 import build, _abi
    build.build()
    return _abi.lib()


def _err(lib):
    return lib.semmoe_last_error().decode()


P = ctypes.c_void_p(4096)


def select(lib, T=4, H=64, E=16, k_max=2, score=0, bias=P, G=4, keep=2, top=2, scale=1.0, ku=2, logits=P, idx=P, w=P,
           pc=None):
    return lib.semmoe_route_select(None, 1, None, 1, logits, None, score, bias, G, keep, top, 1, scale, None, ku, T, H, E,
                                   k_max, idx, w, pc, None, 0, None)


@pytest.mark.parametrize("kw,word", [
    (dict(T=-1), "T = -1"), (dict(E=0), "E = 0"), (dict(E=300), "E = 300"), (dict(k_max=17), "k_max = 17"),
    (dict(score=2), "score 2"), (dict(G=3), "n_group = 3"), (dict(G=0), "n_group = 0"), (dict(keep=0), "topk_group = 0"),
    (dict(keep=5), "topk_group = 5"), (dict(top=3), "group_top = 3"), (dict(top=0), "group_top = 0"),
    (dict(k_max=9, ku=9), "exceeds the 8 experts"), (dict(scale=float("nan")), "scale"),
    (dict(scale=float("inf")), "scale"), (dict(ku=0), "k_uniform = 0"), (dict(idx=None), "null output"),
    (dict(w=None), "null output"), (dict(logits=None), "null x"), (dict(bias=ctypes.c_void_p(2)), "misaligned"),
    (dict(pc=ctypes.c_void_p(8)), "misaligned"), (dict(T=1 << 27), "too large"),
])
def test_select_refusals(lib, kw, word):
    assert select(lib, **kw) == 1
    assert word in _err(lib)


def test_select_needs_its_workspace_and_nothing_for_no_tokens(lib):
    assert select(lib, T=0) == 0
    assert lib.semmoe_route_select_workspace_size(64, 64, 300, 1, 1) == 0
    need = lib.semmoe_route_select_workspace_size(6400, 64, 16, 1, 1)
    rc = lib.semmoe_route_select(P, 1, P, 1, None, None, 0, None, 1, 1, 1, 1, 1.0, None, 2, 6400, 64, 16, 2, P, P, None, P,
                                 need - 1, None)
    assert rc == 1 and "workspace" in _err(lib)


def test_mx4_sizes(lib):
    assert lib.semmoe_mx4_scales_size(128, 128, 1) == 2 * 512
    assert lib.semmoe_mx4_scales_size(1003, 352, 5) == (7 + 5) * 3 * 512
    for bad in ((-1, 64, 1), (4, 0, 1), (4, 48, 1), (4, 64, 0)):
        assert lib.semmoe_mx4_scales_size(*bad) == 0
    assert lib.semmoe_mx4_grouped_ffn_workspace_size(0, 1, 32) >= 512
    for bad in ((-1, 1, 32), (4, 0, 32), (4, 1, 40)):
        assert lib.semmoe_mx4_grouped_ffn_workspace_size(*bad) == 0


@pytest.mark.parametrize("name", ["semmoe_mx4_quantize", "semmoe_mx4_dequantize"])
def test_mx4_quantize_refusals(lib, name):
    def call(dtype=1, groups=2, rows=4, K=64, full=P, codes=P, scales=P):
        if name == "semmoe_mx4_quantize":
            return lib.semmoe_mx4_quantize(full, dtype, groups, rows, K, codes, scales, None)
        return lib.semmoe_mx4_dequantize(codes, scales, groups, rows, K, full, dtype, None)
    for kw, word in ((dict(dtype=2), "dtype 2"), (dict(groups=0), "groups=0"), (dict(rows=-1), "group_rows=-1"),
                     (dict(K=48), "K = 48"), (dict(K=0), "K = 0"), (dict(groups=1 << 16, rows=1 << 16), "too large"),
                     (dict(full=None), "null"), (dict(codes=None), "null"), (dict(scales=None), "null"),
                     (dict(full=ctypes.c_void_p(8)), "aligned"), (dict(codes=ctypes.c_void_p(8)), "aligned"),
                     (dict(scales=ctypes.c_void_p(8)), "aligned")):
        assert call(**kw) == 1, kw
        assert word in _err(lib), kw
    assert call(rows=0, full=None, codes=None, scales=None) == 0


def test_mx4_quantize_rows_refusals(lib):
    def call(x=P, dtype=1, T=4, K=64, map_=P, k=2, n=8, off=P, E=4, codes=P, scales=P):
        return lib.semmoe_mx4_quantize_rows(x, dtype, T, K, map_, k, n, off, E, codes, scales, None)
    for kw, word in ((dict(dtype=2), "dtype"), (dict(K=40), "K = 40"), (dict(E=0), "E = 0"), (dict(E=257), "E = 257"),
                     (dict(T=-1), "T=-1"), (dict(k=0), "k_max=0"), (dict(n=9), "P = 9"), (dict(n=-1), "P = -1"),
                     (dict(x=None), "null"), (dict(map_=None), "null"), (dict(off=None), "null"),
                     (dict(codes=ctypes.c_void_p(4)), "aligned"), (dict(off=ctypes.c_void_p(2)), "misaligned")):
        assert call(**kw) == 1, kw
        assert word in _err(lib), kw
    assert call(n=0, x=None) == 0


def test_mx4_product_refusals(lib):
    def gemm(a=P, sa=P, off=P, pe=P, b=P, sb=P, n=8, E=4, N=64, K=64, out=P, dtype=1):
        return lib.semmoe_mx4_grouped_gemm(a, sa, off, pe, b, sb, n, E, N, K, out, dtype, None)
    for kw, word in ((dict(E=0), "E = 0"), (dict(E=257), "E = 257"), (dict(n=-1), "P = -1"), (dict(K=16), "K = 16"),
                     (dict(N=4), "N = 4"), (dict(N=20), "N = 20"), (dict(dtype=7), "dtype 7"), (dict(a=None), "null"),
                     (dict(sb=None), "null"), (dict(out=ctypes.c_void_p(8)), "aligned"),
                     (dict(pe=ctypes.c_void_p(2)), "misaligned")):
        assert gemm(**kw) == 1, kw
        assert word in _err(lib), kw
    assert gemm(n=0, a=None) == 0

    def ffn(x=P, sx=P, off=P, pe=P, w13=P, s13=P, w2=P, s2=P, n=8, E=4, H=64, I=96, y=P, ws=P, ws_bytes=1 << 20):
        return lib.semmoe_mx4_grouped_ffn(x, sx, off, pe, w13, s13, w2, s2, n, E, H, I, y, ws, ws_bytes, None)
    for kw, word in ((dict(H=40), "K = 40"), (dict(I=40), "I = 40"), (dict(E=0), "E = 0"), (dict(w2=None), "null"),
                     (dict(s13=None), "null"), (dict(ws=None), "workspace"), (dict(ws=ctypes.c_void_p(4112)), "workspace"),
                     (dict(ws_bytes=100), "workspace"), (dict(y=ctypes.c_void_p(8)), "aligned")):
        assert ffn(**kw) == 1, kw
        assert word in _err(lib), kw
    assert ffn(n=0) == 0


def test_binding_refuses_other_types_and_short_buffers():
    from token_expert_routing_gb300 import _abi
    with pytest.raises(ValueError, match="bias"):
        _abi.semmoe_route_select(None, None, None, None, 0, torch.zeros(4, dtype=torch.float64), 1, 1, 1, True, 1.0, None, 1,
                                 2, 8, 4, 1, None, None)
    codes, scales = torch.empty(4 * 32, dtype=torch.uint8), torch.empty(512, dtype=torch.uint8)
    with pytest.raises(ValueError, match="codes"):
        _abi.semmoe_mx4_quantize(torch.zeros(4, 64), 1, 4, 64, codes[:100], scales)
    with pytest.raises(ValueError, match="scales"):
        _abi.semmoe_mx4_dequantize(codes, scales[:100], 1, 4, 64, torch.zeros(4, 64))
    with pytest.raises(ValueError, match="codes"):
        _abi.semmoe_mx4_quantize(torch.zeros(4, 64), 1, 4, 64, codes.to(torch.int32), scales)


def test_compiled_entry_points_cover_the_abi_and_check_their_arguments():
    """Every enqueuing call has its compiled entry; host tensors, wrong argument counts and
    integers past 32 bits are refused before the library is called."""
    from token_expert_routing_gb300 import _abi
    fast = _abi.fast()
    left = {"semmoe_last_error", "semmoe_version", "semmoe_kernel_launches", "semmoe_check_errors"}
    for name, (_, args) in _abi.SIGNATURES.items():
        if name in left:
            continue
        with pytest.raises(TypeError, match=f"expected {len(args)} arguments, got 0"):
            getattr(fast, name)()
    with pytest.raises(ValueError, match="CUDA tensor"):
        fast.semmoe_mx4_quantize(torch.zeros(4, 64), 0, 1, 4, 64, None, None, None)
    with pytest.raises(OverflowError):
        fast.semmoe_mx4_scales_size(1 << 31, 64, 1)
    with pytest.raises(TypeError):
        fast.semmoe_mx4_scales_size(1.5, 64, 1)
    with pytest.raises(TypeError, match="got str"):
        fast.semmoe_mx4_quantize("x", 0, 1, 4, 64, None, None, None)
    assert fast.semmoe_mx4_scales_size(128, 128, 1) == 1024
    assert fast.semmoe_mx4_quantize(None, 0, 1, 4, 48, 256, 256, None) == _abi.SEMMOE_ERR_INVALID_ARG
