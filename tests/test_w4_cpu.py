"""4-bit weights with group scales on the CPU: the oracle against what its definition says, and what the calls refuse."""
import ctypes

import numpy as np
import pytest
import torch

import oracle


@pytest.fixture(scope="module")
def abi():
    from token_expert_routing_gb300 import build, _abi
    build.build()
    return _abi


def _err(lib):
    return lib.semmoe_last_error().decode()


P = ctypes.c_void_p(4096)


@pytest.mark.parametrize("zeros", [True, False])
@pytest.mark.parametrize("scale", ["f32", "bf16"])
def test_oracle_codes_stand_for_the_nearest_values(zeros, scale):
    rng = np.random.default_rng(3)
    x = (rng.standard_normal((40, 256)) * np.exp(rng.normal(0, 3, (40, 1)))).astype(np.float32)
    x[3] = 0
    x[4] = np.abs(x[4])
    code, s, z = oracle.w4_encode(x, 64, zeros, scale)
    assert code.min() >= 0 and code.max() <= 15 and (z is None) == (not zeros)
    v = oracle.w4_values(code, s, z, 64)
    step = np.repeat(s, 64, axis=1)
    # inside the range at most half a step off (a bf16 scale may end the range up to 15 x 2^-8 of a step early)
    slack = 0.5 + (1e-5 if scale == "f32" else 15 * 2.0 ** -8)
    assert (np.abs(v - x) <= slack * step + 1e-30).all()
    assert (v[3] == 0).all()


def test_oracle_product_by_hand():
    w = oracle.w4_values(np.array([[[9, 8, 7, 12]]]), np.array([[[0.5, 2.0]]]), np.array([[[8, 6]]]), 2)
    np.testing.assert_array_equal(w, [[[0.5, 0.0, 2.0, 12.0]]])
    out = oracle.w4_grouped_product([[1, 1, 1, 1], [2, 0, 0, 1]], np.concatenate([w, 2 * w]), [0, 1, 2], [1, 0])
    np.testing.assert_array_equal(out, [[29], [13]])


def quantize(lib, x=P, dtype=1, rows=4, K=256, group=128, codes=P, scales=P, sd=1, zeros=P):
    return lib.semmoe_w4_quantize(x, dtype, rows, K, group, codes, scales, sd, zeros, None)


def dequantize(lib, x=P, dtype=1, rows=4, K=256, group=128, codes=P, scales=P, sd=1, zeros=P):
    return lib.semmoe_w4_dequantize(codes, scales, sd, zeros, rows, K, group, x, dtype, None)


def gemm(lib, x=P, off=P, pe=P, codes=P, scales=P, sd=1, zeros=P, n=8, E=4, N=64, K=256, group=128, out=P):
    return lib.semmoe_w4_grouped_gemm(x, off, pe, codes, scales, sd, zeros, n, E, N, K, group, out, None)


def ffn(lib, x=P, off=P, pe=P, a=P, sa=P, za=P, b=P, sb=P, zb=P, sd=1, n=8, E=4, H=256, I=128, group=128, y=P, ws=P,
        ws_bytes=1 << 20):
    return lib.semmoe_w4_grouped_ffn(x, off, pe, a, sa, za, b, sb, zb, sd, n, E, H, I, group, y, ws, ws_bytes, None)


BAD8 = ctypes.c_void_p(8)
SHAPES = [(dict(group=16), "group = 16"), (dict(group=0), "group = 0"), (dict(group=96), "group = 96"), (dict(group=-128), "group = -128"),
          (dict(K=192), "192 columns"), (dict(K=0), "0 columns"), (dict(K=-128), "-128 columns"), (dict(sd=2), "scale_dtype 2")]


@pytest.mark.parametrize("call", [quantize, dequantize])
@pytest.mark.parametrize("kw,word", SHAPES + [
    (dict(dtype=4), "dtype 4"), (dict(rows=-1), "rows = -1"), (dict(rows=2 ** 31 - 1), "rows ="), (dict(x=None), "null"),
    (dict(codes=None), "null"), (dict(scales=None), "null"), (dict(x=BAD8), "misaligned"), (dict(codes=BAD8), "misaligned"),
    (dict(scales=ctypes.c_void_p(3)), "misaligned")])
def test_conversion_refusals(abi, call, kw, word):
    assert call(abi.lib(), **kw) == 1
    assert word in _err(abi.lib())


@pytest.mark.parametrize("kw,word", SHAPES + [
    (dict(E=0), "E = 0"), (dict(E=257), "E = 257"), (dict(n=-1), "P = -1"), (dict(n=2 ** 31 - 2 ** 16 + 1), "P ="),
    (dict(N=4), "N = 4"), (dict(N=60), "N = 60"), (dict(x=None), "null"), (dict(off=None), "null"), (dict(pe=None), "null"),
    (dict(codes=None), "null"), (dict(scales=None), "null"), (dict(out=None), "null"), (dict(x=BAD8), "misaligned"),
    (dict(out=BAD8), "misaligned"), (dict(codes=BAD8), "misaligned"), (dict(scales=ctypes.c_void_p(2), sd=0), "misaligned"),
    (dict(off=ctypes.c_void_p(2)), "misaligned"), (dict(n=1 << 30, N=256), "P * N too large"), (dict(N=1 << 30), "N or K"),
    (dict(n=2 ** 31 - 2 ** 16, E=256, N=120), "P * N too large")])
def test_product_refusals(abi, kw, word):
    assert gemm(abi.lib(), **kw) == 1
    assert word in _err(abi.lib())


@pytest.mark.parametrize("kw,word", [
    (dict(H=192), "192 columns"), (dict(I=64), "64 columns"), (dict(E=0), "E = 0"), (dict(n=-1), "P = -1"), (dict(sd=5), "scale_dtype 5"),
    (dict(b=None), "null"), (dict(sb=None), "null"), (dict(a=None), "null"), (dict(y=None), "null"), (dict(za=None), "go together"),
    (dict(zb=None), "go together"), (dict(ws=None), "workspace"), (dict(ws=ctypes.c_void_p(4112)), "workspace"),
    (dict(ws_bytes=100), "workspace"), (dict(n=1 << 30, H=256), "P * N too large"), (dict(n=1 << 28, I=1024), "P * I too large"),
    (dict(I=1 << 30), "I or P * I"), (dict(b=BAD8), "misaligned"), (dict(y=BAD8), "misaligned")])
def test_ffn_refusals(abi, kw, word):
    assert ffn(abi.lib(), **kw) == 1
    assert word in _err(abi.lib())


def test_no_rows_are_no_work_and_workspaces(abi):
    lib = abi.lib()
    assert quantize(lib, rows=0, x=None, codes=None) == 0 and dequantize(lib, rows=0, x=None) == 0
    assert gemm(lib, n=0, x=None, out=None) == 0 and ffn(lib, n=0, x=None, ws=None) == 0
    assert lib.semmoe_w4_grouped_ffn_workspace_size(24, 96) >= 24 * 96 * 2
    assert lib.semmoe_w4_grouped_ffn_workspace_size(-1, 96) == 0 and lib.semmoe_w4_grouped_ffn_workspace_size(4, 40) == 0


BF16, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
T, K, E, N, I, G = 10, 128, 3, 72, 96, 32


def entry(name):
    def weights(key, rows, K):
        what = f"{key} " if key else ""
        return {f"{key}c": (U8, rows * K // 2, f"{what}codes"), f"{key}s": (BF16, rows * K // G, f"{what}scales"),
                f"{key}z": (U8, rows * K // G, f"{what}zeros")}
    tables = dict(off=(I32, E + 1, "expert_offsets"), pe=(I32, E, "phys_to_expert"))
    return {
        "quantize": (dict(x=(F32, T * K, "x"), **weights("", T, K)),
                     lambda a, b: a.semmoe_w4_quantize(b["x"], T, K, G, b["c"], b["s"], b["z"])),
        "dequantize": (dict(out=(BF16, T * K, "out"), **weights("", T, K)),
                       lambda a, b: a.semmoe_w4_dequantize(b["c"], b["s"], b["z"], T, K, G, b["out"])),
        "gemm": (dict(x=(BF16, T * K, "x"), **tables, **weights("", E * N, K), out=(BF16, T * N, "out")),
                 lambda a, b: a.semmoe_w4_grouped_gemm(b["x"], b["off"], b["pe"], b["c"], b["s"], b["z"], T, E, N, K, G, b["out"])),
        "ffn": (dict(x=(BF16, T * K, "x"), **tables, **weights("w13", 2 * E * I, K), **weights("w2", E * K, I), y=(BF16, T * K, "y_perm")),
                lambda a, b: a.semmoe_w4_grouped_ffn(b["x"], b["off"], b["pe"], b["w13c"], b["w13s"], b["w13z"], b["w2c"], b["w2s"],
                                                     b["w2z"], T, E, K, I, G, b["y"], torch.empty(1 << 16, dtype=U8))),
    }[name]


@pytest.mark.parametrize("name", ["quantize", "dequantize", "gemm", "ffn"])
def test_every_buffer_is_checked(abi, name):
    spec, call = entry(name)
    good = {k: torch.zeros(n, dtype=t) for k, (t, n, _) in spec.items()}
    with pytest.raises(ValueError, match="expected a CUDA tensor"):
        call(abi, good)
    for key, (t, n, what) in spec.items():
        with pytest.raises(ValueError, match=f"^{what}: expected at least {n} "):
            call(abi, {**good, key: good[key][:n - 1]})
        with pytest.raises(ValueError, match=f"^{what}: expected|unsupported dtype"):
            call(abi, {**good, key: torch.zeros(n, dtype=torch.int64)})


def test_scales_of_one_type(abi):
    spec, call = entry("ffn")
    good = {k: torch.zeros(n, dtype=t) for k, (t, n, _) in spec.items()}
    good["w2s"] = good["w2s"].float()
    with pytest.raises(ValueError, match="one type"):
        call(abi, good)


@pytest.mark.parametrize("n,kw,word", [(0, {}, "P=0"), (4097, {}, "P=4097"), (8, dict(x=None), "null"), (8, dict(K=192), "192 columns")])
def test_wait_selftest_refusals(abi, n, kw, word):
    a = {**dict(x=P, K=256), **kw}
    assert abi.lib().semmoe_selftest_w4_wait(a["x"], P, P, P, P, 1, P, n, 4, 64, a["K"], 128, P, None) == 1
    assert word in _err(abi.lib())
