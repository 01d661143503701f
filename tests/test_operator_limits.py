"""Row counts at the end of 32 bits: refused on the host, where the kernels' strides and tile counts would
run over (no buffer is touched)."""
import ctypes

import pytest

P = ctypes.c_void_p(4096)
LAST, FIRST = 2 ** 31 - 2 ** 16, 2 ** 31 - 2 ** 16 + 1  # the last size taken, the first refused


@pytest.fixture(scope="module")
def lib():
    from token_expert_routing_gb300 import build, _abi
    build.build()
    return _abi.lib()


def calls(lib):
    return {
        "quantize": lambda n: lib.semmoe_mx4_quantize(P, 1, 1, n, 32, P, P, None),
        "dequantize": lambda n: lib.semmoe_mx4_dequantize(P, P, 1, n, 32, P, 1, None),
        "quantize_rows": lambda n: lib.semmoe_mx4_quantize_rows(P, 1, n, 32, P, 1, 8, P, 1, P, P, None),
        "product": lambda n: lib.semmoe_mx4_grouped_gemm(P, P, P, P, P, P, n, 1, 8, 32, P, 1, None),
        "ffn": lambda n: lib.semmoe_mx4_grouped_ffn(P, P, P, P, P, P, P, P, n, 1, 32, 32, P, P, 1, None),
        "select": lambda n: lib.semmoe_route_select(None, 1, None, 1, P, None, 0, None, 1, 1, 1, 1, 1.0, None, 1, n, 0, 1, 1,
                                                    P, P, None, None, 0, None),
    }


@pytest.mark.parametrize("name", ["quantize", "dequantize", "quantize_rows", "product", "ffn", "select"])
def test_rows_at_the_end_of_32_bits(lib, name):
    call = calls(lib)[name]
    for n in (FIRST, 2 ** 31 - 1):
        assert call(n) == 1
        err = lib.semmoe_last_error().decode()
        assert "too large" in err or f"P = {n}" in err or f"T={n}" in err, err
    # the last size passes this check: another argument, wrong on purpose, is what is refused
    wrong = {
        "quantize": lambda: lib.semmoe_mx4_quantize(None, 1, 1, LAST, 32, P, P, None),
        "dequantize": lambda: lib.semmoe_mx4_dequantize(None, P, 1, LAST, 32, P, 1, None),
        "quantize_rows": lambda: lib.semmoe_mx4_quantize_rows(None, 1, LAST, 32, P, 1, 8, P, 1, P, P, None),
        "product": lambda: lib.semmoe_mx4_grouped_gemm(None, P, P, P, P, P, LAST, 1, 8, 32, P, 1, None),
        "ffn": lambda: lib.semmoe_mx4_grouped_ffn(None, P, P, P, P, P, P, P, LAST, 1, 32, 32, P, P, 1, None),
        "select": lambda: lib.semmoe_route_select(None, 1, None, 1, P, None, 0, None, 1, 1, 1, 1, 1.0, None, 1, LAST, 0, 1, 1,
                                                  None, P, None, None, 0, None),
    }[name]
    assert wrong() == 1
    assert "null" in lib.semmoe_last_error().decode()
