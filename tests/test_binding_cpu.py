"""What the compiled entries refuse before any CUDA call: a tensor of another type than the
library reads it as, one of fewer elements than it touches, and an address where the type
has to come from a tensor.  Host tensors stand in: with every buffer right, the refusal is that they are on the host."""
import pytest
import torch


@pytest.fixture(scope="module")
def abi():
    from token_expert_routing_gb300 import build, _abi
    build.build()
    return _abi


BF16, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
T, K, E, N, I, P, KM = 200, 96, 5, 72, 64, 390, 2  # K: one tile of scales, the last block of it unused


def scales(rows_in_groups, K):
    return sum(-(-r // 128) for r in rows_in_groups) * -(-K // 128) * 512


def entry(name):
    """The call and its buffers: argument name -> (type, elements, what the refusal names), in the call's order."""
    P_scales = (P // 128 + E) * 512
    tables = dict(expert_offsets=(I32, E + 1, "expert_offsets"), phys_to_expert=(I32, E, "phys_to_expert"))
    return {
        "mx4_quantize": (dict(x=(BF16, 3 * T * K, "x"), codes=(U8, 3 * T * K // 2, "codes"),
                              scales=(U8, scales([T] * 3, K), "codes scales")),
                         lambda a, b: a.semmoe_mx4_quantize(b["x"], 3, T, K, b["codes"], b["scales"])),
        "mx4_dequantize": (dict(codes=(U8, 3 * T * K // 2, "codes"), scales=(U8, scales([T] * 3, K), "codes scales"),
                                out=(F32, 3 * T * K, "out")),
                           lambda a, b: a.semmoe_mx4_dequantize(b["codes"], b["scales"], 3, T, K, b["out"])),
        "mx4_quantize_rows": (dict(x=(F32, T * K, "x"), pair_to_sorted=(I32, T * KM, "pair_to_sorted"),
                                   expert_offsets=tables["expert_offsets"], codes=(U8, P * K // 2, "codes"),
                                   scales=(U8, P_scales, "codes scales")),
                              lambda a, b: a.semmoe_mx4_quantize_rows(b["x"], T, K, b["pair_to_sorted"], KM, P,
                                                                      b["expert_offsets"], E, b["codes"], b["scales"])),
        "mx4_grouped_gemm": (dict(a=(U8, P * K // 2, "a"), a_scales=(U8, P_scales, "a scales"), **tables,
                                  b=(U8, E * N * K // 2, "b"), b_scales=(U8, scales([N] * E, K), "b scales"),
                                  out=(BF16, P * N, "out")),
                             lambda a, b: a.semmoe_mx4_grouped_gemm(b["a"], b["a_scales"], b["expert_offsets"],
                                                                    b["phys_to_expert"], b["b"], b["b_scales"], P, E, N, K,
                                                                    b["out"])),
        "mx4_grouped_ffn": (dict(x=(U8, P * K // 2, "x"), x_scales=(U8, P_scales, "x scales"), **tables,
                                 w13=(U8, E * 2 * I * K // 2, "w13"), w13_scales=(U8, scales([I] * 2 * E, K), "w13 scales"),
                                 w2=(U8, E * K * I // 2, "w2"), w2_scales=(U8, scales([K] * E, I), "w2 scales"),
                                 y=(BF16, P * K, "y_perm")),
                            lambda a, b: a.semmoe_mx4_grouped_ffn(b["x"], b["x_scales"], b["expert_offsets"],
                                                                  b["phys_to_expert"], b["w13"], b["w13_scales"], b["w2"],
                                                                  b["w2_scales"], P, E, K, I, b["y"], None)),
        "route_select": (dict(x=(BF16, T * K, "x"), w_router=(F32, E * K, "w_router"), **outputs()),
                         lambda a, b: select(a, b, b["x"], b["w_router"], None)),
        "route_select_split": (dict(x=(BF16, T * K, "x"), w_router=(U8, 3 * 16 * K * 2, "w_router"), **outputs()),
                               lambda a, b: select(a, b, b["x"], b["w_router"], None, w_dtype=a.SEMMOE_F32_SPLIT)),
        "route_select_typed": (dict(x=(BF16, T * K, "x"), w_router=(BF16, E * K, "w_router"), **outputs()),
                               lambda a, b: select(a, b, b["x"], b["w_router"], None, w_dtype=a.SEMMOE_BF16)),
        "route_select_logits": (dict(logits_in=(F32, T * E, "logits_in"), **outputs()),
                                lambda a, b: select(a, b, None, None, b["logits_in"])),
    }[name]


def outputs():
    return dict(logits_out=(F32, T * E, "logits_out"), bias=(F32, E, "bias"), k_per_token=(I32, T, "k_per_token"),
                topk_idx=(I32, T * KM, "topk_idx"), topk_w=(F32, T * KM, "topk_w"), pair_counts=(I32, E * 4, "pair_counts"))


def select(a, b, x, w, logits_in, w_dtype=None):
    ws = torch.empty(1 << 20, dtype=torch.uint8)
    a.semmoe_route_select(x, w, logits_in, b["logits_out"], 0, b["bias"], 1, 1, 1, True, 1.0, b["k_per_token"], 0, T, K, E,
                          KM, b["topk_idx"], b["topk_w"], ws, w_dtype=w_dtype, pair_counts=b["pair_counts"])


NAMES = ["mx4_quantize", "mx4_dequantize", "mx4_quantize_rows", "mx4_grouped_gemm", "mx4_grouped_ffn", "route_select",
         "route_select_split", "route_select_typed", "route_select_logits"]


@pytest.mark.parametrize("name", NAMES)
def test_every_buffer_is_checked(abi, name):
    spec, call = entry(name)
    good = {k: torch.zeros(n, dtype=t) for k, (t, n, _) in spec.items()}
    with pytest.raises(ValueError, match="expected a CUDA tensor"):
        call(abi, good)
    larger = {k: torch.zeros(n + 3, dtype=t) for k, (t, n, _) in spec.items()}
    with pytest.raises(ValueError, match="expected a CUDA tensor"):
        call(abi, larger)
    for key, (t, n, what) in spec.items():
        with pytest.raises(ValueError, match=f"^{what}: expected at least {n} "):
            call(abi, {**good, key: good[key][:n - 1]})
        with pytest.raises(ValueError, match=f"^{what}: expected|unsupported dtype"):
            wrong = torch.int16 if (name, key) == ("route_select_split", "w_router") else torch.int64
            call(abi, {**good, key: torch.zeros(n // 3 if wrong == torch.int16 else n, dtype=wrong)})


@pytest.mark.parametrize("name,key", [("mx4_quantize", "x"), ("mx4_dequantize", "out"), ("mx4_quantize_rows", "x"),
                                      ("mx4_grouped_gemm", "out"), ("route_select_logits", "x")])
def test_an_address_has_no_type(abi, name, key):
    """An address was taken for fp32: a bf16 buffer would be read past its end."""
    if name == "route_select_logits":
        with pytest.raises(ValueError, match="expected a tensor"):
            abi.fast().route_select(4096, None, 4096, None, 0, None, 1, 1, 1, 1, 1.0, None, 1, 2, 8, 4, 1, 4096, 4096, None,
                                    None, None, None)
        return
    spec, call = entry(name)
    with pytest.raises(ValueError, match="expected a tensor"):
        call(abi, {k: 4096 if k == key else torch.zeros(n, dtype=t) for k, (t, n, _) in spec.items()})


def test_sizes_that_overflow_are_the_librarys_to_refuse(abi):
    """Products of sizes past 64 bits refuse the buffer; negative ones reach the library."""
    codes, sc, x = torch.zeros(64, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8), torch.zeros(4, 32)
    big = 2 ** 31 - 1
    with pytest.raises(ValueError, match="codes"):
        abi.semmoe_mx4_quantize(x, big, big, big, codes, sc)
    with pytest.raises(ValueError, match="CUDA"):
        abi.semmoe_mx4_quantize(x, -1, 4, 32, codes, sc)
