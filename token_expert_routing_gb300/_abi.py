"""Binding of libsemmoe.so: the C ABI declared in include/semmoe.h.

Argument marshalling only -- every step runs in the library's CUDA kernels.
Calls go through the compiled entry points (``_fast``, csrc/binding.cpp); the same
symbols are declared for ctypes in ``SIGNATURES`` (``lib()``).
Functions carry the C names and take torch tensors (device memory) or None
for pointers; a non-zero status raises SemMoEError with the library's message.
There is no fallback: if the library is missing, every call raises.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libsemmoe.so")

SEMMOE_OK, SEMMOE_ERR_INVALID_ARG, SEMMOE_ERR_UNSUPPORTED, SEMMOE_ERR_CUDA, \
    SEMMOE_ERR_DEVICE_CHECK, SEMMOE_ERR_DEVICE_TIMEOUT = range(6)
SEMMOE_F32, SEMMOE_BF16 = 0, 1
SEMMOE_F32_SPLIT = 2   # router weight only: the output of semmoe_route_split_weight
# grouped-FFN kernel forms (semmoe_grouped_ffn_form)
SEMMOE_FORM_DEFAULT, SEMMOE_FORM_SINGLE, SEMMOE_FORM_PAIR1, SEMMOE_FORM_PAIR, SEMMOE_FORM_SINGLE_TMA_GATHER, \
    SEMMOE_FORM_CUDA_CORE, SEMMOE_FORM_FUSED = range(7)
# scores of semmoe_route_select
SEMMOE_SCORE_SIGMOID, SEMMOE_SCORE_SOFTMAX = 0, 1
# norms of semmoe_norm and semmoe_combine_norm
SEMMOE_NORM_NONE, SEMMOE_NORM_RMS, SEMMOE_NORM_LAYER = range(3)
# device error word bits (semmoe_check_errors)
SEMMOE_DEVERR_EXPERT, SEMMOE_DEVERR_TOKEN_ID, SEMMOE_DEVERR_LUT, SEMMOE_DEVERR_K, SEMMOE_DEVERR_PAIRS, \
    SEMMOE_DEVERR_TIMEOUT, SEMMOE_DEVERR_NONFINITE, SEMMOE_DEVERR_OFFSETS, SEMMOE_DEVERR_RANK = \
    (1 << i for i in range(9))

_DTYPE = {torch.float32: SEMMOE_F32, torch.bfloat16: SEMMOE_BF16}

_vp, _i, _sz, _f = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_float

# name -> (restype, argtypes), in the order of include/semmoe.h
SIGNATURES = {
    "semmoe_last_error": (ctypes.c_char_p, []),
    "semmoe_version": (_i, []),
    "semmoe_kernel_launches": (ctypes.c_ulonglong, []),
    "semmoe_check_errors": (_i, [_vp, ctypes.POINTER(_i)]),
    "semmoe_route_workspace_size": (_sz, [_i, _i, _i, _i, _i]),
    "semmoe_route": (_i, [_vp, _i, _vp, _i, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _sz, _vp]),
    "semmoe_pair_counts_size": (_sz, [_i, _i]),
    "semmoe_pair_counts_stride": (_i, [_i]),
    "semmoe_route_split_size": (_sz, [_i, _i]),
    "semmoe_route_split_weight": (_i, [_vp, _i, _i, _vp, _vp]),
    "semmoe_route_hier_workspace_size": (_sz, [_i, _i, _i, _i, _i]),
    "semmoe_route_hier": (_i, [_vp, _i, _vp, _i, _vp, _vp, _vp, _i, _vp, _i, _i, _i, _i, _i, _vp, _vp, _vp, _vp,
                               _sz, _vp]),
    "semmoe_route_select_workspace_size": (_sz, [_i, _i, _i, _i, _i]),
    "semmoe_route_select": (_i, [_vp, _i, _vp, _i, _vp, _vp, _i, _vp, _i, _i, _i, _i, _f, _vp, _i, _i, _i, _i, _i, _vp,
                                 _vp, _vp, _vp, _sz, _vp]),
    "semmoe_affinity_lookup": (_i, [_vp, _vp, _i, _i, _i, _vp, _vp]),
    "semmoe_remote_count": (_i, [_vp, _vp, _vp, _i, _i, _i, _i, _vp, _vp, _vp]),
    "semmoe_permute_workspace_size": (_sz, [_i, _i, _i]),
    "semmoe_permute": (_i, [_vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp,
                            _vp, _vp, _vp, _sz, _vp]),
    "semmoe_permute_noalloc": (_i, [_vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp,
                                    _vp, _vp, _vp]),
    "semmoe_grouped_ffn_workspace_size": (_sz, [_i, _i, _i]),
    "semmoe_grouped_ffn": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp, _vp, _sz, _vp]),
    "semmoe_grouped_ffn_gather": (_i, [_vp, _vp, _i, _i, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp, _vp, _sz,
                                       _vp]),
    "semmoe_grouped_ffn_form": (_i, [_vp, _vp, _i, _i, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp, _vp, _sz,
                                     _i, _i, _vp]),
    "semmoe_grouped_ffn_combine": (_i, [_vp, _i, _vp, _i, _i, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp,
                                        _vp, _sz, _vp]),
    "semmoe_combine_finish": (_i, [_vp, _vp, _i, _i, _i, _vp, _vp]),
    "semmoe_shared_ffn_workspace_size": (_sz, [_i, _i, _i]),
    "semmoe_shared_ffn": (_i, [_vp, _vp, _vp, _i, _i, _i, _i, _vp, _vp, _sz, _vp]),
    "semmoe_combine": (_i, [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp, _vp]),
    "semmoe_norm": (_i, [_vp, _i, _i, _i, _i, _vp, _vp, _i, _f, _f, _vp, _vp]),
    "semmoe_combine_norm": (_i, [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _vp, _vp, _i, _vp, _vp, _i, _f, _f, _vp, _i,
                                 _i, _f, _vp, _f, _vp, _vp, _vp]),
    "semmoe_mx4_scales_size": (_sz, [_i, _i, _i]),
    "semmoe_mx4_quantize": (_i, [_vp, _i, _i, _i, _i, _vp, _vp, _vp]),
    "semmoe_mx4_dequantize": (_i, [_vp, _vp, _i, _i, _i, _vp, _i, _vp]),
    "semmoe_mx4_quantize_rows": (_i, [_vp, _i, _i, _i, _vp, _i, _i, _vp, _i, _vp, _vp, _vp]),
    "semmoe_mx4_grouped_gemm": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _vp, _i, _vp]),
    "semmoe_mx4_grouped_ffn_workspace_size": (_sz, [_i, _i, _i]),
    "semmoe_mx4_grouped_ffn": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _vp, _vp, _sz, _vp]),
    "semmoe_w4_quantize": (_i, [_vp, _i, _i, _i, _i, _vp, _vp, _i, _vp, _vp]),
    "semmoe_w4_dequantize": (_i, [_vp, _vp, _i, _vp, _i, _i, _i, _vp, _i, _vp]),
    "semmoe_w4_grouped_gemm": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _vp, _i, _i, _i, _i, _i, _vp, _vp]),
    "semmoe_w4_grouped_ffn_workspace_size": (_sz, [_i, _i]),
    "semmoe_w4_grouped_ffn": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _vp, _vp, _sz, _vp]),
    "semmoe_selftest_bounded_wait": (_i, [_vp]),
    "semmoe_selftest_fused_ready_wait": (_i, [_vp, _vp, _vp, _i, _i, _i, _vp, _vp, _sz, _vp]),
    "semmoe_selftest_w4_wait": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _vp, _i, _i, _i, _i, _i, _vp, _vp]),
    "semmoe_selftest_mx4_wait": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _vp, _vp]),
    "semmoe_dp_schedule": (_i, [_vp, _vp, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "semmoe_transition_lookup": (_i, [_vp, _vp, _i, _vp, _i, _i, _i, _i, _vp, _vp]),
}


class SemMoEError(RuntimeError):
    def __init__(self, code: int, msg: str, bits: int = 0):
        super().__init__(f"[semmoe status {code}] {msg}")
        self.code = code
        self.bits = bits   # device error word bits, for SEMMOE_ERR_DEVICE_CHECK / _TIMEOUT


_lib = None
_lock = threading.Lock()


def lib() -> ctypes.CDLL:
    """The loaded library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        with _lock:
            if _lib is None:
                if not os.path.exists(LIB_PATH):
                    raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                                       "`python -m token_expert_routing_gb300.build`")
                handle = ctypes.CDLL(LIB_PATH)
                for name, (res, args) in SIGNATURES.items():
                    fn = getattr(handle, name)
                    fn.restype, fn.argtypes = res, args
                _lib = handle
    return _lib


_fast = None


def fast():
    """The entry points compiled against the library (csrc/binding.cpp): the C
    names, taking tensors, addresses or None for pointers, and returning the C status."""
    global _fast
    if _fast is None:
        lib()   # says how to build what is missing
        try:
            from . import _fast as module
        except ImportError as e:
            raise RuntimeError("the compiled binding is missing: build it with "
                               "`python -m token_expert_routing_gb300.build`") from e
        module.set_raise(_check)
        _fast = module
    return _fast


def _check(rc: int) -> None:
    if rc != SEMMOE_OK:
        raise SemMoEError(rc, lib().semmoe_last_error().decode())


#: the current stream's handle without a Stream object (3 us of a call's host time on Grace), where torch has it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> int:
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(torch.cuda.current_device())
    return torch.cuda.current_stream().cuda_stream


def _workspace(nbytes: int, device, stream) -> torch.Tensor:
    """A workspace for one call on ``stream`` (a Stream, an address or None: the current one).  It is taken
    from that stream's memory: torch may hand it on when it is dropped, which is then in order with the call's kernels."""
    if stream is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream if isinstance(stream, int) else stream.cuda_stream, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(nbytes, dtype=torch.uint8, device=device)


def dtype_code(t: torch.Tensor) -> int:
    try:
        return _DTYPE[t.dtype]
    except KeyError:
        raise ValueError(f"unsupported dtype {t.dtype}") from None


# ---------------------------------------------------------------------------
# one wrapper per C entry point
# ---------------------------------------------------------------------------
def semmoe_version() -> int:
    return lib().semmoe_version()


def semmoe_kernel_launches() -> int:
    return lib().semmoe_kernel_launches()


def semmoe_check_errors(stream=None) -> int:
    """Synchronise the stream and raise if a kernel flagged bad data (the
    error's ``bits`` holds the device error word); returns the bits (0)."""
    bits = ctypes.c_int(0)
    rc = lib().semmoe_check_errors(_stream(stream), ctypes.byref(bits))
    if rc != SEMMOE_OK:
        raise SemMoEError(rc, lib().semmoe_last_error().decode(), bits.value)
    return bits.value


def semmoe_route_workspace_size(T, H, E, x_dtype: int, w_dtype: int) -> int:
    return fast().semmoe_route_workspace_size(T, H, E, x_dtype, w_dtype)


def semmoe_pair_counts_size(T, E) -> int:
    return fast().semmoe_pair_counts_size(T, E)


def semmoe_pair_counts_stride(T) -> int:
    return fast().semmoe_pair_counts_stride(T)


def semmoe_route(x, w_router, logits_in, logits_out, k_per_token, k_uniform, T, H, E, k_max,
                 topk_idx, topk_w, ws=None, stream=None, w_dtype=None, pair_counts=None):
    """Router GEMM + top-k.  ``ws`` defaults to a fresh workspace of the size
    the library asks for (pass one to avoid the allocation); ``w_dtype`` =
    SEMMOE_F32_SPLIT when w_router holds the output of semmoe_route_split_weight;
    ``pair_counts`` (semmoe_pair_counts_size bytes) receives the count table of
    the picks for semmoe_permute."""
    xd = dtype_code(x) if x is not None else SEMMOE_F32
    wd = w_dtype if w_dtype is not None else (dtype_code(w_router) if w_router is not None else SEMMOE_F32)
    if ws is None:
        n = semmoe_route_workspace_size(T, max(H, 1), E, xd, wd)
        ws = _workspace(n, topk_idx.device, stream)
    _check(fast().semmoe_route(x, xd, w_router, wd, logits_in, logits_out,
                              k_per_token, k_uniform, T, H, E, k_max, topk_idx, topk_w,
                              pair_counts, ws, ws.numel() * ws.element_size(), _stream(stream)))


def semmoe_route_split_size(H, E) -> int:
    return fast().semmoe_route_split_size(H, E)


def semmoe_route_split_weight(w, H, E, split, stream=None):
    _check(fast().semmoe_route_split_weight(w, H, E, split, _stream(stream)))


def semmoe_route_hier_workspace_size(T, H, Ep, x_dtype: int, w_dtype: int) -> int:
    return fast().semmoe_route_hier_workspace_size(T, H, Ep, x_dtype, w_dtype)


def semmoe_route_hier(x, w_parent, logits_in, logits_out, sub_logw, N, k_per_token, k_uniform, T, H, Ep, k_max,
                      topk_idx, topk_w, ws=None, stream=None, w_dtype=None, pair_counts=None):
    """Hierarchical sub-expert routing.  ``ws`` defaults to a fresh workspace
    of the size the library asks for; ``w_dtype`` and ``pair_counts`` as in
    semmoe_route."""
    xd = dtype_code(x) if x is not None else SEMMOE_F32
    wd = w_dtype if w_dtype is not None else (dtype_code(w_parent) if w_parent is not None else SEMMOE_F32)
    if ws is None:
        n = semmoe_route_hier_workspace_size(T, max(H, 1), Ep, xd, wd)
        ws = _workspace(n, topk_idx.device, stream)
    _check(fast().semmoe_route_hier(x, xd, w_parent, wd, logits_in, logits_out, sub_logw, N,
                                   k_per_token, k_uniform, T, H, Ep, k_max, topk_idx, topk_w,
                                   pair_counts, ws, ws.numel() * ws.element_size(), _stream(stream)))


def semmoe_route_select_workspace_size(T, H, E, x_dtype: int, w_dtype: int) -> int:
    return fast().semmoe_route_select_workspace_size(T, H, E, x_dtype, w_dtype)


def semmoe_route_select(x, w_router, logits_in, logits_out, score: int, bias, n_group, topk_group, group_top, renorm,
                        scale, k_per_token, k_uniform, T, H, E, k_max, topk_idx, topk_w, ws=None, stream=None,
                        w_dtype=None, pair_counts=None):
    """Router product and expert choice by score, bias and groups.  ``score`` is
    SEMMOE_SCORE_SIGMOID or SEMMOE_SCORE_SOFTMAX, ``bias`` [E] fp32 or None; ``ws``
    defaults to a fresh workspace of the size the library asks for; ``w_dtype``
    and ``pair_counts`` as in semmoe_route."""
    if ws is None and logits_in is None and x is not None and w_router is not None:
        wd = w_dtype if w_dtype is not None else dtype_code(w_router)
        n = fast().semmoe_route_select_workspace_size(T, max(H, 1), E, dtype_code(x), wd)
        if n > 256:
            ws = _workspace(n, topk_idx.device, stream)
    fast().route_select(x, w_router, logits_in, logits_out, score, bias, n_group, topk_group, group_top, renorm, scale,
                        k_per_token, k_uniform, T, H, E, k_max, topk_idx, topk_w, pair_counts, ws, w_dtype, stream)


def semmoe_affinity_lookup(token_ids, lut, V, R, T, pred_rank, stream=None):
    _check(fast().semmoe_affinity_lookup(token_ids, lut, V, R, T, pred_rank, _stream(stream)))


def semmoe_remote_count(topk_idx, pred_rank, expert_rank, T, k_max, E, R, counts, remote, stream=None):
    _check(fast().semmoe_remote_count(topk_idx, pred_rank, expert_rank, T, k_max, E, R,
                                     counts, remote, _stream(stream)))


def semmoe_permute_workspace_size(T, k_max, E) -> int:
    return fast().semmoe_permute_workspace_size(T, k_max, E)


def semmoe_permute(topk_idx, expert_rank, x, T, H, E, R, k_max, P, expert_offsets, rank_offsets,
                   phys_to_expert, expert_counts, sorted_to_pair, pair_to_sorted, x_perm, ws,
                   stream=None, pair_counts=None):
    """``pair_counts``: the router's count table for these topk_idx, or None
    (the permute then counts the pairs itself)."""
    d = dtype_code(x) if x is not None else SEMMOE_F32
    _check(fast().semmoe_permute(topk_idx, expert_rank, x, d, T, H, E, R, k_max, P,
                                expert_offsets, rank_offsets, phys_to_expert,
                                expert_counts, sorted_to_pair, pair_to_sorted, x_perm,
                                pair_counts, ws, ws.numel() * ws.element_size(), _stream(stream)))


def semmoe_permute_noalloc(topk_idx, expert_rank, x, T, H, E, R, k_max, P, expert_offsets, rank_offsets,
                           phys_to_expert, expert_counts, sorted_to_pair, pair_to_sorted, x_perm,
                           stream=None):
    """semmoe_permute without a workspace: for callers that cannot allocate
    device memory (the scratch is a static 96 KiB array inside the library)."""
    d = dtype_code(x) if x is not None else SEMMOE_F32
    _check(fast().semmoe_permute_noalloc(topk_idx, expert_rank, x, d, T, H, E, R, k_max, P,
                                        expert_offsets, rank_offsets, phys_to_expert,
                                        expert_counts, sorted_to_pair, pair_to_sorted,
                                        x_perm, _stream(stream)))


def semmoe_grouped_ffn_workspace_size(P, I, dtype: int) -> int:
    return fast().semmoe_grouped_ffn_workspace_size(P, I, dtype)


def semmoe_grouped_ffn(x_perm, expert_offsets, phys_to_expert, w13, w2, P, E, H, I, y_perm, ws,
                       stream=None):
    _check(fast().semmoe_grouped_ffn(x_perm, expert_offsets, phys_to_expert, w13,
                                    w2, dtype_code(w13), P, E, H, I, y_perm, ws,
                                    ws.numel() * ws.element_size(), _stream(stream)))


def semmoe_grouped_ffn_gather(x, sorted_to_pair, k_max, T, expert_offsets, phys_to_expert, w13, w2, P, E, H, I,
                              y_perm, ws, stream=None):
    _check(fast().semmoe_grouped_ffn_gather(x, sorted_to_pair, k_max, T, expert_offsets,
                                           phys_to_expert, w13, w2, dtype_code(w13), P, E, H, I,
                                           y_perm, ws, ws.numel() * ws.element_size(), _stream(stream)))


def semmoe_grouped_ffn_form(x, sorted_to_pair, k_max, T, expert_offsets, phys_to_expert, w13, w2, P, E, H, I,
                            y_perm, ws, form1, form2, stream=None):
    _check(fast().semmoe_grouped_ffn_form(x, sorted_to_pair, k_max, T, expert_offsets,
                                         phys_to_expert, w13, w2, dtype_code(w13), P, E, H, I,
                                         y_perm, ws, ws.numel() * ws.element_size(), form1, form2,
                                         _stream(stream)))


def semmoe_grouped_ffn_combine(x, x_rows_are_tokens, sorted_to_pair, k_max, T, expert_offsets, phys_to_expert, w13,
                               w2, topk_w, P, E, H, I, acc, ws, stream=None):
    _check(fast().semmoe_grouped_ffn_combine(x, int(bool(x_rows_are_tokens)), sorted_to_pair, k_max, T,
                                            expert_offsets, phys_to_expert, w13, w2, topk_w,
                                            dtype_code(w13), P, E, H, I, acc, ws,
                                            ws.numel() * ws.element_size(), _stream(stream)))


def semmoe_combine_finish(acc, y_shared, T, H, out, stream=None):
    _check(fast().semmoe_combine_finish(acc, y_shared, dtype_code(out), T, H, out, _stream(stream)))


def semmoe_shared_ffn_workspace_size(T, I_s, dtype: int) -> int:
    return fast().semmoe_shared_ffn_workspace_size(T, I_s, dtype)


def semmoe_shared_ffn(x, ws13, ws2, T, H, I_s, y_shared, ws, stream=None):
    _check(fast().semmoe_shared_ffn(x, ws13, ws2, dtype_code(ws13), T, H, I_s,
                                   y_shared, ws, ws.numel() * ws.element_size(),
                                   _stream(stream)))


def semmoe_combine(y_perm, pair_to_sorted, topk_w, y_shared, T, H, k_max, P, out, stream=None):
    _check(fast().semmoe_combine(y_perm, pair_to_sorted, topk_w, y_shared,
                                dtype_code(out), T, H, k_max, P, out, _stream(stream)))


def semmoe_norm(x, T, H, kind: int, weight, bias, weight_offset, eps, out, stream=None):
    """out = the rows of x [T, H], normalised (SEMMOE_NORM_RMS or SEMMOE_NORM_LAYER), times weight_offset + weight, plus
    bias; weight and bias [H] (fp32 or bf16, both of one type) or None.  ``out`` may be x."""
    fast().norm(x, T, H, kind, weight, bias, weight_offset, eps, out, stream)


def semmoe_combine_norm(y_perm, pair_to_sorted, topk_w, y_shared, T, H, k_max, P, post_kind: int, post_weight, post_bias,
                        next_kind: int, next_weight, next_bias, weight_offset, eps, gate, gate_rows, block_scale, residual,
                        residual_scale, out, next_out=None, stream=None):
    """The combine (pair_to_sorted None: dense rows y_perm [T, H]), the norm after it, gate [gate_rows, H], residual,
    and next_out = the next block's norm of out (see include/semmoe.h).  ``out`` may be the residual."""
    fast().combine_norm(y_perm, pair_to_sorted, topk_w, y_shared, T, H, k_max, P, post_kind, post_weight, post_bias,
                        next_kind, next_weight, next_bias, weight_offset, eps, gate, gate_rows, block_scale, residual,
                        residual_scale, out, next_out, stream)


def semmoe_dp_schedule(pred_rank, req_offsets, T, n_req, R, hist, req_rank, req_order, rank_req_offsets,
                       req_tok_start, tok_order, tok_rank, rank_tok_offsets, stream=None):
    _check(fast().semmoe_dp_schedule(pred_rank, req_offsets, T, n_req, R, hist, req_rank,
                                    req_order, rank_req_offsets, req_tok_start, tok_order,
                                    tok_rank, rank_tok_offsets, _stream(stream)))


def semmoe_transition_lookup(topk_idx, k_per_token, k_uniform, trans, T, k_max, E, R, pred_next, stream=None):
    _check(fast().semmoe_transition_lookup(topk_idx, k_per_token, k_uniform, trans, T, k_max, E, R,
                                          pred_next, _stream(stream)))


def semmoe_mx4_scales_size(rows, K, groups) -> int:
    return fast().semmoe_mx4_scales_size(rows, K, groups)


def semmoe_mx4_quantize(x, groups, group_rows, K, codes, scales, stream=None):
    """x [groups * group_rows, K] (fp32 or bf16) to 4-bit codes [rows, K/2] and scales (uint8)."""
    fast().mx4_quantize(x, groups, group_rows, K, codes, scales, stream)


def semmoe_mx4_dequantize(codes, scales, groups, group_rows, K, out, stream=None):
    """The values that codes and scales stand for, in out's type (fp32 or bf16; exact in both)."""
    fast().mx4_dequantize(codes, scales, groups, group_rows, K, out, stream)


def semmoe_mx4_quantize_rows(x, T, K, pair_to_sorted, k_max, P, expert_offsets, E, codes, scales, stream=None):
    """Token rows x [T, K] quantised into expert order (see include/semmoe.h)."""
    fast().mx4_quantize_rows(x, T, K, pair_to_sorted, k_max, P, expert_offsets, E, codes, scales, stream)


def semmoe_mx4_grouped_gemm(a, a_scales, expert_offsets, phys_to_expert, b, b_scales, P, E, N, K, out, stream=None):
    """4-bit rows [P, K] times their expert's 4-bit matrix [N, K] into out [P, N] (fp32 or bf16)."""
    fast().mx4_grouped_gemm(a, a_scales, expert_offsets, phys_to_expert, b, b_scales, P, E, N, K, out, stream)


def semmoe_mx4_grouped_ffn_workspace_size(P, E, I) -> int:
    return fast().semmoe_mx4_grouped_ffn_workspace_size(P, E, I)


def semmoe_mx4_grouped_ffn(x, x_scales, expert_offsets, phys_to_expert, w13, w13_scales, w2, w2_scales, P, E, H, I,
                           y_perm, ws, stream=None):
    """SwiGLU experts on 4-bit rows and weights, y_perm [P, H] bf16."""
    fast().mx4_grouped_ffn(x, x_scales, expert_offsets, phys_to_expert, w13, w13_scales, w2, w2_scales, P, E, H, I,
                           y_perm, ws, stream)


def semmoe_w4_quantize(x, rows, K, group, codes, scales, zeros=None, stream=None):
    """x [rows, K] (fp32 or bf16) to 4-bit codes [rows, K/2], scales [rows, K/group] (fp32 or bf16) and, unless None,
    zero points [rows, K/group] (uint8)."""
    fast().w4_quantize(x, rows, K, group, codes, scales, zeros, stream)


def semmoe_w4_dequantize(codes, scales, zeros, rows, K, group, out, stream=None):
    """The values that codes, scales and zero points (None: 8) stand for, in out's type (fp32 or bf16)."""
    fast().w4_dequantize(codes, scales, zeros, rows, K, group, out, stream)


def semmoe_w4_grouped_gemm(x, expert_offsets, phys_to_expert, codes, scales, zeros, P, E, N, K, group, out, stream=None):
    """bf16 rows x [P, K], sorted by expert, times their expert's 4-bit matrix [N, K] into out [P, N] (bf16)."""
    fast().w4_grouped_gemm(x, expert_offsets, phys_to_expert, codes, scales, zeros, P, E, N, K, group, out, stream)


def semmoe_w4_grouped_ffn_workspace_size(P, I) -> int:
    return fast().semmoe_w4_grouped_ffn_workspace_size(P, I)


def semmoe_w4_grouped_ffn(x, expert_offsets, phys_to_expert, w13, w13_scales, w13_zeros, w2, w2_scales, w2_zeros, P, E, H,
                          I, group, y_perm, ws=None, stream=None):
    """SwiGLU experts on 4-bit weights, x and y_perm [P, H] bf16.  ``ws`` defaults to a fresh workspace of the size
    the library asks for."""
    if ws is None:
        ws = _workspace(fast().semmoe_w4_grouped_ffn_workspace_size(P, I), y_perm.device, stream)
    fast().w4_grouped_ffn(x, expert_offsets, phys_to_expert, w13, w13_scales, w13_zeros, w2, w2_scales, w2_zeros, P, E, H,
                          I, group, y_perm, ws, stream)


def semmoe_selftest_bounded_wait(stream=None):
    """Launch the wait that can never complete (it gives up after 2 s and sets
    the timeout bit); see include/semmoe.h."""
    _check(fast().semmoe_selftest_bounded_wait(_stream(stream)))


def semmoe_selftest_fused_ready_wait(x_perm, w13, w2, P, H, I, y_perm, ws, stream=None):
    """Run the one-launch grouped FFN with GEMM2's readiness waits made
    unreachable (each gives up after 2 s and sets the timeout bit); see
    include/semmoe.h."""
    _check(fast().semmoe_selftest_fused_ready_wait(x_perm, w13, w2, P, H, I, y_perm, ws,
                                                  ws.numel() * ws.element_size(), _stream(stream)))


def semmoe_selftest_w4_wait(x, expert_offsets, phys_to_expert, codes, scales, zeros, P, E, N, K, group, out, stream=None):
    """Run semmoe_w4_grouped_gemm's tensor-core form with its issuing warps' first waits made unreachable (each gives up
    after 2 s and sets the timeout bit); see include/semmoe.h."""
    _check(fast().semmoe_selftest_w4_wait(x, expert_offsets, phys_to_expert, codes, scales, dtype_code(scales), zeros, P, E, N,
                                          K, group, out, _stream(stream)))


def semmoe_selftest_mx4_wait(a, a_scales, expert_offsets, phys_to_expert, b, b_scales, P, E, N, K, out, stream=None):
    """Run the 4-bit product with its issuing warps' first waits made
    unreachable (each gives up after 2 s and sets the timeout bit); see
    include/semmoe.h."""
    _check(fast().semmoe_selftest_mx4_wait(a, a_scales, expert_offsets, phys_to_expert, b, b_scales, P, E, N, K, out,
                                           _stream(stream)))
