"""Which buffers the norms' outputs may share with their inputs."""
import ctypes

import numpy as np
import pytest
import torch

from test_norm_cpu import Q, _err, abi, after, norm  # noqa: F401  (abi: the fixture)

R, S, U = (ctypes.c_void_p(n << 20) for n in (1, 2, 3))  # buffers far from one another


def apart(lib, **kw):
    return after(lib, **{**dict(y=R, q=S, w=U, r=None, pw=None, out=Q), **kw})


@pytest.mark.parametrize("dtype,gate_dtype", [(1, 0), (0, 1)])
@pytest.mark.parametrize("T", [1, 4])
def test_out_is_no_gate_of_another_type(abi, dtype, gate_dtype, T):  # noqa: F811
    """Row t of an fp32 gate lies over rows 2 t and 2 t + 1 of bf16 outputs: other threads have yet to read it."""
    assert apart(abi.lib(), T=T, dtype=dtype, g=Q, gd=gate_dtype, gr=T) == 1
    assert "gate per channel or of another type" in _err(abi.lib())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("k", [0, 3])
@pytest.mark.parametrize("T,H", [(1, 512), (70, 256), (3000, 264), (1200, 2048)])
def test_out_over_a_row_of_its_own_tokens(T, H, k, dtype):
    """The residual, the shared rows, a gate per token of out's type and a dense block's rows may be out itself."""
    from test_gpu_norm import abi as lib, case, run_after
    rng = np.random.default_rng(T + H + k)
    d, P = case(rng, T, H, k, dtype, k > 0, True, "tokens", torch.float32)
    want, z = torch.empty(T, H, dtype=dtype, device="cuda"), torch.empty(T, H, dtype=dtype, device="cuda")
    run_after(d, T, H, k, P, "rms", "layer", 0.0, 0.5, 1.5, want, z)
    for key in ("r", "ys", "g") + (() if k else ("y",)):
        again, z2 = d[key].clone(), torch.empty_like(z)
        run_after({**d, key: again}, T, H, k, P, "rms", "layer", 0.0, 0.5, 1.5, again, z2)
        assert torch.equal(again, want) and torch.equal(z2, z), key
    assert lib().semmoe_check_errors() == 0


ROW = 64 * 2  # bytes of a row of `after` and `norm`


def at(p, rows):
    return ctypes.c_void_p(p.value + rows * ROW)


@pytest.mark.parametrize("kw,word", [
    (dict(r=at(Q, 1)), "out overlaps residual"), (dict(r=at(Q, -3)), "out overlaps residual"),
    (dict(ys=at(Q, 1)), "out overlaps y_shared"), (dict(q=None, y=at(Q, 2)), "out overlaps y_perm"),
    (dict(y=at(Q, -7), n=8), "out overlaps y_perm"), (dict(g=at(Q, -1), gr=4), "out overlaps gate"),
    (dict(g=at(Q, 3), gr=1, gd=0), "out overlaps gate"), (dict(q=at(Q, 1)), "out overlaps pair_to_sorted"),
    (dict(w=Q), "out overlaps topk_w"), (dict(pw=at(Q, 3)), "out overlaps post_weight"), (dict(pb=Q), "out overlaps post_bias"),
    (dict(nxt=1, no=at(Q, 1)), "next_out overlaps out"), (dict(nxt=1, no=at(Q, 4), r=at(Q, 5)), "next_out overlaps residual"),
    (dict(nxt=1, no=at(Q, 4), y=at(Q, 7)), "next_out overlaps y_perm"), (dict(nxt=1, no=at(Q, 4), nb=at(Q, 5)), "next_out overlaps next_bias"),
    (dict(nxt=2, no=at(Q, 4), nw=at(Q, 4)), "next_out overlaps next_weight"),
])
def test_outputs_lie_over_no_other_rows(abi, kw, word):  # noqa: F811
    """Buffers that begin at different rows of one tensor: other threads have yet to read what would be written over."""
    assert apart(abi.lib(), **kw) == 1
    assert word in _err(abi.lib())


@pytest.mark.parametrize("kw,word", [(dict(x=at(Q, 1)), "out overlaps x"), (dict(x=at(Q, -3)), "out overlaps x"),
                                     (dict(x=R, w=at(Q, 3)), "weight or bias"), (dict(x=R, b=at(Q, 2), wd=0), "weight or bias")])
def test_a_norm_lies_over_no_other_rows(abi, kw, word):  # noqa: F811
    assert norm(abi.lib(), out=Q, **{**dict(w=None), **kw}) == 1
    assert word in _err(abi.lib())
