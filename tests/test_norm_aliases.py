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
