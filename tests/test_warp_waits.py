"""Waits of loops that a whole warp runs: one answer for all lanes, and a bounded end."""
import glob
import os
import re

import numpy as np
import pytest
import torch

import oracle
from test_gpu_mx4 import abi, cuda, operands
from parity_utils import np_

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "token_expert_routing_gb300", "csrc")


def kernels():
    """(file, text) of every kernel in which a lane elected of a whole warp issues."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        with open(path) as f:
            for text in re.split(r"^__global__", f.read(), flags=re.M)[1:]:
                if "elect_one()" in text.split("\n}\n")[0]:
                    yield os.path.basename(path), text.split("\n}\n")[0]


def test_warp_wide_loops_wait_with_one_answer():
    """A wait whose lanes may answer differently (mbar_wait, wait_for) is met by one lane alone in these kernels;
    polls of the whole warp are voted on, since elect.sync needs every lane at the same place."""
    found = list(kernels())
    assert {f for f, _ in found} == {"mx4_gemm.cu", "route_tc.cu"}
    for name, text in found:
        for line in text.splitlines():
            code = line.split("//")[0]
            if re.search(r"\b(mbar_wait|wait_for)\(", code):
                assert "lane == 0" in code, (name, line)
            if "mbar_try_wait(" in code:
                assert "__all_sync" in code, (name, line)


def test_the_cluster_choice_waits_with_one_answer():
    """Every lane acquires the copies and the warp then chooses together."""
    with open(os.path.join(CSRC, "route_tc.cu")) as f:
        line = next(l for l in f if "mbar_wait" in l and "recv_bar" in l)
    assert "mbar_wait_warp(" in line


@pytest.mark.gpu
def test_mx4_product_whose_wait_runs_out_ends_and_the_next_is_right():
    import time
    a = abi()
    rng = np.random.default_rng(5)
    count, N, K = [300, 0, 5, 140], 520, 2080
    P, E = sum(count), len(count)
    (x, xs, w, ws), xv, wv = operands(rng, P, E, N, K, count)
    off, pe = np.concatenate([[0], np.cumsum(count)]), np.arange(E)
    args = (x, xs, cuda(off, torch.int32), cuda(pe, torch.int32), w, ws, P, E, N, K)
    y = torch.full((P, N), 77.0, device="cuda")
    t0 = time.perf_counter()
    a.semmoe_selftest_mx4_wait(*args, y)
    with pytest.raises(a.SemMoEError) as ei:
        a.semmoe_check_errors()
    assert ei.value.code == a.SEMMOE_ERR_DEVICE_TIMEOUT
    assert ei.value.bits & a.SEMMOE_DEVERR_TIMEOUT
    assert 0.1 < time.perf_counter() - t0 < 60
    assert (np_(y) == 77.0).all()
    assert a.semmoe_check_errors() == 0
    a.semmoe_mx4_grouped_gemm(*args, y)
    assert a.semmoe_check_errors() == 0
    size = oracle.mx4_grouped_product(np.abs(xv), np.abs(wv), off, pe)
    # K exact products summed in fp32: at most 2^-23 of the sum of magnitudes a step
    assert (np.abs(np_(y) - oracle.mx4_grouped_product(xv, wv, off, pe)) <= K * 2.0 ** -23 * size).all()


def test_mx4_wait_selftest_refusals():
    import ctypes
    from token_expert_routing_gb300 import _abi, build
    build.build()
    p = ctypes.c_void_p(4096)
    call = lambda P=8, a=p, K=64: _abi.lib().semmoe_selftest_mx4_wait(a, p, p, p, p, p, P, 4, 64, K, p, None)  # noqa: E731
    for kw, word in ((dict(P=0), "P=0"), (dict(P=4097), "P=4097"), (dict(a=None), "null"), (dict(K=40), "K = 40")):
        assert call(**kw) == 1, kw
        assert word in _abi.lib().semmoe_last_error().decode(), kw
