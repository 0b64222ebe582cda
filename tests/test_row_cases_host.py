"""The timed cases of the row operators (perf/more_operators.py) bring the workspace that the library asks for."""
import importlib.util
import os
import random

import pytest

from helpers import ROOT, ensure_built, gpu_available

spec = importlib.util.spec_from_file_location("more_operators", os.path.join(ROOT, "perf", "more_operators.py"))
cases = importlib.util.module_from_spec(spec)
spec.loader.exec_module(cases)

# drawn sizes whose gradients need copies of x and w beside dz and the parts
LARGE = [dict(op="matmul_bwd", m=45652, k=1451, n=120, bias=True, act="silu", dtype="bf16"),
         dict(op="matmul_bwd", m=68022, k=933, n=91, bias=True, act="none", dtype="bf16"),
         dict(op="matmul_bwd", m=81, k=5380, n=11478, bias=False, act="silu", dtype="bf16"),
         dict(op="matmul_bwd", m=31000, k=1001, n=250, bias=True, act="gelu", dtype="f32"),
         dict(op="matmul", m=1000, k=8191, n=4096, bias=True, act="relu", dtype="f32", residual=False, keep=False)]


def test_workspaces():
    ensure_built()
    import cnn_convolution_conv2d_amd as c2
    rng = random.Random(1)
    for case in cases.listed() + LARGE + [cases.draw(rng) for _ in range(20000)]:
        given, m, op = cases.workspace_bytes(case), case["m"], case["op"]
        dt = c2.F32 if case["dtype"] == "f32" else c2.BF16
        if op in ("matmul", "matmul_bwd"):
            size = c2.conv2d_matmul_workspace_bytes if op == "matmul" else c2.conv2d_matmul_bwd_workspace_bytes
            assert given >= size(m, case["k"], case["n"], dt), case
        elif op == "rms_bwd":
            assert given >= c2.conv2d_rms_norm_bwd_workspace_bytes(m, case["c"]) > 0, case
        elif op == "rms_linear":
            assert given >= c2.conv2d_int8_matmul_workspace_bytes(m, case["c"], case["n"]), case


@pytest.mark.gpu
@pytest.mark.parametrize("case", LARGE, ids=lambda c: f"{c['op']}-{c['m']}-{c['k']}-{c['n']}-{c['dtype']}")
def test_large_workspaces_on_the_gpu(case, monkeypatch):
    """A pass is not refused, and every output is written."""
    if not gpu_available():
        pytest.skip("no GPU")
    import torch
    ensure_built()
    monkeypatch.setattr(cases, "own", True)
    state = cases.prepare(case, 1)
    for name in ("dx", "dw", "dbias", "y"):
        if state.get(name) is not None:
            state[name].fill_(float("nan"))
    for out in cases.run(state):
        assert out is None or bool(torch.isfinite(out).all())
