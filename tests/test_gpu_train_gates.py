"""Backward pass of SiLU-and-mul from kept rows where gates are very large, against 64-bit formulas."""
import pytest
import torch

import block_quantized_moe_gb300 as ft
from test_gpu_train import DEV, DT, backward_check, gen, normal, save

pytestmark = pytest.mark.gpu
GATES = [3e38, -3e38, 2.4e38, 2.3e38, -2.4e38, 1e38, 1e30, -1e30, 1e10, -1e10, 1000.0, -1000.0, 130.0, 100.0, -100.0, -88.0]


@pytest.mark.parametrize("fmt", [ft.FMT_FP8, ft.FMT_MXFP8])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("inter", [160, 1056])
def test_gradients_at_very_large_gates(fmt, dtype, inter):
    """One gate of each size to a row; the kept values are the operands of the formula, and every
    gradient is finite."""
    rows = len(GATES)
    gu = normal((rows, 2 * inter), 1.0, torch.float32, 1)
    gu[:, 5] = torch.tensor(GATES, device=DEV)
    gu[:, inter + 5] = 0.75
    h, q, s, kept = save(gu.to(DT[dtype]), fmt, DT[dtype])
    assert torch.isfinite(h).all()
    dh = normal((rows, inter), 0.3, torch.float32, 2).clamp(-0.9, 0.9).to(DT[dtype])
    w = torch.rand(rows, generator=gen(3), device=DEV)
    dgu = torch.empty(rows, 2 * inter, dtype=DT[dtype], device=DEV)
    hw, dwt = torch.empty(rows, inter, dtype=DT[dtype], device=DEV), torch.empty(rows, device=DEV)
    ft.ftmoe_silu_mul_backward(q, s, dh, dgu, hw=hw, row_weights=w, dweights=dwt, fmt=fmt)
    backward_check(kept[:, :inter], kept[:, inter:], dh, w, dgu, hw, dwt, inter)
    for t in (dgu, hw, dwt):
        assert torch.isfinite(t).all()


@pytest.mark.parametrize("fmt", [ft.FMT_FP8, ft.FMT_MXFP8])
def test_infinite_and_nan_gates_reach_their_gradients_only(fmt):
    """A gate kept as NaN or from an infinity gives non-finite gradients in its own row, none elsewhere."""
    rows, inter = 5, 160
    gu = normal((rows, 2 * inter), 1.0, torch.bfloat16, 4)
    gu[1, 5], gu[2, 5], gu[3, 5] = float("inf"), float("-inf"), float("nan")
    _, q, s, _ = save(gu, fmt, torch.bfloat16)
    dh = normal((rows, inter), 0.3, torch.bfloat16, 5)
    dgu = torch.empty(rows, 2 * inter, dtype=torch.bfloat16, device=DEV)
    dwt = torch.empty(rows, device=DEV)
    ft.ftmoe_silu_mul_backward(q, s, dh, dgu, dweights=dwt, fmt=fmt)
    assert torch.isfinite(dgu[[0, 4]]).all() and torch.isfinite(dwt[[0, 4]]).all()
    assert not torch.isfinite(dwt[1:4]).any() and not torch.isfinite(dgu[1:4, inter + 5]).any()
