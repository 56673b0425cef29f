"""Segment bounds of any value in the products grouped by expert: cut to [0, rows], or empty."""
import pytest
import torch

import block_quantized_moe_gb300 as ft
from test_gpu_train import DEV, check, normal, product_ref, wgrad_ref

pytestmark = pytest.mark.gpu
LO, HI = -(1 << 31), (1 << 31) - 1
# bounds, and the rows of each expert that follow from them (begin, end)
BOUNDS = [
    ([HI, -5, 3], [(0, 0), (0, 3)]),
    ([HI, LO, HI], [(0, 0), (0, None)]),
    ([LO, HI, LO], [(0, None), (0, 0)]),
    ([4, 2, HI], [(0, 0), (2, None)]),
    ([HI, HI, HI], [(0, 0), (0, 0)]),
    ([LO, LO, -1], [(0, 0), (0, 0)]),
]


@pytest.mark.parametrize("bounds,parts", BOUNDS)
# (the streaming kernel; the tensor cores; the general kernel)
@pytest.mark.parametrize("rows,n,k", [(6, 64, 64), (40, 64, 64), (6, 33, 47)])
def test_bounds_of_any_value(bounds, parts, rows, n, k):
    a, w = normal((rows, k), 1.0, torch.bfloat16, 1), normal((2, n, k), 0.1, torch.bfloat16, 2)
    c = normal((rows, n), 1.0, torch.bfloat16, 3)
    off = torch.tensor(bounds, dtype=torch.int32, device=DEV)
    # rows before and after the output's: nothing may be written there
    base = torch.full((3 * rows, n), float("nan"), device=DEV)
    out = base[rows:2 * rows]
    ft.ftmoe_grouped_matmul(a, off, w, out)
    dw = torch.empty(2, n, k, device=DEV)
    ft.ftmoe_grouped_matmul_wgrad(c, a, off, dw)
    written = torch.zeros(3 * rows, dtype=torch.bool, device=DEV)
    for e, (lo, hi) in enumerate(parts):
        hi = rows if hi is None else hi
        ref, mag = product_ref(a[lo:hi], w[e:], [hi - lo], False)
        check(out[lo:hi], ref, mag, k, "product")
        ref, mag = wgrad_ref(c[lo:hi], a[lo:hi], [hi - lo])
        check(dw[e:e + 1], ref, mag, rows, "weight gradient")
        written[rows + lo:rows + hi] = True
    assert torch.isnan(base[~written]).all()
    assert ft.ftmoe_read_error_flags() == 0


@pytest.mark.parametrize("kept", [False, True])
@pytest.mark.parametrize("n,k,rows", [(64, 64, 5), (33, 47, 5), (64, 64, 0)])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_experts_without_rows_keep_their_bits(n, k, rows, out, kept):
    """Accumulating into an expert without rows leaves every bit: zeros of both signs, NaN, subnormals."""
    k = 64 if kept else k
    c, x = normal((rows, n), 1.0, torch.bfloat16, 4), normal((rows, k), 1.0, torch.bfloat16, 5)
    dw = torch.zeros(3, n, k, dtype=out, device=DEV)
    dw[0, :, ::2], dw[0, 0, 1], dw[2, 0, 3], dw[2, -1], dw[2, 0, 0] = -0.0, float("nan"), 1e-40, -0.0, float("inf")
    old = dw.clone()
    off = torch.tensor([0, 0, rows, rows], dtype=torch.int32, device=DEV)
    if kept:
        q, s = torch.zeros(rows, k, dtype=torch.uint8, device=DEV), torch.full((rows, k // 32), 127, dtype=torch.uint8, device=DEV)
        ft.ftmoe_grouped_matmul_wgrad_saved(c, q, s, off, dw, accumulate=True)
    else:
        ft.ftmoe_grouped_matmul_wgrad(c, x, off, dw, accumulate=True)
    bits = torch.int32 if out == torch.float32 else torch.int16
    for e in (0, 2) if rows else (0, 1, 2):
        assert torch.equal(dw[e].view(bits), old[e].view(bits)), e
