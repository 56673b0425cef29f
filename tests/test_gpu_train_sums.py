"""Long sums of the products grouped by expert with 16-bit outputs, against 64-bit products.

The tensor core cuts off what lies below its accumulator's last bit as it adds: over operands of one
sign that is a bias, growing with the number of additions. Tolerances, from the arithmetic: an
accumulator takes 2,048 terms in 128 additions (a weight gradient of up to 4,096 rows in fp16, 32,768
in bf16: all of them), which lose 2^-23 of the result each; the accumulators are added in fp32, each
sum within 2^-24; the output rounds once.
"""
import pytest
import torch

import block_quantized_moe_gb300 as ft
from test_gpu_train import DEV, DT, U, check, gen, normal, offsets_of, product_ref, saved, wgrad_ref

pytestmark = pytest.mark.gpu
LONG = 200_000


def positive(shape, mid, dtype, seed):
    return (torch.rand(shape, generator=gen(seed), device=DEV) + 0.5).mul_(mid).to(dtype)


def check_sum(got, ref, terms, per, what):
    """got within the tolerance of a sum of `terms` positive products, `per` to an accumulator"""
    tol = (per // 16 * 2.0 ** -23 + (terms // per + 1) * 2.0 ** -24 + U[got.dtype]) * ref.abs()
    err = (got.double() - ref).abs()
    assert (err <= tol).all(), f"{what}: {int((err > tol).sum())} of {err.numel()} outside, worst {float((err / tol.clamp(min=1e-300)).max()):.3g}"


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("input_grad", [False, True])
def test_product_of_long_rows(dtype, input_grad):
    counts, m = [40, 0, 3], 72
    n, k = (LONG, m) if input_grad else (m, LONG)
    a, w = positive((43, LONG), 1.0, DT[dtype], 1), positive((3, n, k), 0.1, DT[dtype], 2)
    got = torch.empty(43, m, dtype=DT[dtype], device=DEV)
    ft.ftmoe_grouped_matmul(a, offsets_of(counts), w, got, input_grad=input_grad)
    check_sum(got, product_ref(a, w, counts, input_grad)[0], LONG, 2048, "product")
    assert ft.ftmoe_read_error_flags() == 0


# many experts without rows: segments that are short on average, one that is not
@pytest.mark.parametrize("experts", [2, 500])
@pytest.mark.parametrize("dtype,rows,per", [("bf16", LONG, 2048), ("fp16", LONG, 2048), ("bf16", 32698, 32768),
                                            ("fp16", 4026, 4096), ("fp16", 32698, 2048)])
def test_weight_gradient_of_many_rows(dtype, rows, per, experts):
    counts = [rows] + [0] * (experts - 2) + [70]
    R, n, k = sum(counts), 136, 160
    dy, x = positive((R, n), 0.1, DT[dtype], 3), positive((R, k), 1.0, DT[dtype], 4)
    dw = torch.empty(experts, n, k, dtype=DT[dtype], device=DEV)
    ft.ftmoe_grouped_matmul_wgrad(dy, x, offsets_of(counts), dw)
    ref, _ = wgrad_ref(dy, x, counts)
    check_sum(dw, ref, rows, per, "weight gradient")
    assert ft.ftmoe_read_error_flags() == 0


@pytest.mark.parametrize("experts", [2, 1000])
@pytest.mark.parametrize("dtype,rows,per", [("bf16", LONG, 4096), ("fp16", LONG, 4096), ("bf16", 32698, 32768), ("fp16", 4026, 4096),
                                            ("fp16", 32698, 4096)])
def test_weight_gradient_of_many_saved_rows(dtype, rows, per, experts):
    """Where a segment takes several accumulators, they take 4,096 terms each."""
    counts = [rows] + [0] * (experts - 2) + [70]
    R, n, k = sum(counts), 136, 160
    dy, x = positive((R, n), 0.1, DT[dtype], 5), positive((R, k), 1.0, torch.bfloat16, 6)
    q, s, v = saved(x)
    dw = torch.empty(experts, n, k, dtype=DT[dtype], device=DEV)
    ft.ftmoe_grouped_matmul_wgrad_saved(dy, q, s, offsets_of(counts), dw)
    ref, _ = wgrad_ref(dy, v, counts)
    check_sum(dw, ref, rows, per, "weight gradient of saved rows")
    assert ft.ftmoe_read_error_flags() == 0


@pytest.mark.parametrize("empty,n,k", [(0, 1100, 2080), (120, 520, 1056), (120, 33, 64)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_saved_rows_long_and_short_segments_in_turn(empty, n, k, accumulate):
    """Segments of one accumulator and of several, one after another on the same CTA pairs."""
    counts = [4096, 4097, 100, 0, 9000, 64, 17000, 3] + [0] * empty
    R = sum(counts)
    dy, x = normal((R, n), 0.5, torch.bfloat16, 7), normal((R, k), 1.0, torch.bfloat16, 8)
    q, s, v = saved(x)
    old = normal((len(counts), n, k), 1.0, torch.bfloat16, 9)
    got = []
    for _ in range(3):
        dw = old.clone()
        ft.ftmoe_grouped_matmul_wgrad_saved(dy, q, s, offsets_of(counts), dw, accumulate=accumulate)
        got.append(dw)
    ref, mag = wgrad_ref(dy, v, counts)
    if accumulate:
        ref, mag = ref + old.double(), mag + old.double().abs()
    check(got[0], ref, mag, max(counts), "weight gradient of saved rows")
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])
    assert ft.ftmoe_read_error_flags() == 0
