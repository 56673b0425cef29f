"""fp32 weight gradients of uneven load: segments that are short on average and a few beyond the 1,024 rows
of one accumulator, whose parts are added in memory. Against 64-bit products.

Tolerances: an accumulator takes 1,024 terms in 64 additions, each losing at most 2^-23 of the partial
sum, and partial sums of independent terms are of the result's size: the error's norm stays below 64 2^-23
of the result's.
"""
import pytest
import torch

import block_quantized_moe_gb300 as ft
from test_gpu_train import DEV, check, normal, offsets_of, product_ref, saved, strided, wgrad_ref

pytestmark = pytest.mark.gpu
COUNTS = [3000, 0, 1100, 5, 70, 0, 1, 1025, 0, 1024, 0, 0, 2049, 0, 0, 64, 0, 0, 0, 0, 33, 0, 0, 0]
# padding of the output's rows: boxes, rows off 16 bytes (stored from registers)
OUTPUTS = [(264, 672, 0), (391, 672, 0), (264, 672, 4), (264, 672, 3), (391, 96, 5), (1100, 2080, 0)]


def output(n, k, pad, old):
    base, dw = strided((old.shape[0], n, k), pad, 0, torch.float32)
    dw.copy_(old)
    return base, dw


@pytest.mark.parametrize("n,k,pad", OUTPUTS)
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("kept", [False, True])
def test_parts_are_added_in_memory(n, k, pad, accumulate, kept):
    counts = COUNTS + [0] * 12   # 8,371 rows: at most 256 an expert on average
    R = sum(counts)
    assert R <= 256 * len(counts) and max(counts) > 1024
    _, dy = strided((R, n), -n % 8, 0, torch.bfloat16)
    dy.copy_(normal((R, n), 0.5, torch.bfloat16, 1))
    x = normal((R, k), 1.0, torch.bfloat16, 2)
    off, old = offsets_of(counts), normal((len(counts), n, k), 1.0, torch.float32, 3)
    if kept:
        q, s, x = saved(x)
    got = []
    for _ in range(2):
        base, dw = output(n, k, pad, old)
        if kept:
            ft.ftmoe_grouped_matmul_wgrad_saved(dy, q, s, off, dw, accumulate=accumulate)
        else:
            ft.ftmoe_grouped_matmul_wgrad(dy, x, off, dw, accumulate=accumulate)
        assert int((~torch.isnan(base)).sum()) == dw.numel()
        got.append(dw)
    ref, mag = wgrad_ref(dy, x, counts)
    if accumulate:
        ref, mag = ref + old.double(), mag + old.double().abs()
    check(got[0], ref, mag, max(counts) + 2, "weight gradient")
    rel = float((got[0].double() - ref).norm() / ref.norm())
    assert rel <= 64 * 2.0 ** -23, rel
    assert torch.equal(got[0], got[1])
    for e, c in enumerate(counts):
        if c == 0:
            assert torch.equal(got[0][e], old[e] if accumulate else torch.zeros_like(old[e]))
    assert ft.ftmoe_read_error_flags() == 0


@pytest.mark.parametrize("accumulate", [False, True])
def test_long_saved_sums(accumulate):
    """Kept rows, segments long on average: the same bound holds."""
    counts = [1, 9000, 300]
    R = sum(counts)
    dy, x = normal((R, 136), 0.5, torch.bfloat16, 4), normal((R, 160), 1.0, torch.bfloat16, 5)
    q, s, v = saved(x)
    got = normal((3, 136, 160), 1.0, torch.float32, 6)
    old = got.double() if accumulate else 0.0
    ft.ftmoe_grouped_matmul_wgrad_saved(dy, q, s, offsets_of(counts), got, accumulate=accumulate)
    ref = wgrad_ref(dy, v, counts)[0] + old
    assert float((got.double() - ref).norm() / ref.norm()) <= 64 * 2.0 ** -23


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("input_grad", [False, True])
def test_other_experts_rows_do_not_change_a_row(out, input_grad):
    """With the same number of rows in the call, a row's product has the same bits however the other
    rows are spread. (The number of rows chooses the kernel, and with it the order of the sum.)"""
    R, n, k = 500, 264, 1040
    a, w = normal((R, n if input_grad else k), 1.0, torch.bfloat16, 7), normal((4, n, k), 0.1, torch.bfloat16, 8)
    results = []
    for counts in ([100, 200, 100, 100], [100, 200, 0, 200], [100, 200, 1, 199]):
        y = torch.empty(R, k if input_grad else n, dtype=out, device=DEV)
        ft.ftmoe_grouped_matmul(a, offsets_of(counts), w, y, input_grad=input_grad)
        results.append(y[:300])
    assert torch.equal(results[0], results[1]) and torch.equal(results[0], results[2])


@pytest.mark.parametrize("kind", ["product", "input_grad", "weight_grad"])
def test_more_experts_than_the_tensor_core_kernel_takes(kind):
    """1,100 experts: the general kernel."""
    counts = [0] * 1100
    for e, c in ((0, 3), (511, 70), (1023, 1), (1024, 40), (1099, 5)):
        counts[e] = c
    R, n, k = sum(counts), 72, 104
    x, c = normal((R, k), 1.0, torch.bfloat16, 9), normal((R, n), 1.0, torch.bfloat16, 10)
    off = offsets_of(counts)
    if kind == "weight_grad":
        dw = torch.full((1100, n, k), float("nan"), device=DEV)
        ft.ftmoe_grouped_matmul_wgrad(c, x, off, dw)
        ref, mag = wgrad_ref(c, x, counts)
        check(dw, ref, mag, 70, kind)
        return
    w = normal((1100, n, k), 0.1, torch.bfloat16, 11)
    a, wide = (x, n) if kind == "product" else (c, k)
    y = torch.empty(R, wide, device=DEV)
    ft.ftmoe_grouped_matmul(a, off, w, y, input_grad=kind == "input_grad")
    ref, mag = product_ref(a, w, counts, kind == "input_grad")
    check(y, ref, mag, k if kind == "product" else n, kind)
