"""Products grouped by expert in 16 bits (three directions) and SiLU-and-mul with activations kept
in 8 bits, against plain 64-bit implementations.

Tolerances, fixed from the arithmetic. A sum of K products in fp32, in any order and however a
tensor core groups it, is within K 2^-24 sum|products| of the exact one (Higham's gamma_K); an
output type then rounds by its unit roundoff: 2^-8 (bf16, 8 significant bits), 2^-11 (fp16, 11
bits; 2^-25 at least), 2^-24 (fp32). Codes and scales are compared bit for bit.
"""
import numpy as np
import pytest
import torch

import block_quantized_moe_gb300 as ft

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = {t: torch.finfo(t).eps / 2 for t in (torch.bfloat16, torch.float16, torch.float32)}  # unit roundoff
TINY = {torch.bfloat16: 1e-38, torch.float16: 2.0 ** -25, torch.float32: 1e-38}
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def normal(shape, std, dtype, seed):
    return torch.randn(shape, generator=gen(seed), device=DEV, dtype=torch.float32).mul_(std).to(dtype)


def strided(shape, pad, shift, dtype):
    """A [.., rows, cols] view with row stride cols + pad, `shift` elements into its storage;
    everything around it holds NaN."""
    lead, cols = shape[:-1], shape[-1]
    n = int(np.prod(lead)) * (cols + pad) + shift + 64
    base = torch.full((n,), float("nan"), dtype=dtype, device=DEV)
    strides = [cols + pad, 1]
    for d in reversed(shape[1:-1]):
        strides.insert(0, strides[0] * d)
    return base, base[shift:].as_strided(shape, strides)


def offsets_of(counts):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device=DEV)


def check(got, ref, mag, terms, what):
    """got within terms * 2^-24 * mag + the rounding of its type of ref."""
    tol = terms * 2.0 ** -24 * mag + U[got.dtype] * (ref.abs() + terms * 2.0 ** -24 * mag) + TINY[got.dtype]
    err = (got.double() - ref).abs()
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst {float((err / tol).nan_to_num(1e9).max()):.3g}"


def product_ref(a, w, counts, input_grad):
    """(reference, magnitude) in 64 bits"""
    width = w.shape[2] if input_grad else w.shape[1]
    ref = torch.zeros(a.shape[0], width, dtype=torch.float64, device=DEV)
    mag = torch.zeros_like(ref)
    lo = 0
    for e, c in enumerate(counts):
        m = w[e].double() if input_grad else w[e].double().T
        ref[lo:lo + c] = a[lo:lo + c].double() @ m
        mag[lo:lo + c] = a[lo:lo + c].double().abs() @ m.abs()
        lo += c
    return ref, mag


# (counts, n, k): one row; few rows; empty experts at both ends; odd widths; tiles' edges; one
# expert; sizes off every tile
SHAPES = [
    ([1], 16, 16),
    ([0, 1, 0], 64, 48),
    ([2, 0, 3, 1], 136, 200),
    ([0, 5, 0, 0, 40, 0], 72, 1000),
    ([31, 32, 33, 1], 256, 128),
    ([127, 128, 129], 264, 512),
    ([255, 256, 257, 0, 2], 384, 320),
    ([700, 3], 520, 776),
    ([0, 0, 0], 64, 64),
    ([5, 9], 33, 47),      # widths that no 16-byte copy takes
    ([17, 1, 64], 1, 7),
    ([64] * 9, 8, 1024),
    ([1, 1200], 264, 136),  # segments long on average
]


@pytest.mark.parametrize("counts,n,k", SHAPES)
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("fp16", "fp32"), ("bf16", "fp32"), ("fp16", "bf16")])
@pytest.mark.parametrize("input_grad", [False, True])
def test_product(counts, n, k, dtype, out, input_grad):
    R, E = sum(counts), len(counts)
    a = normal((R, n if input_grad else k), 1.0, DT[dtype], 1)
    w = normal((E, n, k), 0.1, DT[dtype], 2)
    o = torch.empty(R, k if input_grad else n, dtype=DT[out], device=DEV)
    ft.ftmoe_grouped_matmul(a, offsets_of(counts), w, o, input_grad=input_grad)
    ref, mag = product_ref(a, w, counts, input_grad)
    check(o, ref, mag, n if input_grad else k, "product")
    assert ft.ftmoe_read_error_flags() == 0


@pytest.mark.parametrize("counts", [[1], [1, 0, 1], [0, 0, 4], [5, 0, 0], [0] * 300 + [1, 0, 2] + [0] * 250, [16]])
@pytest.mark.parametrize("n,k", [(8, 8), (24, 2056), (264, 768), (1000, 4104)])
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("fp16", "fp32"), ("bf16", "fp16")])
def test_product_of_a_handful_of_rows(counts, n, k, dtype, out):
    """Decode sizes: rows of one expert and of several, experts without rows around them, weight
    rows that end inside a lane's pieces; rows past the last segment are not written."""
    R, E = sum(counts), len(counts)
    a = normal((R + 1, k), 1.0, DT[dtype], 61)
    w = normal((E, n, k), 0.1, DT[dtype], 62)
    o = torch.full((R + 1, n), float("nan"), dtype=DT[out], device=DEV)
    ft.ftmoe_grouped_matmul(a, offsets_of(counts), w, o)
    ref, mag = product_ref(a[:R], w, counts, False)
    check(o[:R], ref, mag, k, "product")
    assert torch.isnan(o[R]).all()


@pytest.mark.parametrize("pad,shift", [(8, 0), (8, 8), (3, 0), (1, 5), (64, 24)])
@pytest.mark.parametrize("input_grad", [False, True])
def test_product_strides_and_rows_past_the_end(pad, shift, input_grad):
    """Row strides and bases, aligned or not; rows past offsets[E] hold NaN, are not used and not
    written; nothing around the outputs is written."""
    counts, n, k, extra = [3, 0, 65, 20], 136, 264, 7
    R, E = sum(counts), len(counts)
    wide, outw = (n, k) if input_grad else (k, n)
    _, a = strided((R + extra, wide), pad, shift, torch.bfloat16)
    a[:R] = normal((R, wide), 1.0, torch.bfloat16, 3)
    _, w = strided((E, n, k), pad, shift, torch.bfloat16)
    w.copy_(normal((E, n, k), 0.1, torch.bfloat16, 4))
    base, o = strided((R + extra, outw), pad, shift, torch.bfloat16)
    ft.ftmoe_grouped_matmul(a, offsets_of(counts), w, o, input_grad=input_grad)
    ref, mag = product_ref(a[:R], w, counts, input_grad)
    check(o[:R], ref, mag, n if input_grad else k, "product")
    assert torch.isnan(o[R:]).all()
    assert int((~torch.isnan(base)).sum()) == R * outw


@pytest.mark.parametrize("counts,n,k", [([3, 0, 70], 33, 47), ([130, 300], 257, 131), ([40], 1, 1), ([600, 500], 391, 259)])
@pytest.mark.parametrize("out", ["bf16", "fp32"])
def test_odd_widths_in_aligned_rows(counts, n, k, out):
    """Widths that no vector divides, in rows whose starts are 16-byte aligned: the copies end
    inside a vector, and what pads the rows (NaN) is neither used nor written."""
    R, E = sum(counts), len(counts)
    off = offsets_of(counts)

    def padded(shape, dtype, std=None, seed=0):
        base, t = strided(shape, -shape[-1] % 8 + 8, 0, dtype)
        if std is not None:
            t.copy_(normal(shape, std, dtype, seed))
        return base, t
    _, a = padded((R, k), torch.bfloat16, 1.0, 71)
    _, c = padded((R, n), torch.bfloat16, 0.5, 72)
    _, w = padded((E, n, k), torch.bfloat16, 0.1, 73)
    by, y = padded((R, n), DT[out])
    ft.ftmoe_grouped_matmul(a, off, w, y)
    ref, mag = product_ref(a, w, counts, False)
    check(y, ref, mag, k, "product")
    bd, da = padded((R, k), DT[out])
    ft.ftmoe_grouped_matmul(c, off, w, da, input_grad=True)
    ref, mag = product_ref(c, w, counts, True)
    check(da, ref, mag, n, "input gradient")
    bw, dw = padded((E, n, k), DT[out])
    ft.ftmoe_grouped_matmul_wgrad(c, a, off, dw)
    ref, mag = wgrad_ref(c, a, counts)
    check(dw, ref, mag, max(counts), "weight gradient")
    ft.ftmoe_grouped_matmul_wgrad(c, a, off, dw, accumulate=True)
    check(dw, 2 * ref, 2 * mag + ref.abs(), max(counts) + 2 + (2 ** 15 if out == "bf16" else 0), "accumulated")
    for base, t in ((by, y), (bd, da), (bw, dw)):
        assert int((~torch.isnan(base)).sum()) == t.numel()
    assert ft.ftmoe_read_error_flags() == 0


@pytest.mark.parametrize("input_grad", [False, True])
def test_product_keeps_infinities_and_nan_in_their_rows(input_grad):
    """A NaN or infinite row of one expert changes no other row, and gives NaN or infinities itself."""
    counts, n, k = [40, 30, 0, 70], 128, 192
    R, E = sum(counts), len(counts)
    wide = n if input_grad else k
    a = normal((R, wide), 1.0, torch.bfloat16, 5)
    w = normal((E, n, k), 0.1, torch.bfloat16, 6)
    o1 = torch.empty(R, k if input_grad else n, dtype=torch.float32, device=DEV)
    o2 = torch.empty_like(o1)
    ft.ftmoe_grouped_matmul(a, offsets_of(counts), w, o1, input_grad=input_grad)
    b = a.clone()
    b[39], b[70], b[139] = float("nan"), float("inf"), float("-inf")
    ft.ftmoe_grouped_matmul(b, offsets_of(counts), w, o2, input_grad=input_grad)
    keep = torch.ones(R, dtype=torch.bool, device=DEV)
    keep[[39, 70, 139]] = False
    assert torch.equal(o1[keep], o2[keep])
    assert torch.isnan(o2[39]).all() and not torch.isfinite(o2[[70, 139]]).any()


def test_product_offsets_out_of_range_are_clamped():
    """Bounds outside [0, rows] and decreasing ones: clamped or empty, nothing past the rows is written."""
    n = k = 64
    a = normal((10, k), 1.0, torch.bfloat16, 7)
    w = normal((4, n, k), 0.1, torch.bfloat16, 8)
    base = torch.full((20, n), float("nan"), dtype=torch.float32, device=DEV)
    ft.ftmoe_grouped_matmul(a, torch.tensor([-5, 4, 2, 6, 99], dtype=torch.int32, device=DEV), w, base[:10])
    assert torch.isnan(base[10:]).all()
    ref, mag = product_ref(a[:4], w, [4], False)
    # rows 2, 3 belong to expert 0 and to expert 2: either is a valid owner
    check(base[:2], ref[:2], mag[:2], k, "rows of expert 0")
    ref, mag = product_ref(a[6:], w[3:], [4], False)
    check(base[6:10], ref, mag, k, "rows of expert 3")


def test_product_wide_strides_past_32_bits():
    """Expert strides whose element offsets pass 2^31 and 2^32."""
    n, k, E, counts = 72, 128, 3, [5, 70, 33]
    stride = (1 << 31) + 64
    base = torch.empty(2 * stride + n * k, dtype=torch.bfloat16, device=DEV)
    w = base.as_strided((E, n, k), (stride, k, 1))
    w.copy_(normal((E, n, k), 0.1, torch.bfloat16, 9))
    for input_grad in (False, True):
        a = normal((sum(counts), n if input_grad else k), 1.0, torch.bfloat16, 10)
        o = torch.empty(sum(counts), k if input_grad else n, dtype=torch.float32, device=DEV)
        ft.ftmoe_grouped_matmul(a, offsets_of(counts), w, o, input_grad=input_grad)
        ref, mag = product_ref(a, w, counts, input_grad)
        check(o, ref, mag, n if input_grad else k, "product")
    x = normal((sum(counts), k), 1.0, torch.bfloat16, 11)
    dy = normal((sum(counts), n), 1.0, torch.bfloat16, 12)
    ft.ftmoe_grouped_matmul_wgrad(dy, x, offsets_of(counts), w)
    ref, mag = wgrad_ref(dy, x, counts)
    check(w, ref, mag, max(counts), "weight gradient")


def wgrad_ref(dy, x, counts):
    ref = torch.zeros(len(counts), dy.shape[1], x.shape[1], dtype=torch.float64, device=DEV)
    mag = torch.zeros_like(ref)
    lo = 0
    for e, c in enumerate(counts):
        d, v = dy[lo:lo + c].double(), x[lo:lo + c].double()
        ref[e], mag[e] = d.T @ v, d.abs().T @ v.abs()
        lo += c
    return ref, mag


def saved(x):
    """x kept in MXFP8 by the library's quantizer: (codes, scales, the values they stand for)."""
    q, s, _ = ft.quantize_act(x.to(torch.bfloat16), ft.FMT_MXFP8)
    v = q.view(torch.float8_e4m3fn).double().view(x.shape[0], x.shape[1] // 32, 32) * torch.exp2(s.double() - 127)[..., None]
    return q, s, v.view(x.shape)


@pytest.mark.parametrize("counts,n,k", SHAPES)
@pytest.mark.parametrize("dtype,out", [("bf16", "fp32"), ("fp16", "fp16"), ("bf16", "bf16"), ("fp16", "bf16")])
def test_weight_gradient(counts, n, k, dtype, out):
    R, E = sum(counts), len(counts)
    dy, x = normal((R, n), 0.5, DT[dtype], 13), normal((R, k), 1.0, DT[dtype], 14)
    dw = torch.full((E, n, k), float("nan"), dtype=DT[out], device=DEV)
    ft.ftmoe_grouped_matmul_wgrad(dy, x, offsets_of(counts), dw)
    ref, mag = wgrad_ref(dy, x, counts)
    check(dw, ref, mag, max(max(counts), 1), "weight gradient")
    old = normal((E, n, k), 1.0, DT[out], 15)
    dw = old.clone()
    ft.ftmoe_grouped_matmul_wgrad(dy, x, offsets_of(counts), dw, accumulate=True)
    check(dw, ref + old.double(), mag + old.double().abs(), max(counts) + 2, "accumulated")
    for e, c in enumerate(counts):
        if c == 0:
            assert torch.equal(dw[e], old[e])
    assert ft.ftmoe_read_error_flags() == 0


@pytest.mark.parametrize("counts,n,k", [([1], 16, 32), ([0, 3, 0, 17], 136, 96), ([63, 64, 65, 1], 264, 320),
                                        ([300, 0, 129], 128, 544), ([0, 0], 64, 64), ([15, 16, 17], 33, 64),
                                        ([400, 77, 1000], 264, 672)])
@pytest.mark.parametrize("dtype,out", [("bf16", "fp32"), ("fp16", "fp16"), ("bf16", "bf16")])
def test_weight_gradient_from_saved_rows(counts, n, k, dtype, out):
    R, E = sum(counts), len(counts)
    dy, x = normal((R, n), 0.5, DT[dtype], 16), normal((R, k), 1.0, torch.float32, 17)
    if R:
        x[:, :32] *= 2.0 ** 7      # groups of other magnitudes
        x[R // 2] = 0.0
    q, s, v = saved(x)
    dw = torch.full((E, n, k), float("nan"), dtype=DT[out], device=DEV)
    ft.ftmoe_grouped_matmul_wgrad_saved(dy, q, s, offsets_of(counts), dw)
    ref, mag = wgrad_ref(dy, v, counts)
    check(dw, ref, mag, max(max(counts), 1), "weight gradient of saved rows")
    old = normal((E, n, k), 1.0, DT[out], 18)
    dw = old.clone()
    ft.ftmoe_grouped_matmul_wgrad_saved(dy, q, s, offsets_of(counts), dw, accumulate=True)
    check(dw, ref + old.double(), mag + old.double().abs(), max(counts) + 2, "accumulated")
    assert ft.ftmoe_read_error_flags() == 0


@pytest.mark.parametrize("kept", [False, True])
def test_weight_gradient_rows_of_other_experts_do_not_leak(kept):
    """NaN and infinite rows before, after and past an expert's segment leave its gradient alone
    (its last rows share a tile with theirs)."""
    counts, n, k, extra = [37, 21, 50], 136, 160, 9
    R = sum(counts) + extra
    dy, x = normal((R, n), 0.5, torch.bfloat16, 19), normal((R, k), 1.0, torch.bfloat16, 20)
    dy[:37], x[:37], dy[58:], x[58:] = float("nan"), float("inf"), float("-inf"), float("nan")
    dw = torch.zeros(3, n, k, dtype=torch.float32, device=DEV)
    if kept:
        q, s, v = saved(torch.where(torch.isfinite(x), x, torch.zeros_like(x)))
        q[:37], q[58:] = 0x7F, 0x7F    # NaN codes
        s[:37], s[58:] = 0xFF, 0xFE
        ft.ftmoe_grouped_matmul_wgrad_saved(dy, q, s, offsets_of(counts), dw)
    else:
        v = x.double()
        ft.ftmoe_grouped_matmul_wgrad(dy, x, offsets_of(counts), dw)
    ref, mag = wgrad_ref(dy[37:58], v[37:58], [21])
    check(dw[1:2], ref, mag, 21, "middle expert")
    assert torch.isnan(dw[0]).all() and torch.isnan(dw[2]).all()


@pytest.mark.parametrize("pad,shift", [(8, 8), (3, 0), (1, 5), (24, 16)])
def test_weight_gradient_strides(pad, shift):
    counts, n, k = [3, 0, 65, 20], 136, 264
    R, E = sum(counts), len(counts)
    _, dy = strided((R, n), pad, shift, torch.bfloat16)
    dy.copy_(normal((R, n), 0.5, torch.bfloat16, 21))
    _, x = strided((R, k), pad, shift, torch.bfloat16)
    x.copy_(normal((R, k), 1.0, torch.bfloat16, 22))
    base, dw = strided((E, n, k), pad, shift, torch.float32)
    ft.ftmoe_grouped_matmul_wgrad(dy, x, offsets_of(counts), dw)
    ref, mag = wgrad_ref(dy, x, counts)
    check(dw, ref, mag, max(counts), "weight gradient")
    assert int((~torch.isnan(base)).sum()) == E * n * k


@pytest.mark.parametrize("kind", ["product", "input_grad", "weight_grad", "saved"])
@pytest.mark.parametrize("accumulate", [False, True])
def test_long_sums_keep_fp32(kind, accumulate):
    """fp32 outputs of long contractions. An accumulator takes 512 terms in 32 additions (up to
    2,048 in 128 from saved rows), each losing at most 2^-23 of the partial sum, and the partial
    sums are of the result's size (independent terms): the error's norm is below 32 (128) 2^-23 of it."""
    if accumulate and kind in ("product", "input_grad"):
        pytest.skip("only weight gradients accumulate")
    counts, long, m = [1, 9000, 300], 16384, 136
    off = offsets_of(counts)
    if kind in ("product", "input_grad"):
        counts = [70, 0, 40]
        n, k = (m, long) if kind == "product" else (long, m)
        a, w = normal((110, long), 1.0, torch.bfloat16, 63), normal((3, n, k), 0.1, torch.bfloat16, 64)
        got = torch.empty(110, m, device=DEV)
        ft.ftmoe_grouped_matmul(a, offsets_of(counts), w, got, input_grad=kind == "input_grad")
        ref, mag = product_ref(a, w, counts, kind == "input_grad")
    else:
        R = sum(counts)
        dy, x = normal((R, m), 0.5, torch.bfloat16, 65), normal((R, 160), 1.0, torch.bfloat16, 66)
        got = normal((3, m, 160), 1.0, torch.float32, 67)
        old = got.double() if accumulate else 0.0
        if kind == "saved":
            q, s, x = saved(x)
            ft.ftmoe_grouped_matmul_wgrad_saved(dy, q, s, off, got, accumulate=accumulate)
        else:
            ft.ftmoe_grouped_matmul_wgrad(dy, x, off, got, accumulate=accumulate)
        ref, mag = wgrad_ref(dy, x, counts)
        ref = ref + old
    check(got, ref, mag + ref.abs(), long, kind)
    rel = float((got.double() - ref).norm() / ref.norm())
    assert rel <= (128 if kind == "saved" else 32) * 2.0 ** -23, rel


def test_gradients_agree_with_differences():
    """L = <c, product>: L's change along random directions of a and w against the two gradients
    (the product is linear in each, so the difference is exact up to rounding)."""
    counts, n, k = [30, 0, 50, 7], 128, 192
    R, E = sum(counts), len(counts)
    a, w = normal((R, k), 1.0, torch.bfloat16, 23), normal((E, n, k), 0.1, torch.bfloat16, 24)
    c = normal((R, n), 0.5, torch.bfloat16, 25)
    off = offsets_of(counts)
    da = torch.empty(R, k, dtype=torch.float32, device=DEV)
    dw = torch.empty(E, n, k, dtype=torch.float32, device=DEV)
    ft.ftmoe_grouped_matmul(c, off, w, da, input_grad=True)
    ft.ftmoe_grouped_matmul_wgrad(c, a, off, dw)
    va, vw = normal((R, k), 1.0, torch.float32, 26).double(), normal((E, n, k), 1.0, torch.float32, 27).double()

    def loss(a_, w_):
        return float((product_ref(a_, w_, counts, False)[0] * c.double()).sum())
    for grad, v, step in ((da, va, lambda h: (a.double() + h * va, w.double())),
                          (dw, vw, lambda h: (a.double(), w.double() + h * vw))):
        diff = (loss(*step(0.5)) - loss(*step(-0.5)))
        inner = float((grad.double() * v).sum())
        # each gradient value is within gamma_K of exact: 192 2^-24 relative to its terms' sum
        scale = float((grad.double().abs() * v.abs()).sum())
        assert abs(diff - inner) <= 1e-4 * scale


@pytest.mark.parametrize("inter", [1, 7, 32, 100, 128, 250, 768, 1024, 2048, 2080])
@pytest.mark.parametrize("rows", [1, 2, 67])
@pytest.mark.parametrize("fmt", [ft.FMT_FP8, ft.FMT_MXFP8])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_silu_saved(inter, rows, fmt, dtype):
    if fmt == ft.FMT_MXFP8 and inter % 32:
        pytest.skip("MXFP8 rows are whole groups of 32")
    dt = DT[dtype]
    gu = normal((rows, 2 * inter), 2.0, dt, 30)
    gu[0, : inter // 2] = 0.0                     # a group of zeros, or part of one
    gu[rows - 1] *= 12.0                          # exp(-g) beyond fp32's range of 1 + exp(-g)
    h, q, s, kept = save(gu, fmt, dt)
    g, u = gu[:, :inter].double(), gu[:, inter:].double()
    ref = g / (1 + torch.exp(-g)) * u
    # exp, a sum, a quotient and a product: 8 units of fp32, then h's own rounding
    check(h, ref, ref.abs(), 8, "h")
    kg, ku = kept[:, :inter], kept[:, inter:]
    # half a step of e4m3: 2^-4 of the value, or 2^-10 of the group's scale (at most amax/256)
    for half, k8 in ((g, kg), (u, ku)):
        grp = 128 if fmt == ft.FMT_FP8 else 32
        for c in range(0, inter, grp):
            part, amax = half[:, c:c + grp], half[:, c:c + grp].abs().amax(1, keepdim=True)
            # (MXFP8 saturates at 448 of its scale: up to 1/8 of the largest value)
            tol = part.abs() / 16 + amax / 256 * 2.0 ** -10 + (part.abs() >= amax * 0.875) * part.abs() / 8 * (grp == 32)
            assert ((part - k8[:, c:c + grp]).abs() <= tol * 1.0001 + 1e-30).all()
    dh = normal((rows, inter), 0.3, dt, 31)
    w = torch.rand(rows, generator=gen(32), device=DEV)
    dgu = torch.full((rows, 2 * inter), float("nan"), dtype=dt, device=DEV)
    hw = torch.full((rows, inter), float("nan"), dtype=dt, device=DEV)
    dwt = torch.full((rows,), float("nan"), device=DEV)
    ft.ftmoe_silu_mul_backward(q, s, dh, dgu, hw=hw, row_weights=w, dweights=dwt, fmt=fmt)
    backward_check(kg, ku, dh, w, dgu, hw, dwt, inter)
    # without weights and without the optional outputs
    dgu1 = torch.empty_like(dgu)
    ft.ftmoe_silu_mul_backward(q, s, dh, dgu1, fmt=fmt)
    backward_check(kg, ku, dh, torch.ones_like(w), dgu1, None, None, inter)


def save(gu, fmt, dt):
    rows, inter = gu.shape[0], gu.shape[1] // 2
    h = torch.full((rows, inter), float("nan"), dtype=dt, device=DEV)
    q = torch.full((rows, 2 * inter), 0xAA, dtype=torch.uint8, device=DEV)
    groups = -(-inter // 128) if fmt == ft.FMT_FP8 else inter // 32
    s = torch.zeros(rows, 2 * groups, dtype=torch.float32 if fmt == ft.FMT_FP8 else torch.uint8, device=DEV)
    ft.ftmoe_silu_mul_save(gu, h, q, s, fmt=fmt)
    size = 128 if fmt == ft.FMT_FP8 else 32
    scale = s.double() if fmt == ft.FMT_FP8 else torch.exp2(s.double() - 127)
    per = torch.cat([scale[:, :groups].repeat_interleave(size, 1)[:, :inter],
                     scale[:, groups:].repeat_interleave(size, 1)[:, :inter]], 1)
    return h, q, s, q.view(torch.float8_e4m3fn).double() * per


def backward_check(g, u, dh, w, dgu, hw, dwt, inter):
    w, dh = w.double()[:, None], dh.double()
    sig = 1 / (1 + torch.exp(-g))
    silu = g * sig
    dg, du = w * dh * u * sig * (1 + g * (1 - sig)), w * dh * silu
    # a sigmoid, 1 - s (absolute), three products and a sum: 16 units of fp32 of the terms' size
    check(dgu[:, :inter], dg, (w * dh * u).abs() * (sig + silu.abs()), 16, "dg")
    check(dgu[:, inter:], du, du.abs(), 16, "du")
    if hw is not None:
        check(hw, w * silu * u, (w * silu * u).abs(), 16, "hw")
    if dwt is not None:
        ref, mag = (dh * silu * u).sum(1), (dh * silu * u).abs().sum(1)
        check(dwt, ref, mag, inter + 16, "dweights")


@pytest.mark.parametrize("fmt", [ft.FMT_FP8, ft.FMT_MXFP8])
def test_silu_saved_codes_bit_for_bit(fmt):
    """MXFP8: codes and scales those of ftmoe_quantize_act on each half. FP8: the scale is the fp32
    product amax * (1/448), the codes those of the IEEE quotients by it."""
    rows, inter = 33, 416
    gu = normal((rows, 2 * inter), 3.0, torch.bfloat16, 33)
    gu[3] = 0.0
    gu[4, :64] = gu[4, :64] * 2.0 ** -60
    _, q, s, _ = save(gu, fmt, torch.bfloat16)
    groups = s.shape[1] // 2
    for half in (0, 1):
        part = gu[:, half * inter:(half + 1) * inter].contiguous()
        if fmt == ft.FMT_MXFP8:
            want_q, want_s, _ = ft.quantize_act(part, fmt)
        else:
            x = torch.nn.functional.pad(part.float(), (0, groups * 128 - inter)).view(rows, groups, 128).cpu().numpy()
            want = np.abs(x).max(2, keepdims=True) * (np.float32(1) / np.float32(448))
            codes = torch.from_numpy(np.where(want > 0, x / np.where(want > 0, want, np.float32(1)), np.float32(0)))
            want_q = codes.to(torch.float8_e4m3fn).view(torch.uint8).view(rows, -1)[:, :inter].to(DEV)
            want_s = torch.from_numpy(want[:, :, 0]).to(DEV)
        assert torch.equal(q[:, half * inter:(half + 1) * inter], want_q)
        assert torch.equal(s[:, half * groups:(half + 1) * groups], want_s)


@pytest.mark.parametrize("fmt", [ft.FMT_FP8, ft.FMT_MXFP8])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_silu_saved_infinities_nan_and_large_values(fmt, dtype):
    """h where g or u is infinite, NaN, or of any finite size: infinite, NaN and zero where the
    formula is; rows without such values are not touched by their neighbours'."""
    odd = [float("inf"), float("-inf"), float("nan"), 3e38, -3e38, 1e30, -1e30, 1000.0, -1000.0, 0.0, -0.0, 1.0, -80.0]
    pairs = [(g, u) for g in odd for u in (1.0, -2.0, 0.0, float("inf"), float("nan"))]
    inter = 32 * -(-len(pairs) // 32)
    row = torch.zeros(2 * inter, device=DEV)
    row[: len(pairs)] = torch.tensor([p[0] for p in pairs])
    row[inter: inter + len(pairs)] = torch.tensor([p[1] for p in pairs])
    gu = normal((3, 2 * inter), 1.0, torch.float32, 39)
    gu[1] = row
    gu = gu.to(DT[dtype])
    h, _, _, _ = save(gu, fmt, DT[dtype])
    g, u = gu[:, :inter].double(), gu[:, inter:].double()
    ref = (g / (1 + torch.exp(-g)) * u).to(DT[dtype]).double()
    assert torch.equal(torch.isnan(h), torch.isnan(ref))
    keep = ~torch.isnan(ref)
    assert torch.equal(h.double()[keep & torch.isinf(ref)], ref[keep & torch.isinf(ref)])
    fin = keep & torch.isfinite(ref)
    check(h[fin], (g / (1 + torch.exp(-g)) * u)[fin], ref.abs()[fin], 8, "h")


@pytest.mark.parametrize("fmt", [ft.FMT_FP8, ft.FMT_MXFP8])
def test_silu_gradient_agrees_with_differences(fmt):
    """dgu against central differences of sum(dh * w * h) in 64 bits at the kept values."""
    rows, inter = 5, 96
    gu = normal((rows, 2 * inter), 2.0, torch.float32, 34)
    _, q, s, kept = save(gu, fmt, torch.float32)
    dh, w = normal((rows, inter), 1.0, torch.float32, 35), torch.rand(rows, generator=gen(36), device=DEV)
    dgu = torch.empty(rows, 2 * inter, device=DEV)
    ft.ftmoe_silu_mul_backward(q, s, dh, dgu, row_weights=w, fmt=fmt)

    def loss(v):  # per element of the row: only its own h changes
        g, u = v[:, :inter], v[:, inter:]
        return w.double()[:, None] * dh.double() * g / (1 + torch.exp(-g)) * u
    step = 1e-5
    for half in (0, 1):
        d = torch.zeros_like(kept)
        d[:, half * inter:(half + 1) * inter] = step
        diff = (loss(kept + d) - loss(kept - d)) / (2 * step)
        # the difference's own error: step^2 times a third derivative below 1 of terms below 100
        assert ((dgu[:, half * inter:(half + 1) * inter].double() - diff).abs() <= 1e-5 * (1 + diff.abs())).all()


def test_silu_row_count_on_the_device_and_strides():
    """Rows past the device's count are not written; padded strides and bases."""
    rows, valid, inter = 20, 13, 136
    _, gu = strided((rows, 2 * inter), 8, 8, torch.bfloat16)
    gu[:valid] = normal((valid, 2 * inter), 2.0, torch.bfloat16, 37)
    count = torch.tensor([valid], dtype=torch.int32, device=DEV)
    hb, h = strided((rows, inter), 3, 1, torch.bfloat16)
    q = torch.full((rows, 2 * inter), 0xAA, dtype=torch.uint8, device=DEV)
    s = torch.full((rows, 4), -1.0, device=DEV)
    ft.ftmoe_silu_mul_save(gu, h, q, s, fmt=ft.FMT_FP8, rows_dev=count)
    _, q1, s1, kept = save(gu[:valid].contiguous(), ft.FMT_FP8, torch.bfloat16)
    assert torch.equal(q[:valid], q1) and torch.equal(s[:valid], s1)
    assert (q[valid:] == 0xAA).all() and (s[valid:] == -1).all()
    assert int((~torch.isnan(hb)).sum()) == valid * inter
    db, dgu = strided((rows, 2 * inter), 5, 3, torch.bfloat16)
    wb, hw = strided((rows, inter), 8, 8, torch.bfloat16)
    _, dh = strided((rows, inter), 16, 8, torch.bfloat16)
    dh[:valid] = normal((valid, inter), 0.3, torch.bfloat16, 38)
    dwt = torch.full((rows,), -7.0, device=DEV)
    ft.ftmoe_silu_mul_backward(q, s, dh, dgu, hw=hw, dweights=dwt, fmt=ft.FMT_FP8, rows_dev=count)
    backward_check(kept[:, :inter], kept[:, inter:], dh[:valid], torch.ones(valid, device=DEV), dgu[:valid], hw[:valid],
                   dwt[:valid], inter)
    assert int((~torch.isnan(db)).sum()) == valid * 2 * inter and int((~torch.isnan(wb)).sum()) == valid * inter
    assert (dwt[valid:] == -7).all()


def test_no_rows_and_other_streams():
    """Zero rows launch nothing (the weight gradient writes zeros); work goes on the given stream."""
    w = normal((3, 64, 64), 0.1, torch.bfloat16, 40)
    empty = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV)
    ft.ftmoe_grouped_matmul(empty, offsets_of([0, 0, 0]), w, empty.clone())
    dw = torch.full_like(w, float("nan"))
    ft.ftmoe_grouped_matmul_wgrad(empty, empty, offsets_of([0, 0, 0]), dw)
    assert (dw == 0).all()
    side = torch.cuda.Stream()
    a = torch.zeros(200, 64, dtype=torch.bfloat16, device=DEV)
    out = torch.empty(200, 64, dtype=torch.float32, device=DEV)
    off = offsets_of([100, 0, 100])
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        a.fill_(1.0)
        ft.ftmoe_grouped_matmul(a, off, w, out)       # the current stream is `side`
    side.synchronize()
    ref, mag = product_ref(a, w, [100, 0, 100], False)
    check(out, ref, mag, 64, "on another stream")


def test_results_do_not_depend_on_the_call():
    """The same inputs give the same bits, call after call, and a row's result does not depend on
    how many rows the other experts have."""
    counts, n, k = [90, 300, 1, 260], 520, 1032
    R = sum(counts)
    a, w = normal((R, k), 1.0, torch.bfloat16, 41), normal((4, n, k), 0.1, torch.bfloat16, 42)
    c = normal((R, n), 1.0, torch.bfloat16, 43)
    off = offsets_of(counts)
    outs = []
    for _ in range(3):
        y = torch.empty(R, n, dtype=torch.float32, device=DEV)
        dw = torch.empty(4, n, k, dtype=torch.float32, device=DEV)
        ft.ftmoe_grouped_matmul(a, off, w, y)
        ft.ftmoe_grouped_matmul_wgrad(c, a, off, dw)
        outs.append((y, dw))
    for y, dw in outs[1:]:
        assert torch.equal(y, outs[0][0]) and torch.equal(dw, outs[0][1])


def test_graph_replay_with_other_row_counts():
    """Launch shapes depend on sizes only: one captured graph serves other offsets and inputs."""
    E, n, k, R = 6, 264, 320, 500
    a, w = normal((R, k), 1.0, torch.bfloat16, 44), normal((E, n, k), 0.1, torch.bfloat16, 45)
    c = normal((R, n), 1.0, torch.bfloat16, 46)
    off = offsets_of([100, 100, 100, 100, 50, 50])
    y = torch.empty(R, n, dtype=torch.bfloat16, device=DEV)
    da = torch.empty(R, k, dtype=torch.float32, device=DEV)
    dw = torch.empty(E, n, k, dtype=torch.float32, device=DEV)

    def step():
        ft.ftmoe_grouped_matmul(a, off, w, y)
        ft.ftmoe_grouped_matmul(c, off, w, da, input_grad=True)
        ft.ftmoe_grouped_matmul_wgrad(c, a, off, dw)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for counts in ([500, 0, 0, 0, 0, 0], [0, 1, 2, 0, 400, 97], [83, 83, 83, 83, 84, 84]):
        off.copy_(offsets_of(counts))
        graph.replay()
        torch.cuda.synchronize()
        ref, mag = product_ref(a, w, counts, False)
        check(y, ref, mag, k, "product")
        ref, mag = product_ref(c, w, counts, True)
        check(da, ref, mag, n, "input gradient")
        ref, mag = wgrad_ref(c, a, counts)
        check(dw, ref, mag, R, "weight gradient")
    assert ft.ftmoe_read_error_flags() == 0
