"""The gradients' global norm and the AdamW step against the definitions in 64 bits, and the moments'
codes bit for bit."""
import math

import numpy as np
import pytest
import torch

import block_quantized_moe_gb300 as ft

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
HYPER = dict(lr=1e-2, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.1)
EPS32 = 2.0 ** -24


def randn(n, seed, std=1.0, dtype="fp32"):
    return (torch.randn(n, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV) * std).to(DTYPES[dtype])


# ---------------------------------------------------------------------------------
# norm
# ---------------------------------------------------------------------------------

def norm_of(grads, **kw):
    made = ft.make_grad_list(grads)
    ws = torch.full((ft.ftmoe_grad_norm_workspace_bytes(made),), 255, dtype=torch.uint8, device=DEV)
    result = torch.full((2,), -1.0, device=DEV)
    ft.ftmoe_grad_norm(made, result, ws, **kw)
    return result.tolist()


def check_norm(grads, scale=1.0, max_norm=math.inf):
    want = scale * math.sqrt(sum(float(g.double().square().sum()) for g in grads))
    factor = scale * min(1.0, max_norm / (want + 1e-6))
    got = norm_of(grads, scale=scale, max_norm=max_norm)
    # a chain of 8 positive terms in fp32 (the sums of those carry their errors along), half of which the root keeps,
    # and its rounding
    assert abs(got[0] - want) <= 8 * EPS32 * want + 2.0 ** -150, (got, want)
    assert abs(got[1] - factor) <= 9 * EPS32 * factor, (got, factor)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("sizes", [(1,), (7,), (8,), (8191, 8192, 8193), (0, 5, 0, 33), (1_000_003, 1, 70_001), (20_000_000,)])
def test_norm(sizes, dtype):
    grads = [randn(n, n + i, 0.01, dtype) for i, n in enumerate(sizes)]
    check_norm(grads)
    check_norm(grads, scale=2.0 ** -10, max_norm=1e-4)
    check_norm(grads, scale=3.0, max_norm=1e6)


@pytest.mark.parametrize("count", [65, 1024, 1025, 2500])
def test_norm_of_many(count):
    check_norm([randn(i % 97, i, 0.1, "bf16") for i in range(count)])


def test_norm_of_unaligned_and_shaped():
    g = randn(100_000, 1)
    check_norm([g[1:5000], g[5002:70_003], g[70_003:99_999].view(-1, 4)])
    h = g.half()
    check_norm([h[1:5000], h[5001:]])


def test_norm_of_nothing():
    assert norm_of([], scale=2.0) == [0.0, 2.0]
    assert norm_of([torch.empty(0, device=DEV)]) == [0.0, 1.0]
    assert norm_of([torch.zeros(10_000, device=DEV)]) == [0.0, 1.0]


@pytest.mark.parametrize("value", [1e-44, 1e-30, 1e-16, 1e-15, 3e14, 1e16, 1e19, 1e30, 3e38])
def test_norm_beyond_the_range_of_fp32_squares(value):
    g = torch.full((37,), value, device=DEV)
    check_norm([g], scale=0.125)
    g = randn(5000, 3, 1.0)
    g[::100] = value
    check_norm([g, torch.zeros(9, device=DEV)], scale=0.125)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
def test_norm_that_is_not_finite(value, dtype):
    g = randn(9000, 4, 1.0, dtype)
    g[8999] = value
    norm, factor = norm_of([randn(5, 5, 1.0, dtype), g], max_norm=1.0)
    assert (math.isnan(norm) if math.isnan(value) else norm == math.inf) and math.isnan(factor)
    # a norm beyond fp32: no factor either
    if dtype != "fp16":
        norm, factor = norm_of([torch.full((100,), 3e38, dtype=DTYPES[dtype], device=DEV)])
        assert norm == math.inf and math.isnan(factor)


def test_norm_has_the_same_bits_every_time():
    grads = [randn(3_000_001, 1), randn(77, 2)]
    assert len({tuple(norm_of(grads, max_norm=1.0)) for _ in range(5)}) == 1


# ---------------------------------------------------------------------------------
# AdamW
# ---------------------------------------------------------------------------------

MASK = np.uint64(0xFFFFFFFF)
SPREAD = [0x3C6EF373, 0xA54FF53B, 0x510E527F, 0x9B05688D, 0x1F83D9AB, 0x5BE0CD19, 0xCBBB9D5D, 0x629A292B]


def mix(x):
    x = np.asarray(x, dtype=np.uint64) & MASK
    x ^= x >> np.uint64(16)
    x = x * np.uint64(0x6A09E667) & MASK
    x ^= x >> np.uint64(15)
    x = x * np.uint64(0xBB67AE85) & MASK
    return x ^ (x >> np.uint64(16))


def noise(n, seed, step, tensor, first=0):
    """32 random bits of the elements [first, first + n) (first a multiple of 8)."""
    key = mix(mix(mix(seed) + np.uint64(step & 0xFFFFFFFF)) + np.uint64(tensor))
    chunk = np.arange(first // 8, (first + n + 7) // 8, dtype=np.uint64)
    base = mix(mix(key + (chunk >> np.uint64(32))) + (chunk & MASK))
    h = base[:, None] * np.array(SPREAD, dtype=np.uint64)
    return ((h ^ (h >> np.uint64(32))) & MASK).reshape(-1)[:n]


def codes_of(x, bits16, top, least, digits):
    """(codes, bytes) of magnitudes x (fp32 values as float64): steps of 2^(e - digits) with e >= least, taken up
    where the part cut off and 16 random bits pass one."""
    n, groups = x.size, -(-x.size // 32)
    padded = np.zeros(groups * 32)
    padded[:n] = x
    amax = padded.reshape(groups, 32).max(1)
    with np.errstate(divide="ignore"):
        e = np.where(amax >= 2.0 ** -126, np.floor(np.log2(np.maximum(amax, 2.0 ** -126))), -127)
    power = np.maximum(e + (amax > 1.75 * 2.0 ** e) - top, -127)
    y = x * np.repeat(2.0 ** -power, 32)[:n]
    # in fp32 the steps below the least normal end 149 - 126 = 23 bits below it
    fine = 2.0 ** (least - 23)
    y = np.where(y < 2.0 ** least, np.rint(y / fine) * fine, y)
    exponent = np.maximum(np.floor(np.log2(np.maximum(y, 1e-300))), least)
    step = 2.0 ** (exponent - digits)
    q = np.floor(y / step + bits16 / 65536.0) * step
    # a code: digits below the leading one, subnormal ones with exponent 0
    exponent = np.floor(np.log2(np.maximum(q, 1e-300)))
    normal = exponent >= least
    code = np.where(normal, (exponent - least + 1) * 2 ** digits + q / 2.0 ** (exponent - digits) - 2 ** digits,
                    q / 2.0 ** (least - digits))
    return np.minimum(code, 127).astype(np.uint8), (power + 127).astype(np.uint8)


def new_moments(m, v, g, scale):
    """The products and sums of m and v, each rounded to fp32."""
    f = np.float32
    g = g * f(scale)
    m = m * f(HYPER["beta1"]) + g * f(1 - HYPER["beta1"])
    v = v * f(HYPER["beta2"]) + (g * g) * f(1 - HYPER["beta2"])
    return m, v


def new_params(p, m, v, step, lr=HYPER["lr"]):
    m, v, p = m.astype(np.float64), v.astype(np.float64), p.astype(np.float64)
    u = lr / (1 - HYPER["beta1"] ** step) * m / (np.sqrt(v / (1 - HYPER["beta2"] ** step)) + HYPER["eps"])
    return p - lr * HYPER["weight_decay"] * p - u, np.abs(u)


def check_params(got, p, m, v, step, dtype, lr=HYPER["lr"]):
    want, u = new_params(p, m, v, step, lr)
    # the update from fp32 operations (a root, a quotient, the corrections, products: 32 half steps), the sum's rounding, the
    # type's own
    limit = (u + np.abs(lr * HYPER["weight_decay"] * p)) * 32 * EPS32 + np.abs(want) * (2 * EPS32 + (torch.finfo(DTYPES[dtype]).eps / 2 if dtype != "fp32" else 0))
    limit = limit + (2.0 ** -25 if dtype == "fp16" else 1e-44)
    bad = np.abs(got.double().cpu().numpy() - want) > limit
    assert not bad.any(), (np.nonzero(bad)[0][:5], np.abs(got.double().cpu().numpy() - want)[bad][:5], limit[bad][:5])


def state(sizes, gdtype="fp32", pdtype="fp32", narrow=False, copy=None, seed=0, gstd=0.1):
    s = {"params": [randn(n, seed + 10 * i, 0.5, pdtype) for i, n in enumerate(sizes)],
         "grads": [randn(n, seed + 10 * i + 1, gstd, gdtype) for i, n in enumerate(sizes)],
         "m": [randn(n, seed + 10 * i + 2, 0.05) for i, n in enumerate(sizes)],
         "v": [randn(n, seed + 10 * i + 3, 0.1).square() for i, n in enumerate(sizes)]}
    if narrow:
        for kind, top, least, digits in (("m", 8, -6, 3), ("v", 15, -14, 2)):
            made = []
            for t in s[kind]:
                x = t.cpu().numpy()
                c, b = codes_of(np.abs(x).astype(np.float64), np.full(x.size, 32768.0), top, least, digits)
                made.append((torch.from_numpy(c | ((x < 0).astype(np.uint8) << 7)).to(DEV), torch.from_numpy(b).to(DEV)))
            s[kind], s[kind + "_scales"] = [c for c, _ in made], [b for _, b in made]
    if copy:
        s["copies"] = [torch.zeros(n, dtype=DTYPES[copy], device=DEV) for n in sizes]
    return s


def values(codes, scales, dtype):
    """fp32 values of kept moments."""
    x = codes.view(dtype).float().cpu().numpy()
    return x * np.repeat(np.ldexp(np.float32(1), scales.cpu().numpy().astype(np.int32) - 127), 32)[:x.size]


def moments_of(s, i):
    if "m_scales" in s:
        return values(s["m"][i], s["m_scales"][i], torch.float8_e4m3fn), values(s["v"][i], s["v_scales"][i], torch.float8_e5m2)
    return s["m"][i].cpu().numpy(), s["v"][i].cpu().numpy()


def clone(s):
    return {k: [t.clone() for t in v] for k, v in s.items()}


def step_on(s, step=3, seed=5, **kw):
    ft.ftmoe_adamw_step(ft.make_adamw_list(**s), step=step, seed=seed, **{**HYPER, **kw})


def check_step(s, step=3, seed=5, scale=None, pdtype="fp32", copy=None):
    before = clone(s)
    step_on(s, step, seed, grad_scale=None if scale is None else torch.tensor([scale], device=DEV))
    for i in range(len(s["params"])):
        m, v = moments_of(before, i)
        m, v = new_moments(m, v, before["grads"][i].float().cpu().numpy(), 1.0 if scale is None else scale)
        assert torch.equal(s["grads"][i], before["grads"][i])
        check_params(s["params"][i], before["params"][i].double().cpu().numpy(), m, v, step, pdtype)
        if copy:
            assert torch.equal(s["copies"][i], s["params"][i].to(DTYPES[copy]))
        if "m_scales" not in s:
            np.testing.assert_array_equal(s["m"][i].cpu().numpy(), m)
            np.testing.assert_array_equal(s["v"][i].cpu().numpy(), v)
            continue
        h = noise(m.size, seed, step, i)
        c, b = codes_of(np.abs(m).astype(np.float64), (h & np.uint64(0xFFFF)).astype(np.float64), 8, -6, 3)
        np.testing.assert_array_equal(s["m_scales"][i].cpu().numpy(), b)
        np.testing.assert_array_equal(s["m"][i].cpu().numpy(), c | (np.signbit(m).astype(np.uint8) << 7))
        c, b = codes_of(v.astype(np.float64), (h >> np.uint64(16)).astype(np.float64), 15, -14, 2)
        np.testing.assert_array_equal(s["v_scales"][i].cpu().numpy(), b)
        np.testing.assert_array_equal(s["v"][i].cpu().numpy(), np.where(v > 0, np.maximum(c, 1), c))


SIZES = [(1,), (7, 8, 9), (31, 32, 33), (0, 255, 0), (8191, 8192, 8193, 1), (100_003, 64)]


@pytest.mark.parametrize("gdtype", DTYPES)
@pytest.mark.parametrize("sizes", SIZES, ids=str)
def test_step_with_fp32_moments(sizes, gdtype):
    check_step(state(sizes, gdtype))
    check_step(state(sizes, gdtype, copy="bf16"), step=1, scale=0.25, copy="bf16")


@pytest.mark.parametrize("gdtype", DTYPES)
@pytest.mark.parametrize("sizes", SIZES, ids=str)
def test_step_with_8_bit_moments(sizes, gdtype):
    check_step(state(sizes, gdtype, narrow=True))
    check_step(state(sizes, gdtype, narrow=True, copy="fp16"), step=1 << 33, seed=0xFFFFFFFF, scale=0.25, copy="fp16")


@pytest.mark.parametrize("narrow", [False, True])
@pytest.mark.parametrize("pdtype", ["bf16", "fp16"])
def test_16_bit_parameters(pdtype, narrow):
    check_step(state((1000, 33), "bf16", pdtype, narrow), pdtype=pdtype)
    check_step(state((1000, 33), "fp32", pdtype, narrow), pdtype=pdtype)


@pytest.mark.parametrize("narrow", [False, True])
@pytest.mark.parametrize("count", [48, 49, 400, 401, 900])
def test_many_tensors(count, narrow):
    check_step(state([1 + i % 40 for i in range(count)], "bf16", narrow=narrow))


@pytest.mark.parametrize("narrow", [False, True])
def test_wide_ranges(narrow):
    """Moments and gradients of very different sizes in one group; zeros; fp32's largest and smallest."""
    s = state((4096,), "fp32", narrow=False)
    exponent = torch.randint(-60, 15, (4096,), generator=torch.Generator(device=DEV).manual_seed(7), device=DEV).float()
    s["grads"][0] *= torch.exp2(exponent)
    s["m"][0] *= torch.exp2(exponent)
    s["v"][0] *= torch.exp2(2 * exponent).clamp(max=2.0 ** 60)
    s["grads"][0][:64], s["m"][0][:64], s["v"][0][:64] = 0.0, 0.0, 0.0
    s["grads"][0][64:96] = 1e-41
    s["m"][0][64:96], s["v"][0][64:96] = 1e-42, 1e-44
    s["grads"][0][96:128], s["m"][0][96:128], s["v"][0][96:128] = 1e18, 1e37, 1e37
    if narrow:
        for kind, top, least, digits in (("m", 8, -6, 3), ("v", 15, -14, 2)):
            x = s[kind][0].cpu().numpy()
            c, b = codes_of(np.abs(x).astype(np.float64), np.full(x.size, 32768.0), top, least, digits)
            s[kind] = [torch.from_numpy(c | ((x < 0).astype(np.uint8) << 7)).to(DEV)]
            s[kind + "_scales"] = [torch.from_numpy(b).to(DEV)]
    check_step(s)


def test_a_second_moment_above_zero_stays_above_zero():
    """A group with one large gradient and many tiny ones: every v keeps a code, so that no update is
    a moment over eps."""
    s = state((64,), "fp32", narrow=True, gstd=1e-6)
    s["v"][0].zero_(), s["m"][0].zero_()
    s["grads"][0][5] = 1e6
    for t in range(1, 4):
        step_on(s, step=t)
        assert (s["v"][0] > 0).all()
        assert (s["params"][0].abs() < 4).all()


def test_rounding_is_right_on_average():
    """The mean of a moment over 512 seeds: off by at most 5 of its standard deviations, a step's share
    of at most a half over sqrt(512) (and 2^-17 of a step for the 16 random bits)."""
    n, seeds = 4096, 512
    base = state((n,), "fp32", narrow=True)
    m, v = moments_of(base, 0)
    m, v = new_moments(m, v, base["grads"][0].cpu().numpy(), 1.0)
    sums = [np.zeros(n), np.zeros(n)]
    squares = [np.zeros(n), np.zeros(n)]
    for seed in range(seeds):
        s = clone(base)
        step_on(s, seed=seed)
        for k, x in enumerate(moments_of(s, 0)):
            sums[k] += x
            squares[k] += x.astype(np.float64) ** 2
    for k, (x, dtype) in enumerate(((m, torch.float8_e4m3fn), (v, torch.float8_e5m2))):
        scale = np.repeat(2.0 ** (s[("m_scales", "v_scales")[k]][0].cpu().numpy().astype(np.float64) - 127), 32)
        digits, least = ((3, -6), (2, -14))[k]
        step = scale * 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(np.abs(x) / scale, 1e-300))), least) - digits)
        assert (np.abs(sums[k] / seeds - x) <= step * (0.5 * 5 / math.sqrt(seeds) + 2.0 ** -17)).all()
        # and over all elements together: sqrt(n) times closer
        assert abs(((sums[k] / seeds - x) / step).mean()) <= 0.5 * 5 / math.sqrt(seeds * n) + 2.0 ** -17


@pytest.mark.parametrize("narrow", [False, True])
@pytest.mark.parametrize("scale", [math.nan, math.inf, -math.inf])
def test_no_step_for_a_scale_that_is_not_finite(scale, narrow):
    s = state((5000, 3), narrow=narrow, copy="bf16")
    before = clone(s)
    step_on(s, grad_scale=torch.tensor([scale], device=DEV))
    assert all(torch.equal(a, b) for k in s for a, b in zip(s[k], before[k]))


def test_gradients_that_are_not_finite():
    """fp32 moments follow the formula; 8-bit ones are kept as NaN and infinity, and the group's other
    elements stay finite."""
    for narrow in (False, True):
        s = state((64,), narrow=narrow)
        s["grads"][0][3], s["grads"][0][40] = math.nan, math.inf
        step_on(s)
        m, v = moments_of(s, 0)
        assert np.isnan(m[3]) and not np.isfinite(m[40]) and not np.isfinite(v[3]) and np.isinf(v[40])
        rest = np.delete(np.arange(64), [3, 40])
        assert np.isfinite(m[rest]).all() and np.isfinite(v[rest]).all() and torch.isfinite(s["params"][0][torch.from_numpy(rest).to(DEV)]).all()


@pytest.mark.parametrize("narrow", [False, True])
def test_any_alignment_gives_the_same_bits_and_writes_nothing_else(narrow):
    n = 5003
    s = state((n,), "bf16", narrow=narrow, copy="bf16")
    want = clone(s)
    step_on(want)
    for off in (1, 3):
        homes = {k: torch.full((v[0].numel() + 16,), 77, dtype=v[0].dtype, device=DEV) for k, v in s.items()}
        t = {}
        for k, v in s.items():
            t[k] = [homes[k][off:off + v[0].numel()]]
            t[k][0].copy_(v[0])
        step_on(t)
        for k in s:
            assert torch.equal(t[k][0], want[k][0]), k
            assert (homes[k][:off].float() == 77).all() and (homes[k][off + s[k][0].numel():].float() == 77).all(), k


@pytest.mark.parametrize("narrow", [False, True])
def test_constants_on_the_device_and_replayed_graphs(narrow):
    """A graph captured once, replayed as step, learning rate and gradient scale change."""
    s = state((3000, 77), "bf16", narrow=narrow, copy="bf16")
    grads = s["grads"]
    lr, step = torch.zeros(1, device=DEV), torch.zeros(1, dtype=torch.int64, device=DEV)
    made, norms = ft.make_adamw_list(**s), ft.make_grad_list(grads)
    ws = torch.empty(ft.ftmoe_grad_norm_workspace_bytes(norms), dtype=torch.uint8, device=DEV)
    result = torch.zeros(2, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ft.ftmoe_grad_norm(norms, result, ws, max_norm=1.0)
        ft.ftmoe_adamw_step(made, seed=9, lr_dev=lr, step_dev=step, grad_scale=result[1:], **{**HYPER, "lr": 123.0})
    for t in range(1, 5):
        before = clone(s)
        lr.fill_(0.01 / t)
        step.fill_(t)
        for i, g in enumerate(grads):
            g.copy_(randn(g.numel(), 50 + 2 * t + i, 0.1, "bf16"))
        graph.replay()
        before["grads"] = grads
        scale = float(result[1])
        for i in range(2):
            m, v = moments_of(before, i)
            m, v = new_moments(m, v, grads[i].float().cpu().numpy(), scale)
            check_params(s["params"][i], before["params"][i].double().cpu().numpy(), m, v, t, "fp32", lr=float(lr))
            if not narrow:
                np.testing.assert_array_equal(s["m"][i].cpu().numpy(), m)
            else:
                c, _ = codes_of(np.abs(m).astype(np.float64), (noise(m.size, 9, t, i) & np.uint64(0xFFFF)).astype(np.float64), 8, -6, 3)
                np.testing.assert_array_equal(s["m"][i].cpu().numpy() & 127, c)


def test_more_than_32_bits_of_elements():
    """2^32 + 1000 elements: the ends and the places around 2^31 and 2^32 against the formulas, codes bit for bit, and the
    norm of as many gradients."""
    n = (1 << 32) + 1000
    gen = torch.Generator(device=DEV).manual_seed(3)
    g = torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    p = torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    m, v = (torch.zeros(n, dtype=torch.uint8, device=DEV) for _ in range(2))
    ms, vs = (torch.full((-(-n // 32),), b, dtype=torch.uint8, device=DEV) for b in (118, 105))
    places = [(a, min(a + 2048, n)) for a in (0, (1 << 31) - 1024, (1 << 32) - 1024)]
    for a, b in places:
        g[a:b] = (torch.randn(b - a, generator=gen, device=DEV) * 0.1).to(torch.bfloat16)
        p[a:b] = torch.randn(b - a, generator=gen, device=DEV).to(torch.bfloat16)
        m[a:b] = torch.randint(0, 255, (b - a,), generator=gen, device=DEV).clamp(max=126).to(torch.uint8)
        v[a:b] = torch.randint(1, 124, (b - a,), generator=gen, device=DEV).to(torch.uint8)
    check_norm([g])
    cut = {k: [t[a:b].clone() for a, b in places] for k, t in (("p", p), ("m", m), ("v", v))}
    scales = {k: [t[a // 32:-(-b // 32)].clone() for a, b in places] for k, t in (("m", ms), ("v", vs))}
    step_on({"params": [p], "grads": [g], "m": [m], "v": [v], "m_scales": [ms], "v_scales": [vs]}, step=7, seed=11)
    for i, (a, b) in enumerate(places):
        mm, vv = values(cut["m"][i], scales["m"][i], torch.float8_e4m3fn), values(cut["v"][i], scales["v"][i], torch.float8_e5m2)
        mm, vv = new_moments(mm, vv, g[a:b].float().cpu().numpy(), 1.0)
        check_params(p[a:b], cut["p"][i].double().cpu().numpy(), mm, vv, 7, "bf16")
        h = noise(b - a, 11, 7, 0, first=a)
        c, bytes_ = codes_of(np.abs(mm).astype(np.float64), (h & np.uint64(0xFFFF)).astype(np.float64), 8, -6, 3)
        np.testing.assert_array_equal(m[a:b].cpu().numpy(), c | (np.signbit(mm).astype(np.uint8) << 7))
        np.testing.assert_array_equal(ms[a // 32:-(-b // 32)].cpu().numpy(), bytes_)
        c, _ = codes_of(vv.astype(np.float64), (h >> np.uint64(16)).astype(np.float64), 15, -14, 2)
        np.testing.assert_array_equal(v[a:b].cpu().numpy(), np.where(vv > 0, np.maximum(c, 1), c))


def test_another_stream():
    s = state((100_000,), narrow=True)
    want = clone(s)
    step_on(want)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    ft.ftmoe_adamw_step(ft.make_adamw_list(**s), step=3, seed=5, stream=stream, **HYPER)
    stream.synchronize()
    assert all(torch.equal(a, b) for k in s for a, b in zip(s[k], want[k]))


def test_betas_of_zero_and_steps_of_a_device_below_one():
    s = state((100,))
    want = clone(s)
    ft.ftmoe_adamw_step(ft.make_adamw_list(**s), step=1, lr=0.1, beta1=0.0, beta2=0.0, weight_decay=0.0)
    g = want["grads"][0].double()
    assert torch.equal(s["m"][0], want["grads"][0])
    # |update| = lr |g| / (|g| + eps)
    assert float(((want["params"][0] - s["params"][0]).double() - 0.1 * g / (g.abs() + 1e-8)).abs().max()) <= 1e-6
    for t in (0, -5, 1):
        again = clone(want)
        ft.ftmoe_adamw_step(ft.make_adamw_list(**again), step_dev=torch.tensor([t], device=DEV), lr=0.1, beta1=0.0, beta2=0.0,
                            weight_decay=0.0)
        assert torch.allclose(again["params"][0], s["params"][0], atol=1e-6)


def test_no_tensors():
    ft.ftmoe_adamw_step(ft.make_adamw_list([], [], [], []))


@pytest.mark.parametrize("narrow", [False, True])
@pytest.mark.parametrize("gdtype", ["bf16", "fp32"])
@pytest.mark.parametrize("pdtype,copy", [("bf16", "fp16"), ("fp16", "bf16"), ("bf16", "bf16"), ("fp16", "fp16")])
def test_copies_of_16_bit_parameters(pdtype, copy, gdtype, narrow):
    """The copy is the new parameter as it is kept, in the copy's type."""
    check_step(state((20_000, 33, 7), gdtype, pdtype, narrow, copy), pdtype=pdtype, copy=copy)
