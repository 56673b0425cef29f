"""The training and 16-bit operators of the routed experts, as measured workloads.

What is measured: matrix products grouped by expert over ragged row counts (the product with
the weights, the gradient of its input, the gradient of the weights), and activations kept in
8 bits between the forward and the backward pass (SiLU-and-mul that saves its gate/up rows and
its backward pass from them; the weight gradient from saved rows).

Rows are sorted by expert; the rows of expert e are [offsets[e], offsets[e + 1]). Sizes are the
repository's benchmark geometries: 2048/768 with 8 experts, 4096/1024 with 64 experts, 7168/2048
with 256 experts at 24,576 routes, and a 32-expert bank with the same routes (a training shard).

`run` computes the plain form in 32-bit torch operations, or, where `own` is set, makes the
calls of the library. `exact` gives the same outputs from the definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------

def _product(name, kind, rows, experts, n, k, skew, dtype, out, fmt="none"):
    return {"name": name, "kind": kind, "rows": rows, "experts": experts, "n": n, "k": k, "skew": skew,
            "dtype": dtype, "out": out, "fmt": fmt}


def listed():
    return [
        # one decoded token, two of its eight experts on this GPU: the gate/up product, latency
        _product("matmul decode 1 token", "matmul", 2, 8, 1536, 2048, 0.0, "bf16", "bf16"),
        # eight decoded tokens, top-8 of 64 experts: about one row per expert that is hit
        _product("matmul decode 8 tokens", "matmul", 64, 64, 2048, 4096, 1.0, "fp16", "fp16"),
        # a prompt of 4,096 tokens, top-6 of 256 experts: 96 rows per expert, weight traffic
        _product("matmul prompt 256 experts", "matmul", 24576, 256, 4096, 7168, 0.25, "bf16", "bf16"),
        # a training shard of 32 experts with uneven load: about 768 rows per expert, tensor work
        _product("matmul train 32 experts", "matmul", 24576, 32, 4096, 7168, 0.6, "bf16", "bf16"),
        # gradient of the down product's input for an odd number of routes
        _product("input grad 1111 rows", "dgrad", 1111, 64, 4096, 1024, 0.5, "fp16", "fp16"),
        # gradient of the gate/up product's input, fp32 rows for the sum over a token's experts
        _product("input grad train", "dgrad", 24576, 32, 4096, 7168, 0.6, "bf16", "fp32"),
        # weight gradient of a small bank, fp32 as an optimizer's accumulator holds it
        _product("weight grad 333 rows", "wgrad", 333, 8, 1536, 2048, 0.5, "bf16", "fp32"),
        # weight gradient of the training shard
        _product("weight grad train", "wgrad", 24576, 32, 4096, 7168, 0.6, "bf16", "bf16"),
        # weight gradient from input rows saved in 8 bits (a power-of-two scale per 32)
        _product("saved weight grad 8191 rows", "wgrad8", 8191, 64, 2048, 4096, 0.5, "bf16", "fp32", "mxfp8"),
        # the training shard's weight gradient from rows saved in 8 bits
        _product("saved weight grad train", "wgrad8", 24576, 32, 4096, 7168, 0.6, "bf16", "bf16", "mxfp8"),
        # SiLU-and-mul that saves gate/up in 8 bits, and its backward pass: a small step
        {"name": "silu saved 64 rows", "kind": "silu", "rows": 64, "inter": 1024, "dtype": "bf16", "fmt": "mxfp8"},
        # the same for a training step's 24,576 routes
        {"name": "silu saved 24576 rows", "kind": "silu", "rows": 24576, "inter": 2048, "dtype": "bf16", "fmt": "fp8"},
    ]


def _log_int(rng, lo, hi, step=1):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return min(hi, max(lo, (v + step // 2) // step * step))


def draw(rng):
    kind = rng.choice(["matmul", "matmul", "dgrad", "wgrad", "wgrad8", "silu"])
    rows = _log_int(rng, 1, 24576)
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    if kind == "silu":
        fmt = rng.choice(["fp8", "mxfp8"])
        return {"kind": kind, "rows": rows, "inter": _log_int(rng, 128, 2048, 32 if fmt == "mxfp8" else 8),
                "dtype": dtype, "fmt": fmt}
    fmt = "mxfp8" if kind == "wgrad8" else "none"
    experts = _log_int(rng, 4, 256 if kind in ("matmul", "dgrad") else 64)
    n = _log_int(rng, 256, 4096, 8)
    k = _log_int(rng, 512, 7168, 32)
    if kind in ("wgrad", "wgrad8"):  # no more gradient values than the listed shard's
        while experts * n * k > 32 * 4096 * 7168:
            experts = max(4, experts // 2)
    out = rng.choice([dtype, dtype, "fp32"])
    return {"kind": kind, "rows": rows, "experts": experts, "n": n, "k": k, "skew": round(rng.uniform(0.0, 0.6), 2),
            "dtype": dtype, "out": out, "fmt": fmt}


def _counts(case):
    """Rows per expert in descending order: shares of a log-normal load of the case's skew,
    rounded to whole rows by largest remainder."""
    rows, experts = case["rows"], case["experts"]
    # quantiles of the normal distribution by the logistic approximation, enough for a load profile
    q = (np.arange(experts) + 0.5) / experts
    share = np.exp(-case["skew"] * np.log(q / (1 - q)) / 1.702)
    share = share / share.sum() * rows
    counts = np.floor(share).astype(np.int64)
    order = np.argsort(-(share - counts), kind="stable")
    counts[order[: rows - int(counts.sum())]] += 1
    return counts


def work(case):
    rows = case["rows"]
    if case["kind"] == "silu":
        inter = case["inter"]
        scales = 4 * -(-inter // 128) if case["fmt"] == "fp8" else inter // 32
        # gate/up and dh read; h, dgate/up and the weighted h written; the 8-bit rows and their
        # scales written by the forward and read by the backward pass; a weight in, its gradient out
        per_row = 4 * inter + 2 * inter + 2 * inter + 4 * inter + 2 * inter + 2 * (2 * inter + 2 * scales) + 8
        return {"bytes": rows * per_row, "flops": rows * inter * 30}
    n, k, experts = case["n"], case["k"], case["experts"]
    out_bytes = 4 if case["out"] == "fp32" else 2
    flops = 2 * rows * n * k
    if case["kind"] in ("matmul", "dgrad"):
        hit = int((_counts(case) > 0).sum())
        width_in, width_out = (k, n) if case["kind"] == "matmul" else (n, k)
        moved = hit * n * k * 2 + rows * width_in * 2 + rows * width_out * out_bytes
    else:
        x_row = 2 * k if case["kind"] == "wgrad" else k + k // 32
        moved = rows * n * 2 + rows * x_row + experts * n * k * out_bytes
    return {"bytes": moved + 4 * (experts + 1), "flops": flops}


# ---------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------

def _normal(shape, std, dtype, gen):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=gen)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    rows = case["rows"]
    if case["kind"] == "silu":
        inter, fmt = case["inter"], case["fmt"]
        groups = -(-inter // 128) if fmt == "fp8" else inter // 32
        s = {"gu": _normal((rows, 2 * inter), 1.4, dt, gen), "dh": _normal((rows, inter), 0.05, dt, gen),
             "weights": torch.rand(rows, generator=gen, device="cuda"),
             "h": torch.empty(rows, inter, dtype=dt, device="cuda"),
             "q": torch.empty(rows, 2 * inter, dtype=torch.uint8, device="cuda"),
             "scales": torch.empty(rows, 2 * groups, device="cuda", dtype=torch.float32 if fmt == "fp8" else torch.uint8),
             "dgu": torch.empty(rows, 2 * inter, dtype=dt, device="cuda"),
             "hw": torch.empty(rows, inter, dtype=dt, device="cuda"),
             "dweights": torch.empty(rows, device="cuda")}
        return {"case": case, **s}
    n, k, experts = case["n"], case["k"], case["experts"]
    counts = _counts(case)
    counts = counts[np.random.RandomState(seed % (1 << 32)).permutation(experts)]
    offsets = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).cuda()
    s = {"case": case, "offsets": offsets, "most": int(counts.max())}
    odt = DTYPES[case["out"]]
    if case["kind"] in ("matmul", "dgrad"):
        wide_in, wide_out = (k, n) if case["kind"] == "matmul" else (n, k)
        s["a"] = _normal((rows, wide_in), 1.0 if case["kind"] == "matmul" else 0.05, dt, gen)
        s["w"] = _normal((experts, n, k), 0.02, dt, gen)
        s["out"] = torch.empty(rows, wide_out, dtype=odt, device="cuda")
        return s
    s["dy"] = _normal((rows, n), 0.05, dt, gen)
    x = _normal((rows, k), 1.0, dt, gen)
    if case["kind"] == "wgrad":
        s["x"] = x
    else:
        q, scales, _ = _save(x.float(), case["fmt"])
        s["q"] = q.view(torch.uint8)
        s["scales"] = scales
    s["dw"] = torch.empty(experts, n, k, dtype=odt, device="cuda")
    return s


# ---------------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------------

def _save(x, fmt):
    """fp32 rows -> (e4m3 codes, scales, the values they stand for)."""
    rows, cols = x.shape
    size = 128 if fmt == "fp8" else 32
    groups = -(-cols // size)
    padded = torch.nn.functional.pad(x, (0, groups * size - cols)).view(rows, groups, size)
    amax = padded.abs().amax(2, keepdim=True)
    if fmt == "fp8":
        kept = scale = amax / 448.0
        codes = torch.where(scale > 0, padded / scale, torch.zeros_like(padded)).to(torch.float8_e4m3fn)
    else:
        power = (torch.frexp(amax)[1] - 9).clamp(-127, 127)
        power = torch.where(amax > 0, power, torch.full_like(power, -127))
        scale = torch.ldexp(torch.ones_like(amax), power)
        codes = torch.ldexp(padded, -power).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
        kept = (power + 127).to(torch.uint8)
    value = (codes.float() * scale).view(rows, groups * size)[:, :cols]
    codes = codes.view(torch.uint8).view(rows, groups * size)[:, :cols].contiguous()
    return codes, kept.view(rows, groups), value


def _read(q, scales, fmt):
    """(codes, scales) -> fp32 rows."""
    size = 128 if fmt == "fp8" else 32
    scale = scales if fmt == "fp8" else torch.ldexp(torch.ones_like(scales, dtype=torch.float32), scales.int() - 127)
    return q.view(torch.float8_e4m3fn).float() * scale.repeat_interleave(size, 1)[:, : q.shape[1]]


def _by_expert(rows, offsets, most):
    """rows [R, c] -> fp32 [E, most, c], zero past each expert's rows."""
    at = offsets[:-1, None] + torch.arange(most, device="cuda")
    inside = at < offsets[1:, None]
    return rows.float()[at.clamp(max=rows.shape[0] - 1)] * inside[..., None]


def _in_rows(padded, offsets, rows):
    """The inverse: [E, most, c] -> [R, c]."""
    r = torch.arange(rows, device="cuda", dtype=torch.int32)
    e = torch.searchsorted(offsets[1:], r, right=True)
    return padded[e, r - offsets[e]]


def _plain(s):
    case = s["case"]
    kind = case["kind"]
    if kind == "silu":
        gu, dh, w = s["gu"].float(), s["dh"].float(), s["weights"][:, None]
        inter = case["inter"]
        g, u = gu[:, :inter], gu[:, inter:]
        h = g * torch.sigmoid(g) * u
        g, u = _save(g, case["fmt"])[2], _save(u, case["fmt"])[2]
        sig = torch.sigmoid(g)
        silu = g * sig
        kept = silu * u
        dg = w * dh * u * (sig + silu * (1 - sig))
        du = w * dh * silu
        dt = s["gu"].dtype
        return {"h": h.to(dt), "dgu": torch.cat([dg, du], 1).to(dt), "hw": (w * kept).to(dt),
                "dweights": (dh * kept).sum(1)}
    odt = DTYPES[case["out"]]
    if kind in ("matmul", "dgrad"):
        a, w = _by_expert(s["a"], s["offsets"], s["most"]), s["w"].float()
        y = torch.bmm(a, w.transpose(1, 2) if kind == "matmul" else w)
        return _in_rows(y, s["offsets"], case["rows"]).to(odt)
    x = s["x"] if kind == "wgrad" else _read(s["q"], s["scales"], case["fmt"])
    dy, x = _by_expert(s["dy"], s["offsets"], s["most"]), _by_expert(x, s["offsets"], s["most"])
    return torch.bmm(dy.transpose(1, 2), x).to(odt)


# ---------------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------------

def _library(s):
    import block_quantized_moe_gb300 as ft
    case = s["case"]
    kind = case["kind"]
    if kind == "silu":
        fmt = ft.FMT_FP8 if case["fmt"] == "fp8" else ft.FMT_MXFP8
        ft.ftmoe_silu_mul_save(s["gu"], s["h"], s["q"], s["scales"], fmt=fmt)
        ft.ftmoe_silu_mul_backward(s["q"], s["scales"], s["dh"], s["dgu"], hw=s["hw"], row_weights=s["weights"],
                                   dweights=s["dweights"], fmt=fmt)
        return {"h": s["h"], "dgu": s["dgu"], "hw": s["hw"], "dweights": s["dweights"]}
    if kind in ("matmul", "dgrad"):
        ft.ftmoe_grouped_matmul(s["a"], s["offsets"], s["w"], s["out"], input_grad=kind == "dgrad")
        return s["out"]
    if kind == "wgrad":
        ft.ftmoe_grouped_matmul_wgrad(s["dy"], s["x"], s["offsets"], s["dw"])
    else:
        ft.ftmoe_grouped_matmul_wgrad_saved(s["dy"], s["q"], s["scales"], s["offsets"], s["dw"])
    return s["dw"]


def run(state):
    return _library(state) if own else _plain(state)


# ---------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------

def _e4m3_64(v):
    """Nearest E4M3 value, ties to even, saturating: steps of 2^(e - 3), e >= -6."""
    e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -20))).clamp(min=-6.0)
    step = torch.exp2(e - 3.0)
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def _kept_64(x, fmt):
    """The values that rows kept in 8 bits stand for: per 128 columns amax / 448 as an fp32
    number, or per 32 columns the power of two floor(log2 amax) - 8. A code is that of the
    fp32 quotient, as the format has it."""
    group = (torch.arange(x.shape[1], device="cuda") // (128 if fmt == "fp8" else 32)).expand(x.shape)
    amax = torch.zeros_like(x).scatter_reduce(1, group, x.abs(), "amax").gather(1, group)
    if fmt == "fp8":
        scale = (amax / 448.0).float().double()
    else:
        scale = torch.exp2((torch.floor(torch.log2(amax.clamp(min=1e-300))) - 8.0).clamp(-127.0, 127.0))
    quotient = (x / scale.clamp(min=1e-300)).float().double()
    return torch.where(scale > 0, _e4m3_64(quotient) * scale, torch.zeros_like(x))


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "silu":
        inter = case["inter"]
        gu, dh, w = s["gu"].double(), s["dh"].double(), s["weights"].double()[:, None]
        g, u = gu[:, :inter], gu[:, inter:]
        h = g / (1 + torch.exp(-g)) * u
        g, u = _kept_64(g, case["fmt"]), _kept_64(u, case["fmt"])
        e = torch.exp(-g)
        silu = g / (1 + e)
        slope = (1 + e + g * e) / (1 + e) ** 2
        return {"h": h, "dgu": torch.cat([w * dh * u * slope, w * dh * silu], 1), "hw": w * silu * u,
                "dweights": torch.einsum("ri,ri->r", dh, silu * u)}
    bounds = s["offsets"].tolist()
    out = s["out"] if kind in ("matmul", "dgrad") else s["dw"]
    got = torch.zeros(out.shape, dtype=torch.float64, device="cuda")
    for e in range(case["experts"]):
        part = slice(bounds[e], bounds[e + 1])
        if kind == "matmul":
            got[part] = s["a"][part].double() @ s["w"][e].double().T
        elif kind == "dgrad":
            got[part] = s["a"][part].double() @ s["w"][e].double()
        elif kind == "wgrad":
            got[e] = s["dy"][part].double().T @ s["x"][part].double()
        else:
            x = s["q"][part].view(torch.float8_e4m3fn).double().view(-1, case["k"] // 32, 32)
            x = x * torch.exp2(s["scales"][part].double() - 127.0)[..., None]
            got[e] = s["dy"][part].double().T @ x.view(-1, case["k"])
    return got
