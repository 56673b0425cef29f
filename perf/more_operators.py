"""The operators around the routed experts' products, as measured workloads.

What is measured: routing tokens to experts (scores of the router's logits, a bias for balance,
groups, top-k, renormalised weights) and its gradient; the global norm of many gradients with the
factor that clips it; an AdamW step over many tensors at once, with its moments in 32 bits or in 8.

Sizes are the repository's benchmark geometries: 64 experts with top-8, 256 experts with top-6 at
up to 4,096 tokens, and the gate/up bank of a 32-expert training shard, 4096 x 7168 per expert.

Moments in 8 bits: per 32 consecutive elements a power of two (a byte b for 2^(b - 127)), the first
moment in e4m3 and the second in e5m2, so that the largest of the 32 is at most the format's
largest. Each value is rounded up or down at random in proportion to what is cut off, by 16 random
bits of a hash of (seed, step, tensor, element); a second moment above zero is never rounded to zero.

`run` computes the plain form in elementary torch operations, or, where `own` is set, makes the
calls of the library. `exact` gives the same outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
LR, BETA1, BETA2, EPS, DECAY, STEP = 1e-4, 0.9, 0.999, 1e-8, 0.1, 1000  # one AdamW step in mid-training
MAX_NORM = 1.0

# odd 32-bit integers near the fractional parts of sqrt(2) and sqrt(3), and of sqrt(5) to sqrt(29)
MIX_A, MIX_B = 0x6A09E667, 0xBB67AE85
SPREAD = (0x3C6EF373, 0xA54FF53B, 0x510E527F, 0x9B05688D, 0x1F83D9AB, 0x5BE0CD19, 0xCBBB9D5D, 0x629A292B)
LOW = 0xFFFFFFFF


# ---------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------

def _route(name, kind, tokens, experts, topk, score, renorm, bias, groups, keep, best, scale, dtype):
    return {"name": name, "kind": kind, "tokens": tokens, "experts": experts, "topk": topk, "score": score,
            "renorm": renorm, "bias": bias, "groups": groups, "keep": keep, "best": best, "scale": scale,
            "dtype": dtype}


def _tensors(name, kind, count, largest, dtype, state="none", copy="none"):
    return {"name": name, "kind": kind, "count": count, "largest": largest, "dtype": dtype, "state": state, "copy": copy}


def listed():
    return [
        # one decoded token, top-8 of 64 experts: latency
        _route("route decode 1 token", "route", 1, 64, 8, "softmax", True, False, 1, 1, 1, 1.0, "fp32"),
        # eight decoded tokens, top-6 of 256 experts with balance bias and groups: latency
        _route("route decode 8 tokens", "route", 8, 256, 6, "sigmoid", True, True, 8, 4, 2, 2.5, "fp32"),
        # an odd batch, weights not renormalised, groups by their best expert
        _route("route 1111 tokens", "route", 1111, 96, 5, "softmax", False, False, 4, 2, 1, 16.0, "fp16"),
        # a prompt of 4,096 tokens, top-6 of 256 experts, logits in 16 bits
        _route("route prompt 4096 tokens", "route", 4096, 256, 6, "softmax", True, False, 1, 1, 1, 1.0, "bf16"),
        # a training batch, balance bias and groups
        _route("route train 32768 tokens", "route", 32768, 256, 8, "sigmoid", True, True, 8, 4, 2, 2.5, "fp32"),
        # the router's gradient for an odd batch
        _route("route grad 333 tokens", "grad", 333, 64, 8, "sigmoid", True, False, 1, 1, 1, 1.0, "fp32"),
        # the router's gradient of a training batch, through every expert's score
        _route("route grad train", "grad", 32768, 256, 6, "softmax", False, False, 1, 1, 1, 1.0, "bf16"),
        # the router's matrices and norms of a small model, fp32 gradients of odd sizes
        _tensors("norm 24 small tensors", "norm", 24, 65537, "fp32"),
        # the gate/up gradient of a training shard of 32 experts
        _tensors("norm expert shard", "norm", 1, 32 * 4096 * 7168, "bf16"),
        # the same small tensors' AdamW step
        _tensors("adamw 24 small tensors", "adamw", 24, 65537, "fp32", "fp32"),
        # the shard's step: fp32 master and moments, 16-bit gradient and the bank that products read
        _tensors("adamw expert shard", "adamw", 1, 32 * 4096 * 7168, "bf16", "fp32", "bf16"),
        # the shard's step with moments in 8 bits
        _tensors("adamw expert shard 8 bits", "adamw", 1, 32 * 4096 * 7168, "bf16", "8bit", "bf16"),
    ]


def _log_int(rng, lo, hi, step=1):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return min(hi, max(lo, (v + step // 2) // step * step))


def draw(rng):
    kind = rng.choice(["route", "route", "grad", "norm", "adamw", "adamw"])
    if kind in ("route", "grad"):
        groups = rng.choice([1, 1, 4, 8])
        experts = max(16, _log_int(rng, 8, 256) // groups * groups)
        keep = rng.randint(1, groups)
        topk = rng.randint(1, min(8, keep * (experts // groups)))
        return {"kind": kind, "tokens": _log_int(rng, 1, 32768), "experts": experts, "topk": topk,
                "score": rng.choice(["softmax", "sigmoid"]), "renorm": rng.choice([True, False]),
                "bias": rng.choice([True, False]), "groups": groups, "keep": keep, "best": rng.choice([1, 2]),
                "scale": rng.choice([1.0, 2.5]), "dtype": rng.choice(["fp32", "fp32", "bf16", "fp16"])}
    case = {"kind": kind, "count": _log_int(rng, 1, 40), "largest": _log_int(rng, 1, 1 << 26),
            "dtype": rng.choice(["fp32", "bf16", "fp16"]), "state": "none", "copy": "none"}
    if kind == "adamw":
        case["state"] = rng.choice(["fp32", "8bit"])
        case["copy"] = rng.choice(["none", "bf16", "fp16"])
    return case


def _sizes(case):
    """Elements of each tensor: the largest, and fractions of it, odd ones among them."""
    return [case["largest"] // (i + 1) + i for i in range(case["count"])]


def _span(sizes):
    """Elements of a buffer that holds tensors of these sizes, each at a multiple of 64."""
    return sum(-(-n // 64) * 64 for n in sizes)


def _views(flat, sizes, per=1):
    """The tensors in it (their groups of `per` elements)."""
    at = [_span(sizes[:i]) // per for i in range(len(sizes))]
    return [flat[a: a + -(-n // per)] for a, n in zip(at, sizes)]


def work(case):
    if case["kind"] in ("route", "grad"):
        tokens, experts, topk = case["tokens"], case["experts"], case["topk"]
        size = 4 if case["dtype"] == "fp32" else 2
        if case["kind"] == "route":
            return {"bytes": tokens * (experts * size + topk * 8) + (4 * experts if case["bias"] else 0),
                    "flops": tokens * experts * 10}
        # the chosen experts' logits for sigmoid scores, every expert's for plain softmax scores
        logits = topk if case["score"] == "sigmoid" else 0 if case["renorm"] else experts
        return {"bytes": tokens * (topk * 12 + logits * size + experts * size), "flops": tokens * (experts * 4 + topk * 8)}
    n = sum(_sizes(case))
    grad = 4 if case["dtype"] == "fp32" else 2
    if case["kind"] == "norm":
        return {"bytes": n * grad + 8, "flops": 2 * n}
    moments = 16 * n if case["state"] == "fp32" else 4 * n + sum(4 * -(-k // 32) for k in _sizes(case))
    return {"bytes": n * (8 + grad + (0 if case["copy"] == "none" else 2)) + moments, "flops": 16 * n}


# ---------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------

def _normal(shape, std, dtype, gen):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=gen)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"case": case, "seed": seed % (1 << 32)}
    dt = DTYPES[case["dtype"]]
    if case["kind"] in ("route", "grad"):
        tokens, experts, topk = case["tokens"], case["experts"], case["topk"]
        s["logits"] = _normal((tokens, experts), 1.5, dt, gen)
        s["bias"] = _normal((experts,), 0.1, torch.float32, gen) if case["bias"] else None
        s["ids"] = torch.empty(tokens, topk, dtype=torch.int32, device="cuda")
        s["weights"] = torch.empty(tokens, topk, device="cuda")
        if case["kind"] == "grad":
            ids, weights = _plain_route(s)
            s["ids"].copy_(ids)
            s["weights"].copy_(weights)
            s["dweights"] = _normal((tokens, topk), 0.1, torch.float32, gen)
            s["dlogits"] = torch.empty(tokens, experts, dtype=dt, device="cuda")
        if own:
            import block_quantized_moe_gb300 as ft
            s["router"] = ft.make_router(experts, topk, score=ft.SCORE_SOFTMAX if case["score"] == "softmax" else ft.SCORE_SIGMOID,
                                         renormalize=case["renorm"], groups=case["groups"], group_topk=case["keep"],
                                         group_best=case["best"], scale=case["scale"])
        return s
    sizes = _sizes(case)
    grads = _normal((_span(sizes),), 1e-3, dt, gen)
    s["grads"] = _views(grads, sizes)
    if case["kind"] == "norm":
        s["result"] = torch.empty(2, device="cuda")
        if own:
            import block_quantized_moe_gb300 as ft
            s["list"] = ft.make_grad_list(s["grads"])
            s["workspace"] = torch.empty(ft.ftmoe_grad_norm_workspace_bytes(s["list"]), dtype=torch.uint8, device="cuda")
        return s
    s["scale"] = torch.full((1,), 0.5, device="cuda")  # the factor that clips the gradients
    # each kind in one buffer, as programs keep them; the moments are those that a few thousand such gradients leave
    flat = {"params": _normal(grads.shape, 0.02, torch.float32, gen), "m": _normal(grads.shape, 1e-4, torch.float32, gen),
            "v": _normal(grads.shape, 2e-4, torch.float32, gen).square_().add_(1e-8)}
    if case["state"] == "8bit":
        flat["m"], flat["m_scales"], flat["v"], flat["v_scales"] = _kept(flat["m"], flat["v"], 0, 0)
    if case["copy"] != "none":
        flat["copies"] = flat["params"].to(DTYPES[case["copy"]])
    s["flat"] = flat
    for k in ("params", "m", "v", "copies"):
        s[k] = _views(flat[k], sizes) if k in flat else None
    for k in ("m_scales", "v_scales"):
        s[k] = _views(flat[k], sizes, 32) if k in flat else None
    if own:
        import block_quantized_moe_gb300 as ft
        s["list"] = ft.make_adamw_list(s["params"], s["grads"], s["m"], s["v"], m_scales=s["m_scales"],
                                       v_scales=s["v_scales"], copies=s["copies"])
    return s


# ---------------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------------

def _scores(x, score):
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-x))
    e = torch.exp(x - x.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _plain_route(s):
    """Scores in 64 bits: values next to a border decide which expert it is."""
    case = s["case"]
    score = _scores(s["logits"].double(), case["score"])
    value = score if s["bias"] is None else score + s["bias"]
    if case["groups"] > 1:
        grouped = value.view(case["tokens"], case["groups"], -1)
        best = grouped.sort(dim=2, descending=True)[0][:, :, : case["best"]].sum(2)
        kept = best.sort(dim=1, descending=True, stable=True)[1][:, : case["keep"]]
        out = torch.ones_like(best, dtype=torch.bool).scatter_(1, kept, False)
        value = grouped.masked_fill(out[:, :, None], -math.inf).view_as(value)
    ids = value.sort(dim=1, descending=True, stable=True)[1][:, : case["topk"]]
    w = score.gather(1, ids)
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return ids.int(), (w * case["scale"]).float()


def _plain_grad(s):
    case = s["case"]
    ids, scale = s["ids"].long(), case["scale"]
    x = s["logits"].float()
    score = _scores(x, case["score"])
    dw = s["dweights"] * scale
    if case["renorm"]:
        chosen = score.gather(1, ids)
        total = chosen.sum(1, keepdim=True)
        dw = (dw - (dw * chosen).sum(1, keepdim=True) / total) / total
    dscore = torch.zeros_like(x).scatter_(1, ids, dw)
    if case["score"] == "sigmoid":
        dx = dscore * score * (1.0 / (1.0 + torch.exp(x)))
    else:
        dx = score * (dscore - (dscore * score).sum(1, keepdim=True))
    return dx.to(s["logits"].dtype)


def _plain_norm(s):
    total = sum(g.float().square().sum(dtype=torch.float64) for g in s["grads"])  # a long sum
    norm = total.sqrt()
    return torch.stack([norm, (MAX_NORM / (norm + 1e-6)).clamp(max=1.0)]).float()


def _mix(x):
    x = x ^ (x >> 16)
    x = x * MIX_A & LOW
    x = x ^ (x >> 15)
    x = x * MIX_B & LOW
    return x ^ (x >> 16)


def _noise(n, seed, step, tensor):
    """32 random bits for each element: chunks of eight share a hash."""
    key = _mix(_mix(_mix(seed) + step & LOW) + tensor & LOW)
    chunk = torch.arange(-(-n // 8), device="cuda")
    base = _mix(_mix(key + (chunk >> 32) & LOW) + chunk & LOW)
    h = base[:, None] * torch.tensor(SPREAD, device="cuda")
    return ((h >> 32 ^ h) & LOW).view(-1)[:n]


def _by_scale(x):
    """[n] -> [groups, 32], zero past the end."""
    return torch.nn.functional.pad(x, (0, -x.numel() % 32)).view(-1, 32)


def _codes(x, noise, top, least, cut):
    """(codes, scale bytes) of |x|: the format's largest value is 1.75 * 2^top, its normal values
    begin at 2^least, `cut` bits of an fp32 number are beyond its own. Products by powers of two
    that put 2^least on fp32's first normal number make the bits above `cut` the code."""
    x = _by_scale(x)
    bits = x.view(torch.int32).amax(1, keepdim=True)
    power = ((bits + 0x1FFFFF >> 23) - 127 - top).clamp(min=-127)
    one = torch.ones((), device="cuda")
    x = x * torch.ldexp(one, -power) * 2.0 ** (-126 - least)
    codes = x.view(torch.int32) + (_by_scale(noise).int() << cut - 16) >> cut
    return codes, (power + 127).to(torch.uint8).view(-1)


def _kept(m, v, seed, tensor, step=0):
    """The moments in 8 bits: e4m3 codes, scale bytes, e5m2 codes, scale bytes."""
    n = m.numel()
    noise = _noise(n, seed, step, tensor)
    low, high = noise & 0xFFFF, noise >> 16
    del noise
    q, m_scales = _codes(m.abs(), low, 8, -6, 20)
    q = q.view(-1)[:n] + 128 * (m.view(torch.int32) < 0)
    r, v_scales = _codes(v, high, 15, -14, 21)
    r = torch.maximum(r.view(-1)[:n], (v > 0).int())
    return (q.to(torch.uint8).view(torch.float8_e4m3fn), m_scales.view(torch.float8_e8m0fnu),
            r.to(torch.uint8).view(torch.float8_e5m2), v_scales.view(torch.float8_e8m0fnu))


def _value(codes, scales):
    n = codes.numel()
    scales = torch.ldexp(torch.ones((), device="cuda"), scales.view(torch.uint8).int() - 127)
    return (_by_scale(codes.float()) * scales[:, None]).view(-1)[:n]


def _plain_adamw_one(s, i):
    case = s["case"]
    g = s["grads"][i].float() * s["scale"]
    m, v = s["m"][i], s["v"][i]
    if case["state"] == "8bit":
        m, v = _value(m, s["m_scales"][i]), _value(v, s["v_scales"][i])
    m = m * BETA1 + g * (1 - BETA1)
    v = v * BETA2 + g * g * (1 - BETA2)
    del g
    denominator = v.sqrt() / math.sqrt(1 - BETA2 ** STEP) + EPS
    s["params"][i].mul_(1 - LR * DECAY).sub_(m / denominator * (LR / (1 - BETA1 ** STEP)))
    del denominator
    if s["copies"] is not None:
        s["copies"][i].copy_(s["params"][i])
    if case["state"] == "8bit":
        kept = _kept(m, v, s["seed"], i, STEP)
        s["m"][i].copy_(kept[0])
        s["m_scales"][i].copy_(kept[1])
        s["v"][i].copy_(kept[2])
        s["v_scales"][i].copy_(kept[3])
    else:
        s["m"][i].copy_(m)
        s["v"][i].copy_(v)


def _plain(s):
    kind = s["case"]["kind"]
    if kind == "route":
        ids, weights = _plain_route(s)
        return {"ids": ids, "weights": weights}
    if kind == "grad":
        return _plain_grad(s)
    if kind == "norm":
        return _plain_norm(s)
    [_plain_adamw_one(s, i) for i in range(len(s["grads"]))]
    return s["flat"]


# ---------------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------------

def _library(s):
    import block_quantized_moe_gb300 as ft
    kind = s["case"]["kind"]
    if kind == "route":
        ft.ftmoe_route_tokens(s["logits"], s["router"], s["ids"], s["weights"], bias=s["bias"])
        return {"ids": s["ids"], "weights": s["weights"]}
    if kind == "grad":
        ft.ftmoe_route_tokens_backward(s["logits"], s["router"], s["ids"], s["weights"], s["dweights"], s["dlogits"])
        return s["dlogits"]
    if kind == "norm":
        ft.ftmoe_grad_norm(s["list"], s["result"], s["workspace"], max_norm=MAX_NORM)
        return s["result"]
    ft.ftmoe_adamw_step(s["list"], step=STEP, lr=LR, beta1=BETA1, beta2=BETA2, eps=EPS, weight_decay=DECAY,
                        grad_scale=s["scale"], seed=s["seed"])
    return s["flat"]


def run(state):
    return _library(state) if own else _plain(state)


# ---------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------

def _exact_route(case, s):
    x = s["logits"].double()
    if case["score"] == "softmax":
        score = torch.exp(x - torch.logsumexp(x, 1, keepdim=True))
    else:
        score = torch.where(x < 0, torch.exp(x) / (1 + torch.exp(x)), 1 / (1 + torch.exp(-x)))
    value = score.clone()
    if s["bias"] is not None:
        value += s["bias"].double()
    size = case["experts"] // case["groups"]
    rows = torch.arange(case["tokens"], device="cuda")
    if case["groups"] > 1:
        rest, total = value.view(-1, case["groups"], size).clone(), 0.0
        for _ in range(min(case["best"], size)):
            top = rest.max(2)
            total = total + top[0]
            rest.scatter_(2, top[1][:, :, None], -math.inf)
        keep = torch.zeros_like(total)
        for _ in range(case["keep"]):
            best = (total == total.amax(1, keepdim=True)).int().argmax(1)
            keep[rows, best], total[rows, best] = 1.0, -math.inf
        value[keep.repeat_interleave(size, 1) == 0] = -math.inf
    picked = []
    for _ in range(case["topk"]):
        best = (value == value.amax(1, keepdim=True)).int().argmax(1)
        picked.append(best)
        value[rows, best] = -math.inf
    w = torch.stack([score[rows, e] for e in picked], 1)
    return case["scale"] * (w / w.sum(1, keepdim=True) if case["renorm"] else w)


def _exact_grad(case, s):
    """By the Jacobian: the weights' gradients from dlog w_i / dx_e."""
    x, ids, c = s["logits"].double(), s["ids"].long(), s["dweights"].double()
    hit = torch.zeros(*ids.shape, case["experts"], dtype=torch.float64, device="cuda").scatter_(2, ids[:, :, None], 1.0)
    if case["score"] == "softmax":
        score = torch.softmax(x, 1)
        log_slope = hit - score[:, None, :]
    else:
        score = torch.sigmoid(x)
        log_slope = hit * torch.sigmoid(-x)[:, None, :]
    w = score.gather(1, ids)
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True)
        log_slope = log_slope - torch.einsum("tk,tke->te", w, log_slope)[:, None, :]
    return case["scale"] * torch.einsum("tk,tke->te", w * c, log_slope)


def _exact_round(x, noise, top, least, digits):
    """64-bit values rounded to steps of 2^(e - digits), e >= least, up with the chance of what is cut off."""
    x, n = _by_scale(x), x.numel()
    amax = x.amax(1, keepdim=True)
    e = torch.floor(torch.log2(amax.clamp(min=1e-300)))
    e = e + (amax > 1.75 * torch.exp2(e)) - top
    e = e.clamp(min=-127.0)
    x = x * torch.exp2(-e)
    step = torch.exp2(torch.floor(torch.log2(x.clamp(min=1e-300))).clamp(min=least) - digits)
    q = torch.floor(x / step + _by_scale(noise) / 65536.0) * step
    return q.view(-1)[:n], torch.exp2(e).view(-1)


def _exact_adamw(case, s, i):
    def stands_for(codes, scales):
        groups = scales.view(torch.uint8).double().sub_(127).exp2_()
        return codes.double() * groups.repeat_interleave(32)[: codes.numel()]
    g = s["grads"][i].double() * 0.5
    m, v = s["m"][i], s["v"][i]
    if case["state"] == "8bit":
        m, v = stands_for(m, s["m_scales"][i]), stands_for(v, s["v_scales"][i])
    m = BETA1 * m.double() + (1 - BETA1) * g
    v = BETA2 * v.double() + (1 - BETA2) * g ** 2
    p = s["params"][i].double()
    p = p - LR * DECAY * p - LR * (m / (1 - BETA1 ** STEP)) / (torch.sqrt(v / (1 - BETA2 ** STEP)) + EPS)
    out = {"params": p, "m": m, "v": v}
    if s["copies"] is not None:
        out["copies"] = p
    if case["state"] == "8bit":
        noise = _noise(m.numel(), s["seed"], STEP, i)
        q, out["m_scales"] = _exact_round(m.abs(), noise & 0xFFFF, 8, -6.0, 3)
        out["m"] = torch.where(m < 0, -q, q)
        q, out["v_scales"] = _exact_round(v, noise >> 16, 15, -14.0, 2)
        out["v"] = torch.where(v > 0, q.clamp(min=2.0 ** -16), q)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "route":
        return {"ids": None, "weights": _exact_route(case, s)}
    if case["kind"] == "grad":
        return _exact_grad(case, s)
    if case["kind"] == "norm":
        norm = math.sqrt(sum(float(torch.linalg.vector_norm(g.double())) ** 2 for g in s["grads"]))
        return torch.tensor([norm, min(1.0, MAX_NORM / (norm + 1e-6))], dtype=torch.float64)
    sizes, out = _sizes(case), {k: v.double() for k, v in s["flat"].items()}
    for i in range(len(sizes)):
        for k, v in _exact_adamw(case, s, i).items():
            _views(out[k], sizes, 32 if k.endswith("scales") else 1)[i].copy_(v)
    return out
