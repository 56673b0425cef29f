"""Routing and its gradient against the definitions in 64 bits."""
import math

import numpy as np
import pytest
import torch

import block_quantized_moe_gb300 as ft

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS32 = 2.0 ** -24  # half a step of fp32


def reference(x, r, bias=None):
    """(ids, weights) of fp64 logits [T, E], a token at a time."""
    T, E = x.shape
    ids, weights = np.full((T, r.topk), -1), np.zeros((T, r.topk))
    size = E // r.groups
    for t in range(T):
        ok = x[t] > -np.inf
        row = np.where(ok, np.minimum(np.nan_to_num(x[t], nan=0.0, neginf=0.0), np.finfo(np.float32).max), -np.inf)
        if not ok.any():
            continue
        with np.errstate(over="ignore"):
            e = np.exp(row - row.max())
            score = e / e.sum() if r.score == ft.SCORE_SOFTMAX else 1 / (1 + np.exp(-row))
        value = score if bias is None else score + np.minimum(np.nan_to_num(bias, nan=-np.inf), np.finfo(np.float32).max)
        ok = ok & (value > -np.inf) if bias is not None else ok
        value = np.where(ok, value, -np.inf)
        if r.groups > 1:
            best = []
            for g in range(r.groups):
                top = np.sort(value[g * size:(g + 1) * size])[::-1][:r.group_best]
                best.append(sum(top[top > -np.inf]) if (top > -np.inf).any() else -np.inf)
            kept = np.argsort(-np.array(best), kind="stable")[:r.group_topk]
            ok = ok & np.isin(np.arange(E) // size, kept)
        order = np.where(ok, row if bias is None else value, -np.inf)
        chosen = [e for e in np.argsort(-order, kind="stable")[:r.topk] if ok[e]]
        ids[t, :len(chosen)] = chosen
        if r.renormalize and chosen:  # exp(-t) s with t = min(largest, 0): no underflow
            c = row[chosen]
            low = min(c.max(), 0.0)
            with np.errstate(over="ignore"):
                s = np.exp(c - c.max()) if r.score == ft.SCORE_SOFTMAX else 1 / (np.exp(low) + np.exp(low - c))
            weights[t, :len(chosen)] = s / s.sum()
        else:
            weights[t, :len(chosen)] = score[chosen]
    return ids, weights * float(np.float32(r.scale))


def route(x, r, bias=None, tokens_dev=None):
    T = x.shape[0]
    ids = torch.full((T, r.topk), -7, dtype=torch.int32, device=DEV)
    w = torch.full((T, r.topk), math.nan, device=DEV)
    ft.ftmoe_route_tokens(x, r, ids, w, bias=bias, tokens_dev=tokens_dev)
    return ids, w


def check(x, r, bias=None):
    ids, w = route(x, r, bias)
    x64 = x.double().cpu().numpy()
    want_ids, want = reference(x64, r, None if bias is None else bias.double().cpu().numpy())
    np.testing.assert_array_equal(ids.cpu().numpy(), want_ids)
    # exponentials of fp32 arguments d (rounded: |d| half steps), of two half steps themselves; a sum of up to
    # 1,024 in a tree of 10 levels and 32 terms a lane at most, a quotient, the scale: 48 half steps more
    finite = np.where(np.isfinite(x64), x64, 0.0)
    d = np.minimum(np.abs(finite).max(1, keepdims=True) * 2, 110.0)
    got = w.double().cpu().numpy()
    assert (np.abs(got - want) <= want * (d + 50) * EPS32 + 1e-37).all(), np.abs(got / np.maximum(want, 1e-300) - 1).max()
    assert ft.ftmoe_read_error_flags() == 0
    return ids, w


def logits(T, E, dtype, seed, std=1.5, pad=0):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    wide = torch.randn(T, E + pad, generator=gen, device=DEV) * std
    return wide.to(DTYPES[dtype])[:, pad // 2:pad // 2 + E]


def router(E, k, score="softmax", **kw):
    return ft.make_router(E, k, score=ft.SCORE_SOFTMAX if score == "softmax" else ft.SCORE_SIGMOID, **kw)


# (experts, topk, groups, groups kept, best): lanes that hold one expert to 32; groups of whole lanes and others
SHAPES = [(1, 1, 1, 1, 1), (2, 2, 2, 1, 1), (7, 3, 1, 1, 1), (16, 4, 4, 2, 2), (32, 8, 1, 1, 1), (60, 6, 4, 2, 2), (64, 8, 1, 1, 1),
          (96, 5, 4, 2, 1), (128, 32, 1, 1, 1), (160, 6, 8, 3, 2), (256, 6, 8, 4, 2), (256, 8, 32, 5, 1), (257, 8, 1, 1, 1),
          (384, 8, 3, 1, 2), (512, 10, 16, 16, 2), (1000, 9, 8, 2, 1), (1024, 32, 32, 16, 2)]
SHAPES = [s if s[1] <= s[3] * (s[0] // s[2]) else (s[0], s[3] * (s[0] // s[2]), *s[2:]) for s in SHAPES]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_against_64_bits(shape, score):
    E, k, groups, keep, best = shape
    for i, (dtype, renorm, biased, pad) in enumerate([("fp32", True, True, 0), ("bf16", False, False, 0), ("fp16", True, True, 3),
                                                      ("fp32", False, False, 5), ("bf16", True, True, 8)]):
        x = logits(37, E, dtype, 100 * E + i, pad=pad)
        bias = torch.linspace(-0.2, 0.2, E, device=DEV).flip(0).contiguous() if biased else None
        r = router(E, k, score, renormalize=renorm, groups=groups, group_topk=keep, group_best=best, scale=2.5 if renorm else 1.0)
        check(x, r, bias)


@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 127, 1111])
def test_numbers_of_tokens(T):
    check(logits(T, 64, "fp32", T), router(64, 8))
    check(logits(T, 64, "bf16", T), router(64, 8, "sigmoid", groups=8, group_topk=4, group_best=2), torch.zeros(64, device=DEV))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_ties_go_to_the_lower_expert(score):
    """Logits of few values, biases of one value and of two; every expert alike."""
    x = torch.randint(-2, 3, (64, 256), device=DEV, generator=torch.Generator(device=DEV).manual_seed(1)).float()
    x[:8] = 0.0
    for kw in (dict(), dict(groups=8, group_topk=3, group_best=2), dict(groups=4, group_topk=2)):
        r = router(256, 8, score, **kw)
        check(x, r)
        check(x, r, torch.full((256,), 0.25, device=DEV))
        check(x, r, (torch.arange(256, device=DEV) % 2).float())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,kw", [(64, {}), (256, dict(groups=8, group_topk=4, group_best=2)), (96, dict(groups=4, group_topk=3)),
                                  (1024, {})])
def test_values_nearer_than_fp32(score, E, kw):
    """Biases that bring every value of a token within fp32's rounding of 0.8: the order is that of
    64 bits. (One token's bias suits one token, so each has a call of its own.)"""
    x = logits(8, E, "fp32", E)
    for t in range(8):
        row = x[t].double()
        s = torch.softmax(row, 0) if score == "softmax" else torch.sigmoid(row)
        check(x[t:t + 1], router(E, 6, score, **kw), (0.8 - s).float())


def test_values_that_differ_by_a_few_units():
    """Pairs of logits one fp32 step apart, with equal biases and with zeros."""
    x = logits(64, 128, "fp32", 9)
    x[:, 64:] = torch.nextafter(x[:, :64], torch.full_like(x[:, :64], 100.0))
    for score in ("softmax", "sigmoid"):
        check(x, router(128, 8, score), torch.zeros(128, device=DEV))
        check(x, router(128, 8, score, groups=2, group_topk=1, group_best=2), torch.full((128,), 0.5, device=DEV))


@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_masked_experts(score, biased):
    """Logits of -inf, NaN, +inf and the type's lowest value; rows of nothing else."""
    low = torch.finfo(torch.float32).min
    x = logits(16, 32, "fp32", 3)
    x[0] = -math.inf
    x[1] = math.nan
    x[2] = low
    x[3, ::2] = -math.inf
    x[4, 1:] = -math.inf
    x[5, 5:] = math.nan
    x[6, 3] = math.inf
    x[7, 4:9] = math.inf
    x[8, 2:] = low
    x[9] = -200.0 - torch.arange(32, device=DEV)  # sigmoids below fp32's range
    x[10] = 90.0 + torch.arange(32, device=DEV)   # sigmoids of one
    x[11] = math.inf
    x[12, 8:] = -math.inf                         # one group of four left
    bias = torch.linspace(-0.1, 0.1, 32, device=DEV) if biased else None
    for kw in (dict(), dict(groups=4, group_topk=2, group_best=2), dict(renormalize=False)):
        check(x, router(32, 6, score, **kw), bias)
    ids, w = route(x, router(32, 6, score), bias)
    assert (ids[:2] == -1).all() and (w[:2] == 0).all() and (ids[2] >= 0).all()
    assert torch.equal(ids[4], torch.tensor([0] + [-1] * 5, dtype=torch.int32, device=DEV))
    assert torch.allclose(w[2], torch.full((6,), 1 / 6, device=DEV))


@pytest.mark.parametrize("E", [8, 32, 64, 256])
@pytest.mark.parametrize("biased", [False, True])
def test_fewer_experts_than_slots(E, biased):
    """Rows of 0 to 8 experts that can be chosen, next to each other and apart."""
    x = logits(34, E, "fp32", E)
    for t in range(17):
        x[t, t % 9:] = -math.inf
        mask = torch.ones(E, dtype=torch.bool, device=DEV)
        mask[torch.arange(t % 9, device=DEV) * (E // 8) % E] = False
        x[17 + t].masked_fill_(mask, -math.inf)
    bias = torch.linspace(-0.1, 0.1, E, device=DEV) if biased else None
    for score in ("softmax", "sigmoid"):
        check(x, router(E, 8, score), bias)
        check(x, router(E, 4, score, groups=4, group_topk=2, group_best=2), bias)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_the_best_next_to_each_other(score, biased):
    """The chosen in one lane's experts, or few lanes'."""
    x = logits(64, 256, "fp32", 12, std=0.5)
    for t in range(64):
        x[t, 3 * t:3 * t + 2 + t % 11] += 6.0
    bias = torch.linspace(-0.1, 0.1, 256, device=DEV) if biased else None
    check(x, router(256, 8, score), bias)
    check(x, router(256, 12, score, groups=8, group_topk=3, group_best=2), bias)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("E,groups,best", [(256, 8, 2), (256, 8, 1), (64, 8, 2), (96, 4, 2), (512, 16, 2)])
def test_groups_nearer_than_fp32(E, groups, best, biased, score):
    """Groups of the same logits but for one unit in the last place here and there: their scores differ by
    less than fp32 holds, or not at all."""
    size = E // groups
    x = logits(48, size, "fp32", E + groups, std=0.3).repeat(1, groups)
    pick = torch.randint(0, E, (48, 3), generator=torch.Generator(device=DEV).manual_seed(E), device=DEV)
    up = torch.nextafter(x, torch.full_like(x, 9.0))
    x.scatter_(1, pick, up.gather(1, pick))
    top = x.view(48, groups, size).argmax(2) + torch.arange(groups, device=DEV) * size  # the best of some groups too
    x[24:].scatter_(1, top[24:, ::3], up[24:].gather(1, top[24:, ::3]))
    bias = torch.linspace(-0.1, 0.1, size, device=DEV).repeat(groups) if biased else None
    check(x, router(E, 6, score, groups=groups, group_topk=groups // 2, group_best=best), bias)


def test_masking_biases():
    x = logits(8, 32, "fp32", 4)
    bias = torch.zeros(32, device=DEV)
    bias[::3], bias[1::3] = -math.inf, math.nan
    check(x, router(32, 8, "sigmoid"), bias)
    bias = torch.zeros(32, device=DEV)
    bias[5], bias[6] = math.inf, torch.finfo(torch.float32).min
    check(x, router(32, 8, "softmax"), bias)
    check(x, router(32, 32, "sigmoid"), bias)


def test_tokens_behind_the_count_are_inactive():
    x = logits(9, 64, "fp32", 5)
    x[5:] = math.nan
    for n in (0, 5, 9, 12, -3):
        count = torch.tensor([n], dtype=torch.int32, device=DEV)
        m = min(max(n, 0), 9)
        ids, w = route(x, router(64, 4), tokens_dev=count)
        want, ww = route(x, router(64, 4))
        assert torch.equal(ids[:m], want[:m]) and torch.equal(w[:m], ww[:m])
        assert (ids[m:] == -1).all() and (w[m:] == 0).all()


# ---------------------------------------------------------------------------------
# gradient
# ---------------------------------------------------------------------------------

def exact_gradient(x, r, ids, dw):
    """fp64 gradient by autograd of the weights' formula, of the active routes."""
    x = x.double().clone().requires_grad_()
    active = ids >= 0
    at = ids.long().clamp(min=0)
    if r.renormalize:
        c = x.gather(1, at).masked_fill(~active, -math.inf)
        if r.score == ft.SCORE_SOFTMAX:
            w = torch.softmax(c, 1)
        else:  # softmax of log-sigmoids
            w = torch.softmax(torch.nn.functional.logsigmoid(x.gather(1, at)).masked_fill(~active, -math.inf), 1)
    else:
        s = torch.softmax(x, 1) if r.score == ft.SCORE_SOFTMAX else torch.sigmoid(x)
        w = s.gather(1, at)
    w = torch.where(active, w, torch.zeros_like(w))
    (r.scale * w * torch.where(active, dw.double(), torch.zeros_like(w))).sum().backward()
    return x.grad.nan_to_num(nan=0.0)  # rows without an active route


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("E,k", [(1, 1), (2, 1), (7, 3), (64, 8), (96, 5), (129, 4), (256, 6), (256, 16), (256, 17), (500, 32), (512, 16), (513, 16), (1024, 9)])
def test_gradient(E, k, renorm, score):
    for T, dtype, out, pad in ((33, "fp32", "fp32", 0), (5, "bf16", "bf16", 0), (6, "fp16", "fp32", 3), (4, "fp32", "fp16", 8)):
        x = logits(T, E, dtype, E + T, pad=pad)
        r = router(E, k, score, renormalize=renorm, scale=2.5)
        ids, w = route(x, r)
        if T == 33:
            ids[3], ids[4, :k // 2], ids[5, -1] = -1, -1, -1
            # the weights of the routes that are left
            ref = x.double().gather(1, ids.long().clamp(min=0))
            if renorm:
                ref = ref if score == "softmax" else torch.nn.functional.logsigmoid(ref)
                w = torch.softmax(ref.masked_fill(ids < 0, -math.inf), 1).float() * 2.5
            w = torch.where(ids >= 0, w, torch.full_like(w, math.nan))
        dw = torch.randn(T, k, device=DEV, generator=torch.Generator(device=DEV).manual_seed(E))
        dw = torch.where(ids >= 0, dw, torch.full_like(dw, math.nan))
        wide = torch.full((T, E + pad), 7.0, dtype=DTYPES[out], device=DEV)
        d = wide[:, :E]
        ft.ftmoe_route_tokens_backward(x, r, ids, w, dw, d)
        want = exact_gradient(x, r, ids, dw)
        # the terms r_i, w_i R / c and s_e R in fp32 (weights off by 50 + |x| half steps, sums of 32)
        terms = torch.where(ids >= 0, (w * dw).double().abs(), torch.zeros_like(w, dtype=torch.float64)).sum(1, keepdim=True)
        limit = terms * 200 * EPS32 + want.abs() * torch.finfo(DTYPES[out]).eps / 2 + torch.finfo(DTYPES[out]).tiny * 2.0 ** -8
        assert ((d.double() - want).abs() <= limit).all()
        assert (wide[:, E:] == 7.0).all()
        assert T != 33 or (d[3] == 0).all()
    assert ft.ftmoe_read_error_flags() == 0


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_gradient_against_differences(score, renorm):
    """Central differences of the library's own weights: of step h their error is h^2 / 6 of the third
    derivative (below the scale) and the weights' rounding over h."""
    E, k, h = 12, 4, 2.0 ** -7
    x = logits(1, E, "fp32", 21)
    r = router(E, k, score, renormalize=renorm)
    ids, w = route(x, r)
    dw = torch.tensor([[0.5, -1.0, 2.0, 0.25]], device=DEV)
    d = torch.empty_like(x)
    ft.ftmoe_route_tokens_backward(x, r, ids, w, dw, d)
    for e in range(E):
        total = 0.0
        for sign in (1, -1):
            y = x.clone()
            y[0, e] += sign * h
            at, ww = route(y, r)
            assert sorted(at[0].tolist()) == sorted(ids[0].tolist())  # no expert changes places
            by_expert = dict(zip(at[0].tolist(), ww[0].tolist()))
            total += sign * sum(by_expert[i] * g for i, g in zip(ids[0].tolist(), dw[0].tolist()))
        assert abs(total / (2 * h) - float(d[0, e])) <= 4 * h * h + 4 * 100 * EPS32 / h


def test_gradient_of_repeated_and_wrong_ids():
    """An expert that occurs twice gets both terms; an id out of range is reported and left out."""
    E, k = 64, 4
    x = logits(3, E, "fp32", 6)
    r = router(E, k, "sigmoid", renormalize=False)
    ids = torch.tensor([[5, 5, 9, 5], [1, 64, 2, 3], [1 << 30, -1, -5, 0]], dtype=torch.int32, device=DEV)
    s = torch.sigmoid(x.double())
    w = s.gather(1, ids.long().clamp(0, E - 1)).float()
    dw = torch.arange(1.0, 13.0, device=DEV).view(3, 4)
    d = torch.full_like(x, 7.0)
    ft.ftmoe_route_tokens_backward(x, r, ids, w, dw, d)
    want = torch.zeros(3, E, dtype=torch.float64, device=DEV)
    for t, i, g in ((0, 5, 1 + 2 + 4), (0, 9, 3), (1, 1, 5), (1, 2, 7), (1, 3, 8), (2, 0, 12)):
        want[t, i] = g * s[t, i] * (1 - s[t, i])
    assert ((d.double() - want).abs() <= want.abs() * 32 * EPS32).all()
    assert ft.ftmoe_read_error_flags() == ft.ERR_EXPERT_ID_RANGE
    assert ft.ftmoe_read_error_flags() == 0


@pytest.mark.parametrize("T", [1, 2, 3, 15, 16, 17, 2500, 20001])
def test_gradients_of_any_number_of_tokens(T):
    """Whatever the number of tokens, each token's row is that of the token alone, and nothing behind the last is written."""
    x = logits(T, 64, "fp32", T)
    for renorm, score in ((False, "softmax"), (True, "sigmoid")):
        r = router(64, 4, score, renormalize=renorm)
        ids, w = route(x, r)
        ids[T // 2] = -1
        wide = torch.full((T + 20, 64), 7.0, device=DEV)
        ft.ftmoe_route_tokens_backward(x, r, ids, w, torch.ones_like(w).cumsum(1), wide[:T])
        assert (wide[T:] == 7.0).all() and (wide[T // 2] == 0).all()
        for t in {0, T // 3, T - 1}:
            alone = torch.empty(1, 64, device=DEV)
            ft.ftmoe_route_tokens_backward(x[t:t + 1], r, ids[t:t + 1], w[t:t + 1], torch.ones_like(w[:1]).cumsum(1), alone)
            assert torch.equal(alone[0], wide[t])
        want = exact_gradient(x, r, ids, torch.ones_like(w).cumsum(1))
        assert ((wide[:T].double() - want).abs() <= 4 * 4 * 200 * EPS32 + want.abs() * EPS32).all()


def test_gradient_of_masked_logits():
    """Experts of logits -inf and NaN have no gradient; rows without routes read no logits."""
    x = logits(4, 32, "fp32", 8)
    x[0, ::2], x[1, 3:], x[2], x[3, 4] = -math.inf, math.nan, math.nan, math.inf
    for score in ("softmax", "sigmoid"):
        for renorm in (False, True):
            r = router(32, 6, score, renormalize=renorm)
            ids, w = route(x, r)
            d = torch.full_like(x, 7.0)
            ft.ftmoe_route_tokens_backward(x, r, ids, w, torch.ones_like(w), d)
            assert torch.isfinite(d).all() and (d[0, ::2] == 0).all() and (d[1, 3:] == 0).all() and (d[2] == 0).all()


@pytest.mark.parametrize("value", [0.0, math.nan, math.inf, -math.inf, 3e38])
@pytest.mark.parametrize("E,k", [(64, 8), (256, 6), (600, 17)])
def test_logits_of_tokens_without_routes_make_no_difference(E, k, value):
    """Whatever such rows hold, every row has the same bits, those that share a warp with one too."""
    x = logits(1000, E, "fp32", E)
    for score in ("softmax", "sigmoid"):
        for renorm in (False, True):
            r = router(E, k, score, renormalize=renorm)
            ids, w = route(x, r)
            ids[1::3], ids[500:510] = -1, -1
            dw = torch.linspace(-1.0, 1.0, k, device=DEV).repeat(1000, 1)
            want, d = torch.full_like(x, 7.0), torch.full_like(x, 7.0)
            ft.ftmoe_route_tokens_backward(x, r, ids, w, dw, want)
            y = torch.where((ids < 0).all(1, keepdim=True), torch.full_like(x, value), x)
            ft.ftmoe_route_tokens_backward(y, r, ids, w, dw, d)
            assert torch.equal(d, want) and (d[1::3] == 0).all() and (d[500:510] == 0).all()


def test_zero_tokens():
    x, r = torch.empty(0, 64, device=DEV), router(64, 4)
    ids, w = route(x, r)
    ft.ftmoe_route_tokens_backward(x, r, ids, w, w.clone(), x.clone())


def test_rows_far_apart():
    """Rows 2^30 elements apart: offsets beyond 32 bits in elements and bytes."""
    T, E, ld = 5, 64, 1 << 30
    wide = torch.zeros((T - 1) * ld + E, dtype=torch.float16, device=DEV)
    x = torch.as_strided(wide, (T, E), (ld, 1))
    x.copy_(logits(T, E, "fp16", 40))
    dense = x.contiguous()
    for r, bias in ((router(E, 4), None), (router(E, 4, "sigmoid"), torch.linspace(-0.1, 0.1, E, device=DEV))):
        ids, w = route(x, r, bias)
        want, ww = route(dense, r, bias)
        assert torch.equal(ids, want) and torch.equal(w, ww)
        dwant = torch.empty_like(dense)
        ft.ftmoe_route_tokens_backward(dense, r, want, ww, torch.ones_like(ww), dwant)
        wide2 = torch.zeros((T - 1) * ld + E, dtype=torch.float16, device=DEV)
        d = torch.as_strided(wide2, (T, E), (ld, 1))
        ft.ftmoe_route_tokens_backward(x, r, ids, w, torch.ones_like(w), d)
        assert torch.equal(d, dwant)


def test_another_stream_and_a_replayed_graph():
    x, r = logits(65, 256, "fp32", 30), router(256, 6, "sigmoid", groups=8, group_topk=4, group_best=2)
    bias = torch.linspace(-0.2, 0.2, 256, device=DEV)
    want, ww = route(x, r, bias)
    dw = torch.ones_like(ww)
    dwant = torch.empty_like(x)
    ft.ftmoe_route_tokens_backward(x, r, want, ww, dw, dwant)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    ids, w, d = torch.zeros_like(want), torch.zeros_like(ww), torch.zeros_like(x)
    stream.wait_stream(torch.cuda.current_stream())
    ft.ftmoe_route_tokens(x, r, ids, w, bias=bias, stream=stream)
    ft.ftmoe_route_tokens_backward(x, r, ids, w, dw, d, stream=stream)
    stream.synchronize()
    assert torch.equal(ids, want) and torch.equal(w, ww) and torch.equal(d, dwant)
    graph = torch.cuda.CUDAGraph()
    live = torch.zeros_like(x)
    with torch.cuda.graph(graph):
        ft.ftmoe_route_tokens(live, r, ids, w, bias=bias)
        ft.ftmoe_route_tokens_backward(live, r, ids, w, dw, d)
    for t in (x, x.flip(0).contiguous()):
        live.copy_(t)
        graph.replay()
        a, b = route(t, r, bias)
        assert torch.equal(ids, a) and torch.equal(w, b)
