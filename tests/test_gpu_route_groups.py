"""The groups of a routing whose values are large beside their sums: biases of both signs within a group, and sums beyond
fp32's range. Ids against the definition in 64 bits, exactly."""
import numpy as np
import pytest
import torch

import block_quantized_moe_gb300 as ft

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
LARGEST = float(np.finfo(np.float32).max)


def choice64(x, r, bias):
    """Ids of fp64 logits [T, E] (finite, or -inf for never) with fp64 biases [E] (finite)."""
    T, E = x.shape
    size, rows = E // r.groups, np.arange(T)[:, None]
    if r.score == ft.SCORE_SOFTMAX:
        top = x.max(1, keepdims=True)
        e = np.exp(x - np.where(top > -np.inf, top, 0.0))
        s = e / np.maximum(e.sum(1, keepdims=True), 1e-300)
    else:
        s = 1 / (1 + np.exp(-x))
    value = np.where(x > -np.inf, s + bias, -np.inf)
    top = -np.sort(-value.reshape(T, r.groups, size), axis=2)[:, :, :r.group_best]
    score = np.where(top[:, :, 0] > -np.inf, np.where(top > -np.inf, top, 0.0).sum(2), -np.inf)
    kept = np.zeros((T, r.groups), dtype=bool)
    kept[rows, np.argsort(-score, axis=1, kind="stable")[:, :r.group_topk]] = True
    value = np.where(np.repeat(kept, size, axis=1), value, -np.inf)
    ids = np.argsort(-value, axis=1, kind="stable")[:, :r.topk]
    return np.where(value[rows, ids] > -np.inf, ids, -1)


def check_ids(x, r, bias):
    T = x.shape[0]
    ids = torch.full((T, r.topk), -7, dtype=torch.int32, device=DEV)
    w = torch.full((T, r.topk), float("nan"), device=DEV)
    ft.ftmoe_route_tokens(x, r, ids, w, bias=bias)
    np.testing.assert_array_equal(ids.cpu().numpy(), choice64(x.double().cpu().numpy(), r, bias.double().cpu().numpy()))
    assert torch.equal(w > 0, ids >= 0) or not r.renormalize
    assert ft.ftmoe_read_error_flags() == 0


def logits(T, E, seed):
    return torch.randn(T, E, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV) * 1.5


# groups of whole lanes of two experts and of 32, groups of 20 that are not whole lanes, one expert a lane, sixteen
@pytest.mark.parametrize("E,groups,topk", [(64, 32, 8), (256, 8, 8), (160, 8, 6), (32, 16, 4), (512, 16, 10), (64, 32, 16)])
@pytest.mark.parametrize("score", [ft.SCORE_SOFTMAX, ft.SCORE_SIGMOID])
@pytest.mark.parametrize("large", [64.0, 1e4, 1e6])
def test_biases_that_cancel_within_a_group(E, groups, topk, score, large):
    """One expert of each group forced by a large bias, the others held back by the same: a group's score is near 0,
    the rounding of its values that of the bias."""
    size = E // groups
    bias = torch.full((E,), -large, device=DEV)
    bias[torch.arange(groups, device=DEV) * size + torch.arange(groups, device=DEV) % size] = large
    check_ids(logits(1 << 14, E, E), ft.make_router(E, topk, score=score, groups=groups, group_topk=groups // 2, group_best=2), bias)


@pytest.mark.parametrize("E,groups", [(64, 8), (160, 8)])
def test_a_group_of_large_biases_beside_others(E, groups):
    """One group whose values cancel, among groups of balance biases; one held back as a whole."""
    size = E // groups
    bias = torch.linspace(-0.1, 0.1, E, device=DEV)
    bias[size:2 * size:2], bias[size + 1:2 * size:2] = 3e4, -3e4
    bias[size], bias[size + 2:2 * size:2] = 3e4, -3e4
    bias[3 * size:4 * size] = -1e9
    for score in (ft.SCORE_SOFTMAX, ft.SCORE_SIGMOID):
        for keep in (1, 4, 7):
            check_ids(logits(1 << 13, E, E + keep), ft.make_router(E, 4, score=score, groups=groups, group_topk=keep, group_best=2), bias)


@pytest.mark.parametrize("E,groups", [(32, 4), (160, 8), (256, 8)])
def test_sums_above_fp32(E, groups):
    """Groups whose two best sum to more than fp32's largest number, and one just below it."""
    size = E // groups
    bias = torch.zeros(E, device=DEV)
    for g, (a, b) in ((1, (LARGEST, 1e38)), (2, (LARGEST, 2e38)), (3, (LARGEST * 0.5, LARGEST * 0.49))):
        bias[g * size], bias[g * size + 1] = a, b
    for score in (ft.SCORE_SOFTMAX, ft.SCORE_SIGMOID):
        for keep in (1, 2, 3):
            check_ids(logits(300, E, E), ft.make_router(E, 5, score=score, groups=groups, group_topk=keep, group_best=2), bias)


@pytest.mark.parametrize("E,groups", [(32, 4), (160, 8), (256, 8)])
@pytest.mark.parametrize("low", [-LARGEST, -1e38])
def test_sums_below_fp32(E, groups, low):
    """Groups masked by the type's lowest value, whose two best sum to less than fp32 holds, are still ahead of groups
    of which nothing can be chosen."""
    size = E // groups
    x, bias = logits(300, E, E), torch.full((E,), low, device=DEV)
    x[:100, 2 * size:3 * size] = -float("inf")  # nothing left
    x[100:200, :size] = -float("inf")
    x[200:250, size:] = -float("inf")
    x[250:260] = -float("inf")
    bias[:size] = 0.0
    if groups > 4:
        bias[5 * size:6 * size] = low / 2
    for score in (ft.SCORE_SOFTMAX, ft.SCORE_SIGMOID):
        for keep in (1, 2, 3):
            for topk in (4, min(32, keep * size)):
                r = ft.make_router(E, topk, score=score, groups=groups, group_topk=keep, group_best=2)
                check_ids(x, r, bias)
