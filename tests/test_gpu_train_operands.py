"""Operands of the training example's expert_ffn as a model hands them over."""
import pytest
import torch

import block_quantized_moe_gb300 as ft
import synth
from examples.train_experts import expert_ffn

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
T, H, INTER, E, TOPK = 37, 128, 96, 5, 3


def operands(seed=1, active=None):
    ids = synth.routes(T, TOPK, E, seed, active_per_token=active, device=DEV)
    banks = [torch.stack([synth.expert_weight_fp32(n, k, seed, e, tag, DEV, std=0.1) for e in range(E)]).to(torch.bfloat16)
             for n, k, tag in ((2 * INTER, H, "g"), (H, INTER, "d"))]
    return [synth.activations_bf16(T, H, seed + 1, DEV), synth.routing_weights(T, TOPK, seed + 2, DEV), *banks], ids


def step(args, ids, dout, needs=(True,) * 4):
    args = [t.detach().requires_grad_(n) for t, n in zip(args, needs)]
    out = expert_ffn(*args, ids)
    out.backward(dout)
    return out.detach(), [t.grad for t in args]


def wider(t):
    """The same values as columns of a tensor whose other columns hold something else."""
    w = torch.full((*t.shape[:-1], t.shape[-1] + 5), 7, dtype=t.dtype, device=DEV)
    w[..., 2:-3] = t
    return w[..., 2:-3]


@pytest.mark.parametrize("change", [wider, lambda t: t.T.contiguous().T, lambda t: wider(t.repeat_interleave(2, 0))[::2]])
def test_strides(change):
    """Column slices, transposed storage and every other row: the same bits as from dense operands."""
    args, ids = operands()
    dout = synth.activations_bf16(T, H, 9, DEV)
    want, grads = step(args, ids, dout)
    x, weights = change(args[0]), change(args[1])
    got, other = step([x, weights, *args[2:]], change(ids), change(dout))
    assert torch.equal(got, want)
    for a, b in zip(other, grads):
        assert torch.equal(a, b)
    assert ft.ftmoe_read_error_flags() == 0


def test_second_derivatives_are_refused():
    args, ids = operands()
    args = [t.detach().requires_grad_() for t in args]
    out = expert_ffn(*args, ids).float()
    dx, = torch.autograd.grad(out.square().sum(), args[0], create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        (dx.float().square().sum() + args[0].float().square().sum()).backward()


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_weights_of_inactive_routes_are_not_used(value):
    """What an inactive route's weight holds changes nothing, and its own gradient is zero; also where
    the first grouped row's is not finite."""
    args, ids = operands(active=[k % 4 for k in range(T)])
    inactive = ids < 0
    assert inactive.any() and not inactive.all()
    dout = synth.activations_bf16(T, H, 9, DEV)
    want, grads = step(args, ids, dout)
    weights = args[1].masked_fill(inactive, value)
    got, other = step([args[0], weights, *args[2:]], ids, dout)
    assert torch.equal(got, want)
    for a, b in zip(other, grads):
        assert torch.isfinite(a).all() and torch.equal(a, b)
    assert (other[1][inactive] == 0).all()
    first = int(torch.nonzero(ids == ids[ids >= 0].min())[0, 0])  # the token of the first grouped row
    dout[first] = value
    _, other = step([args[0], weights, *args[2:]], ids, dout)
    assert (other[1][inactive] == 0).all() and not torch.isfinite(other[1][first][~inactive[first]]).any()


@pytest.mark.parametrize("needs", [(True, False, False, False), (False, True, False, False), (False, False, True, False),
                                   (False, False, False, True), (True, True, False, False)])
def test_gradients_that_are_not_needed_are_not_computed(needs, monkeypatch):
    args, ids = operands()
    dout = synth.activations_bf16(T, H, 9, DEV)
    _, want = step(args, ids, dout)
    made = []
    for name in ("ftmoe_grouped_matmul_wgrad", "ftmoe_grouped_matmul_wgrad_saved"):
        def call(*a, _f=getattr(ft, name), _name=name, **kw):
            made.append(_name)
            return _f(*a, **kw)
        monkeypatch.setattr(ft, name, call)
    _, got = step(args, ids, dout, needs)
    for need, a, b in zip(needs, got, want):
        assert torch.equal(a, b) if need else a is None
    assert made == ["ftmoe_grouped_matmul_wgrad"] * needs[3] + ["ftmoe_grouped_matmul_wgrad_saved"] * needs[2]


def test_no_tokens():
    args, ids = operands()
    got, grads = step([args[0][:0], args[1][:0], *args[2:]], ids[:0], args[0][:0])
    assert got.shape == (0, H)
    for g, a in zip(grads, [args[0][:0], args[1][:0], *args[2:]]):
        assert g.shape == a.shape and (g == 0).all()
    assert ft.ftmoe_read_error_flags() == 0
