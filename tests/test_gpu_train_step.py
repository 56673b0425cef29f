"""The training step of the example: forward and gradients against torch's own in 64 bits."""
import pytest
import torch

import block_quantized_moe_gb300 as ft
import synth
from examples.train_experts import expert_ffn

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def reference(x, weights, w1, w2, ids):
    """The expert FFN of the active routes with torch operations in the inputs' type."""
    inter = w2.shape[2]
    out = torch.zeros_like(x)
    for e in range(w1.shape[0]):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        gu = x[t] @ w1[e].T
        g, u = gu[:, :inter], gu[:, inter:]
        out = out.index_add(0, t, (g * torch.sigmoid(g) * u) @ w2[e].T * weights[t, j, None])
    return out


@pytest.mark.parametrize("tokens,active", [(1, [3]), (37, None), (64, [k % 4 for k in range(64)]), (5, [0] * 5)])
def test_step_against_autograd(tokens, active):
    H, inter, E, topk = 256, 160, 6, 3
    if active is not None:
        active = [min(a, topk) for a in active]
    ids = synth.routes(tokens, topk, E, 11, active_per_token=active, device=DEV)
    x = synth.activations_bf16(tokens, H, 12, DEV)
    w = synth.routing_weights(tokens, topk, 13, DEV)
    w1 = torch.stack([synth.expert_weight_fp32(2 * inter, H, 14, e, "g", DEV, std=0.1) for e in range(E)]).to(torch.bfloat16)
    w2 = torch.stack([synth.expert_weight_fp32(H, inter, 14, e, "d", DEV, std=0.1) for e in range(E)]).to(torch.bfloat16)
    args = [t.detach().clone().requires_grad_() for t in (x, w, w1, w2)]
    out = expert_ffn(*args, ids)
    dout = synth.activations_bf16(tokens, H, 15, DEV)
    out.backward(dout)
    exact = [t.detach().double().requires_grad_() for t in (x, w, w1, w2)]
    ref = reference(*exact, ids)
    ref.backward(dout.double())
    # forward: 16-bit gate/up, h and output, each rounded by at most 2^-8, in the norm
    out, ref = out.detach(), ref.detach()
    assert float((out.double() - ref).norm()) <= 3 * 2.0 ** -8 * float(ref.norm()) + 1e-30
    # gradients: from values kept in e4m3, off by at most 2^-4 each (a group's saturating maximum
    # by 2^-3); the norm of the error of a sum of independent terms stays below 2^-4 of the result's
    for name, got, want in zip(("x", "weights", "w_gateup", "w_down"), args, exact):
        want = torch.zeros_like(want) if want.grad is None else want.grad
        err, norm = float((got.grad.double() - want).norm()), float(want.norm())
        assert err <= 2.0 ** -4 * norm + 1e-30, (name, err / max(norm, 1e-30))
    assert ft.ftmoe_read_error_flags() == 0


def test_example_trains():
    import sys

    from examples import train_experts
    argv, sys.argv = sys.argv, ["train_experts.py", "--steps", "1", "--tokens", "256"]
    try:
        first = train_experts.main()
        sys.argv[2] = "12"
        last = train_experts.main()
    finally:
        sys.argv = argv
    assert last < 0.8 * first
