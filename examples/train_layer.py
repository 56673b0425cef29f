"""Training steps of a whole routed layer: router, experts, gradient clipping and AdamW on libftmoe.

    python examples/train_layer.py [--steps 20 --tokens 1024 --hidden 1024 --inter 512 --experts 16 --topk 4 --moments 8bit]

route(x, w_router, router, bias) is a torch function that gives the routing weights (with gradients of x and of the
router's matrix) and the expert ids:

    logits  = x w_router^T, fp32 (a product grouped by expert with one expert)
    ids, weights = ftmoe_route_tokens(logits + the balance bias in the choice)
    dlogits = ftmoe_route_tokens_backward(dweights)
    dx      = dlogits w_router,  dw_router = dlogits^T x

Together with expert_ffn of train_experts.py that is the layer. After the backward pass the gradients' global
norm gives the factor that clips them, and one AdamW call steps the fp32 parameters of every tensor and writes the
16-bit copies that the products read; the moments are kept in fp32 or in 8 bits. After each step the balance
bias of an expert rises where it got fewer tokens than the mean and falls where it got more.

Run as a program it fits a layer to a random teacher's outputs and prints the loss, the norm and the largest load.
"""
import argparse
import os
import sys

import torch
from torch.autograd.function import once_differentiable

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_quantized_moe_gb300 as ft  # noqa: E402
from examples.train_experts import expert_ffn  # noqa: E402


class _Route(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w_router, router, bias):
        T, dev = x.shape[0], x.device
        all_rows = torch.arange(2, dtype=torch.int32, device=dev) * T  # the rows of the one "expert"
        logits = torch.empty(T, router.num_experts, device=dev)
        ft.ftmoe_grouped_matmul(x, all_rows, w_router[None], logits)
        ids = torch.empty(T, router.topk, dtype=torch.int32, device=dev)
        weights = torch.empty(T, router.topk, device=dev)
        ft.ftmoe_route_tokens(logits, router, ids, weights, bias=bias)
        ctx.save_for_backward(x, w_router, logits, ids, weights, all_rows)
        ctx.router = router
        ctx.mark_non_differentiable(ids)
        return weights, ids

    @staticmethod
    @once_differentiable
    def backward(ctx, dweights, _):
        x, w_router, logits, ids, weights, all_rows = ctx.saved_tensors
        dlogits = torch.empty(logits.shape, dtype=x.dtype, device=x.device)
        ft.ftmoe_route_tokens_backward(logits, ctx.router, ids, weights, dweights.contiguous(), dlogits)
        dx, dw = torch.empty_like(x), torch.empty_like(w_router)
        ft.ftmoe_grouped_matmul(dlogits, all_rows, w_router[None], dx, input_grad=True)
        ft.ftmoe_grouped_matmul_wgrad(dlogits, x, all_rows, dw[None])
        return dx, dw, None, None


def route(x, w_router, router, bias=None):
    """(weights fp32 [T, topk], expert ids int32 [T, topk]) of x [T, H] for the router's matrix w_router
    [E, H], both bf16; bias fp32 [E] is added to the scores for the choice."""
    if x.dim() != 2 or tuple(w_router.shape) != (router.num_experts, x.shape[1]):
        raise ValueError(f"x is {tuple(x.shape)}, w_router {tuple(w_router.shape)}: expected [T, H] and [{router.num_experts}, H]")
    if x.dtype != torch.bfloat16 or w_router.dtype != torch.bfloat16:
        raise ValueError(f"x is {x.dtype}, w_router {w_router.dtype}: expected bf16")
    return _Route.apply(x.contiguous(), w_router.contiguous(), router, bias)


def layer(x, w_router, w_gateup, w_down, router, bias=None):
    """The routed layer's output [T, H] and the expert ids."""
    weights, ids = route(x, w_router, router, bias)
    return expert_ffn(x, weights, w_gateup, w_down, ids), ids


class Optimizer:
    """AdamW over fp32 parameters with 16-bit working copies. step() takes the copies' .grad: the norm, the factor that clips
    them and the step are three launches, none of which waits for the host."""

    def __init__(self, params, eight_bit=False, lr=2e-3, weight_decay=0.01, max_norm=1.0):
        self.params = [p.detach().contiguous() for p in params]
        self.copies = [p.to(torch.bfloat16).requires_grad_() for p in self.params]
        dev = self.params[0].device
        self.state = {}
        for name, dtype in (("m", torch.float8_e4m3fn), ("v", torch.float8_e5m2)):
            if eight_bit:
                self.state[name] = [torch.zeros(p.shape, dtype=torch.uint8, device=dev).view(dtype) for p in self.params]
                self.state[name + "_scales"] = [torch.zeros(-(-p.numel() // 32), dtype=torch.uint8, device=dev) for p in self.params]
            else:
                self.state[name] = [torch.zeros_like(p) for p in self.params]
        self.options = dict(lr=lr, weight_decay=weight_decay)
        self.max_norm, self.t = max_norm, 0
        self.norm = torch.empty(2, device=dev)  # the norm, and the factor

    def step(self):
        self.t += 1
        grads = [c.grad.contiguous() for c in self.copies]
        listed = ft.make_grad_list(grads)
        workspace = torch.empty(ft.ftmoe_grad_norm_workspace_bytes(listed), dtype=torch.uint8, device=self.norm.device)
        ft.ftmoe_grad_norm(listed, self.norm, workspace, max_norm=self.max_norm)
        tensors = ft.make_adamw_list(self.params, grads, copies=[c.detach() for c in self.copies], **self.state)
        ft.ftmoe_adamw_step(tensors, step=self.t, grad_scale=self.norm[1:], seed=self.t, **self.options)
        for c in self.copies:
            c.grad = None


def main():
    import synth
    parser = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    parser.add_argument("--steps", type=int, default=20)
    parser.add_argument("--moments", choices=("fp32", "8bit"), default="8bit")
    for name, default in (("tokens", 1024), ("hidden", 1024), ("inter", 512), ("experts", 16), ("topk", 4)):
        parser.add_argument("--" + name, type=int, default=default)
    args = parser.parse_args()
    T, H, inter, E, topk, dev = args.tokens, args.hidden, args.inter, args.experts, args.topk, "cuda"
    router = ft.make_router(E, topk, score=ft.SCORE_SIGMOID)

    def bank(n, k, tag):
        return torch.stack([synth.expert_weight_fp32(n, k, 7, e, tag, dev, std=0.05) for e in range(E)])

    def matrices(tag):
        return synth.expert_weight_fp32(E, H, 7, 0, tag + "-router", dev, std=0.05), bank(2 * inter, H, tag + "-gateup"), bank(H, inter, tag + "-down")
    x = synth.activations_bf16(T, H, 3, dev)
    with torch.no_grad():
        target = layer(x, *(w.to(torch.bfloat16) for w in matrices("teacher")), router)[0].float()
    optimizer = Optimizer(matrices("student"), eight_bit=args.moments == "8bit")
    bias = torch.zeros(E, device=dev)
    for step in range(args.steps):
        out, ids = layer(x, *optimizer.copies, router, bias)
        loss = (out.float() - target).square().mean()
        loss.backward()
        optimizer.step()
        load = torch.bincount(ids.reshape(-1), minlength=E).float()
        bias += 1e-3 * torch.sign(load.mean() - load)
        print(f"step {step}: loss {loss.item():.6f}, norm {optimizer.norm[0].item():.4f}, largest load {load.max().item() / load.mean().item():.2f}",
              flush=True)
    return loss.item()


if __name__ == "__main__":
    main()
