"""A training step of the routed expert FFN on libftmoe's 16-bit products.

    python examples/train_experts.py [--steps 20 --tokens 1024 --hidden 1024 --inter 512 --experts 16 --topk 4]

expert_ffn(x, route_weights, w_gateup, w_down, expert_ids) is a torch function with gradients of
x, the routing weights and both weight banks. Between the passes it keeps, per token, the input row
in MXFP8 and, per route, the gate/up row in MXFP8: 1 + 1/32 bytes an element instead of two, and
neither SiLU's output nor the down product's. The backward pass:

    dh       = input gradient of the down product for the routes' output gradient
    dgate/up, weight * h, dweight = SiLU-and-mul backward from the kept rows
    dw_down  = weight gradient from (output gradient, weight * h)
    dx       = input gradient of the gate/up product, summed over a token's routes
    dw_gateup = weight gradient from (dgate/up, the kept input rows)

Run as a program it fits a bank of experts to a random teacher's outputs and prints the loss.
"""
import argparse
import os
import sys

import torch
from torch.autograd.function import once_differentiable

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_quantized_moe_gb300 as ft  # noqa: E402


class _ExpertFFN(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, route_weights, w_gateup, w_down, expert_ids):
        """x [T, H] and the banks w_gateup [E, 2I, H], w_down [E, H, I] in bf16; route_weights
        fp32 [T, topk]; expert_ids int32 [T, topk], < 0 for an inactive route. Returns [T, H]."""
        # (rows and routes are handed on by address: dense)
        x, route_weights, expert_ids = x.contiguous(), route_weights.contiguous(), expert_ids.contiguous()
        T, H = x.shape
        E, inter = w_down.shape[0], w_down.shape[2]
        topk, dev = expert_ids.shape[1], x.device
        routes = T * topk
        i32 = dict(dtype=torch.int32, device=dev)
        counts, offsets = torch.empty(E, **i32), torch.empty(E + 1, **i32)
        dst2src, route2dst = torch.empty(routes, **i32), torch.empty(routes, **i32)
        ft.ftmoe_segment_routes(expert_ids, E, counts, offsets, dst2src, route2dst)
        active = offsets[E:]  # the number of grouped rows, on the device

        rows = torch.empty(routes, H, dtype=x.dtype, device=dev)
        ft.ftmoe_gather_rows_scales(x, None, dst2src, rows, None, n_dst_dev=active)
        gu = torch.empty(routes, 2 * inter, dtype=x.dtype, device=dev)
        ft.ftmoe_grouped_matmul(rows, offsets, w_gateup, gu)
        h = torch.empty(routes, inter, dtype=x.dtype, device=dev)
        gu_q = torch.empty(routes, 2 * inter, dtype=torch.uint8, device=dev)
        gu_s = torch.empty(routes, 2 * inter // 32, dtype=torch.uint8, device=dev)
        ft.ftmoe_silu_mul_save(gu, h, gu_q, gu_s, fmt=ft.FMT_MXFP8, rows_dev=active)
        y = torch.empty(routes, H, dtype=torch.float32, device=dev)
        ft.ftmoe_grouped_matmul(h, offsets, w_down, y)
        out = torch.empty_like(x)
        if T:  # (the other calls take no rows as nothing to do)
            ft.ftmoe_combine(y, expert_ids, route_weights, out, route2dst=route2dst)

        x_q, x_s, _ = ft.quantize_act(x, ft.FMT_MXFP8)
        ctx.save_for_backward(x_q, x_s, gu_q, gu_s, route_weights, w_gateup, w_down, expert_ids, offsets, dst2src,
                              route2dst)
        return out

    @staticmethod
    @once_differentiable  # (the kernels' results have no gradients of their own)
    def backward(ctx, dout):
        (x_q, x_s, gu_q, gu_s, route_weights, w_gateup, w_down, expert_ids, offsets, dst2src,
         route2dst) = ctx.saved_tensors
        dout = dout.contiguous()
        need_x, _, need_gateup, need_down, _ = ctx.needs_input_grad  # (a frozen bank has no gradient to compute)
        dx = dw_gateup = dw_down = None
        (T, H), (E, _, inter), dev = dout.shape, w_down.shape, dout.device
        routes, active = dst2src.shape[0], offsets[E:]
        grouped, used = route2dst.long().clamp(min=0), route2dst >= 0
        # the weight of each grouped row (inactive routes add nothing to row 0, whatever their weight)
        row_weights = torch.zeros(routes, device=dev).index_add_(0, grouped, route_weights.reshape(-1).where(used, 0.0))

        dy = torch.empty(routes, H, dtype=dout.dtype, device=dev)
        ft.ftmoe_gather_rows_scales(dout, None, dst2src, dy, None, n_dst_dev=active)
        dh = torch.empty(routes, inter, dtype=dout.dtype, device=dev)
        ft.ftmoe_grouped_matmul(dy, offsets, w_down, dh, input_grad=True)
        dgu = torch.empty(routes, 2 * inter, dtype=dout.dtype, device=dev)
        hw = torch.empty_like(dh) if need_down else None
        drow = torch.zeros(routes, device=dev)
        ft.ftmoe_silu_mul_backward(gu_q, gu_s, dh, dgu, hw=hw, row_weights=row_weights, dweights=drow,
                                   fmt=ft.FMT_MXFP8, rows_dev=active)
        if need_down:
            dw_down = torch.empty_like(w_down)
            ft.ftmoe_grouped_matmul_wgrad(dy, hw, offsets, dw_down)
        if need_x:
            dx_rows = torch.empty(routes, H, dtype=torch.float32, device=dev)
            ft.ftmoe_grouped_matmul(dgu, offsets, w_gateup, dx_rows, input_grad=True)
            dx = torch.empty_like(dout)
            if T:
                ft.ftmoe_combine(dx_rows, expert_ids, torch.ones_like(route_weights), dx, route2dst=route2dst)
        if need_gateup:
            rows_q = torch.empty(routes, H, dtype=torch.uint8, device=dev)
            rows_s = torch.empty(routes, H // 32, dtype=torch.uint8, device=dev)
            ft.ftmoe_gather_rows_scales(x_q, x_s, dst2src, rows_q, rows_s, n_dst_dev=active)
            dw_gateup = torch.empty_like(w_gateup)
            ft.ftmoe_grouped_matmul_wgrad_saved(dgu, rows_q, rows_s, offsets, dw_gateup)
        dweights = drow[grouped].where(used, 0.0).view_as(route_weights)
        return dx, dweights, dw_gateup, dw_down, None


def expert_ffn(x, route_weights, w_gateup, w_down, expert_ids):
    """The routed FFN's output [T, H] for x bf16 [T, H], route_weights fp32 [T, topk], the banks w_gateup
    bf16 [E, 2 I, H] and w_down bf16 [E, H, I], and expert_ids int32 [T, topk] (< 0: an inactive
    route); H and I multiples of 32. x, the weights and the ids may have any strides."""
    if w_down.dim() != 3 or x.dim() != 2 or expert_ids.dim() != 2:
        raise ValueError("expert_ffn takes x [T, H], banks of three axes and expert_ids [T, topk]")
    (T, H), (E, _, inter) = x.shape, w_down.shape
    for name, t, shape, dtype in (("x", x, (T, H), torch.bfloat16), ("w_gateup", w_gateup, (E, 2 * inter, H), torch.bfloat16),
                                  ("w_down", w_down, (E, H, inter), torch.bfloat16),
                                  ("expert_ids", expert_ids, (T, expert_ids.shape[1]), torch.int32),
                                  ("route_weights", route_weights, (T, expert_ids.shape[1]), torch.float32)):
        if tuple(t.shape) != shape or t.dtype != dtype:
            raise ValueError(f"{name} is {t.dtype} {tuple(t.shape)}, expected {dtype} {shape}")
        if t.device != w_down.device or not t.is_cuda:
            raise ValueError(f"{name} is on {t.device}: all operands have to be on one CUDA device")
    if H % 32 or inter % 32:
        raise ValueError(f"hidden size {H} and intermediate size {inter} have to be multiples of 32 (MXFP8 groups)")
    return _ExpertFFN.apply(x, route_weights, w_gateup, w_down, expert_ids)


def main():
    import synth
    parser = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    parser.add_argument("--steps", type=int, default=20)
    for name, default in (("tokens", 1024), ("hidden", 1024), ("inter", 512), ("experts", 16), ("topk", 4)):
        parser.add_argument("--" + name, type=int, default=default)
    args = parser.parse_args()
    T, H, inter, E, topk, dev = args.tokens, args.hidden, args.inter, args.experts, args.topk, "cuda"
    ids = synth.routes_fast(T, topk, E, 1, dev)
    logits = torch.zeros(T, topk, device=dev, requires_grad=True)

    def bank(n, k, tag):
        return torch.stack([synth.expert_weight_fp32(n, k, 7, e, tag, dev, std=0.05) for e in range(E)]).to(torch.bfloat16)
    teacher = bank(2 * inter, H, "teacher-gateup"), bank(H, inter, "teacher-down")
    w1, w2 = (w.float().requires_grad_() for w in (bank(2 * inter, H, "gateup"), bank(H, inter, "down")))
    optimizer = torch.optim.Adam([w1, w2, logits], lr=2e-3)
    x = synth.activations_bf16(T, H, 3, dev)
    target = expert_ffn(x, synth.routing_weights(T, topk, 5, dev), *teacher, ids).float()
    for step in range(args.steps):
        optimizer.zero_grad()
        out = expert_ffn(x, torch.softmax(logits, 1), w1.to(torch.bfloat16), w2.to(torch.bfloat16), ids)
        loss = (out.float() - target).square().mean()
        loss.backward()
        optimizer.step()
        print(f"step {step}: loss {loss.item():.6f}", flush=True)
    return loss.item()


if __name__ == "__main__":
    main()
