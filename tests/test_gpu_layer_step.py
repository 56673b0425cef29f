"""The operators around the experts' products together: a training step of a routed layer, and the router in front of
the fused forward."""
import math

import pytest
import torch

import block_quantized_moe_gb300 as ft
import synth
from examples.train_experts import expert_ffn
from examples.train_layer import Optimizer, layer, route

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def parameters(E, H, inter, std=0.1):
    return [torch.randn(shape, generator=torch.Generator(device=DEV).manual_seed(5 + i), device=DEV) * std
            for i, shape in enumerate(((E, H), (E, 2 * inter, H), (E, H, inter)))]


def plain_weights(x, w_router, ids, score, scale):
    """The routing weights of given expert ids, with torch operations in the inputs' type."""
    logits = x @ w_router.T
    s = torch.softmax(logits, 1) if score == ft.SCORE_SOFTMAX else torch.sigmoid(logits)
    w = s.gather(1, ids.long())
    return scale * w / w.sum(1, keepdim=True)


def plain_experts(x, w, w1, w2, ids):
    out, inter = torch.zeros_like(x), w2.shape[2]
    for e in range(w1.shape[0]):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        gu = x[t] @ w1[e].T
        g, u = gu[:, :inter], gu[:, inter:]
        out = out.index_add(0, t, (g * torch.sigmoid(g) * u) @ w2[e].T * w[t, j, None])
    return out


@pytest.mark.parametrize("score", [ft.SCORE_SOFTMAX, ft.SCORE_SIGMOID])
@pytest.mark.parametrize("tokens", [1, 33, 257])
def test_layer_gradients(tokens, score):
    E, H, inter, topk = 8, 256, 160, 3
    x = synth.activations_bf16(tokens, H, 12, DEV)
    ws = [w.to(torch.bfloat16) for w in parameters(E, H, inter)]
    router = ft.make_router(E, topk, score=score, scale=2.5)
    args = [t.detach().clone().requires_grad_() for t in (x, *ws)]
    weights, ids = route(args[0], args[1], router, torch.linspace(-0.1, 0.1, E, device=DEV))
    weights.retain_grad()
    out = expert_ffn(args[0], weights, args[2], args[3], ids)
    with torch.no_grad():
        assert torch.equal(layer(*args, router, torch.linspace(-0.1, 0.1, E, device=DEV))[0], out)
    dout = synth.activations_bf16(tokens, H, 15, DEV)
    out.backward(dout)
    # The experts' part and the router's apart. dweights are sums over the intermediate columns of terms that are off by up to
    # 2^-4 each (values kept in e4m3), and the router's gradient takes differences of them, r_i - w_i R / c: sums and differences
    # may be far smaller than their terms, so their relative errors have no bound by themselves, and the
    # router's part is held to the formula for the dweights that it got.
    x1, x2, w_router, w1, w2 = (t.detach().double().requires_grad_() for t in (x, x, *ws))
    w_given = plain_weights(x2, w_router, ids, score, 2.5)
    w_leaf = w_given.detach().requires_grad_()
    ref = plain_experts(x1, w_leaf, w1, w2, ids)
    ref.backward(dout.double())
    w_given.backward(weights.grad.double())
    # as the experts' own step: three 16-bit roundings in the output, values kept in e4m3 in the gradients; the
    # router's gradients: dlogits, the result and (x) the sum of the two parts rounded to bf16
    assert float((out.detach().double() - ref.detach()).norm()) <= 3 * 2.0 ** -8 * float(ref.detach().norm())
    rounding = 2.1 * 2.0 ** -8
    for name, got, want, limit in (("router", args[1].grad, w_router.grad, rounding * float(w_router.grad.norm())),
                                   ("gateup", args[2].grad, w1.grad, 2.0 ** -4 * float(w1.grad.norm())),
                                   ("down", args[3].grad, w2.grad, 2.0 ** -4 * float(w2.grad.norm())),
                                   ("x", args[0].grad, x1.grad + x2.grad, 2.0 ** -4 * float(x1.grad.norm()) + 2 * rounding * float(x2.grad.norm()))):
        err = float((got.double() - want).norm())
        assert err <= limit, (name, err, limit)
    assert ft.ftmoe_read_error_flags() == 0


def test_route_against_the_formula_alone():
    """The router's product, choice and gradients by themselves: 16-bit operands, a 16-bit dlogits."""
    T, E, H, topk = 100, 16, 128, 4
    x, w = synth.activations_bf16(T, H, 2, DEV).requires_grad_(), parameters(E, H, 8)[0].to(torch.bfloat16).requires_grad_()
    weights, ids = route(x, w, ft.make_router(E, topk, score=ft.SCORE_SIGMOID))
    dw = torch.randn(T, topk, device=DEV)
    weights.backward(dw)
    x64, w64 = x.detach().double().requires_grad_(), w.detach().double().requires_grad_()
    s = torch.sigmoid(x64 @ w64.T).gather(1, ids.long())
    ref = s / s.sum(1, keepdim=True)
    ref.backward(dw.double())
    # logits of 128 products in fp32; the weights' logarithms are off by what the logits are, 128 half steps of their largest term
    limit = 128 * 2.0 ** -24 * float((x64.abs() @ w64.abs().T).detach().max())
    assert float((weights.detach().double() - ref.detach()).abs().max()) <= limit
    for got, want in ((x.grad, x64.grad), (w.grad, w64.grad)):  # dlogits and the result rounded to bf16
        assert float((got.double() - want).norm()) <= 2.1 * 2.0 ** -8 * float(want.norm())


@pytest.mark.parametrize("eight_bit", [False, True])
def test_step_of_the_layer(eight_bit):
    """Two steps: the norm and the clipped update against the formulas in 64 bits, the copies the
    parameters' rounding."""
    E, H, inter, topk, T = 8, 256, 160, 3, 200
    optimizer = Optimizer(parameters(E, H, inter), eight_bit, lr=0.01, weight_decay=0.1, max_norm=0.5)
    router = ft.make_router(E, topk)
    x = synth.activations_bf16(T, H, 12, DEV)
    moments = [(torch.zeros_like(p, dtype=torch.float64), torch.zeros_like(p, dtype=torch.float64)) for p in optimizer.params]
    for t in (1, 2):
        out, _ = layer(x, *optimizer.copies, router)
        out.float().square().sum().backward()
        grads = [c.grad.double() for c in optimizer.copies]
        before = [p.double() for p in optimizer.params]
        optimizer.step()
        norm = math.sqrt(sum(float(g.square().sum()) for g in grads))
        assert norm > 0.5 and abs(float(optimizer.norm[0]) - norm) <= 1e-6 * norm
        for i, (g, p) in enumerate(zip(grads, before)):
            g = g * (0.5 / (norm + 1e-6))
            m, v = moments[i]
            terms = 0.9 * m.abs() + 0.1 * g.abs()
            m.mul_(0.9).add_(0.1 * g)
            v.mul_(0.999).add_(0.001 * g * g)
            rate = 0.01 / (1 - 0.9 ** t) / ((v / (1 - 0.999 ** t)).sqrt() + 1e-8)
            u = rate * m
            want = p - 0.01 * 0.1 * p - u
            got = optimizer.params[i].double()
            # fp32: the update's 32 half steps and the factor's 9; m is a sum of two terms, each off by a few half steps of
            # its own, which may cancel: the half steps are those of the terms. 8 bits: in the second step the kept m and v are off
            # by up to a step (1/8 and 1/4 of their value, more below the normal range), so the update's size only is held to
            if not eight_bit or t == 1:
                assert ((got - want).abs() <= 64 * 2.0 ** -24 * (rate * terms + 0.001 * p.abs()) + 2.0 ** -23 * p.abs()).all()
            else:
                assert float((got - want).norm()) <= 0.25 * float(u.norm())
            assert torch.equal(optimizer.copies[i].detach(), optimizer.params[i].to(torch.bfloat16))
            if eight_bit:  # go on from what is kept
                for k, kind in enumerate(("m", "v")):
                    scales = optimizer.state[kind + "_scales"][i].double().sub(127).exp2().repeat_interleave(32)
                    moments[i][k].copy_((optimizer.state[kind][i].double().reshape(-1) * scales).view_as(moments[i][k]))


def test_router_in_front_of_the_fused_forward():
    """A padded batch, captured: the tokens behind the count get zeros, the others what the forward gives alone."""
    T, H, inter, E, topk = 8, 512, 256, 8, 3
    wg = torch.stack([synth.expert_weight_fp32(2 * inter, H, 3, e, "g", DEV) for e in range(E)])
    wd = torch.stack([synth.expert_weight_fp32(H, inter, 3, e, "d", DEV) for e in range(E)])
    kept = [ft.quantize_weights(wg), ft.quantize_weights(wd)]
    banks = [ft.make_bank(q, s) for q, s, _ in kept]
    x = synth.activations_bf16(T, H, 1, DEV)
    w_router = torch.randn(1, E, H, generator=torch.Generator(device=DEV).manual_seed(1), device=DEV).to(torch.bfloat16)
    router, shape = ft.make_router(E, topk), ft.moe_shape(T, H, inter, topk, E)
    ws = torch.empty(ft.ftmoe_forward_workspace_bytes(shape), dtype=torch.uint8, device=DEV)
    offsets, count = torch.tensor([0, T], dtype=torch.int32, device=DEV), torch.full((1,), T, dtype=torch.int32, device=DEV)
    logits, out = torch.empty(T, E, device=DEV), torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
    ids, weights = torch.empty(T, topk, dtype=torch.int32, device=DEV), torch.empty(T, topk, device=DEV)

    def step():
        ft.ftmoe_grouped_matmul(x, offsets, w_router, logits)
        ft.ftmoe_route_tokens(logits, router, ids, weights, tokens_dev=count)
        ft.ftmoe_moe_forward(shape, x, ids, weights, *banks, out, ws)
    step()
    torch.cuda.synchronize()
    whole = out.clone()
    assert (ids >= 0).all() and whole.abs().sum() > 0
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for n in (5, 0, T):
        count.fill_(n)
        out.fill_(7.0)
        graph.replay()
        assert torch.equal(out[:n], whole[:n]) and (out[n:] == 0).all() and (ids[n:] == -1).all()
    assert ft.ftmoe_read_error_flags() == 0


def test_calls_from_several_threads():
    """Four threads with streams and tensors of their own, calling at once: what each gets is what it gets alone."""
    import threading
    E, topk, T, n = 256, 6, 700, 50_000
    router = ft.make_router(E, topk, score=ft.SCORE_SIGMOID, groups=8, group_topk=4, group_best=2)

    def work(seed, stream):
        gen = torch.Generator(device=DEV).manual_seed(seed)
        logits, bias = torch.randn(T, E, generator=gen, device=DEV), torch.randn(E, generator=gen, device=DEV) * 0.1
        ids, weights = torch.empty(T, topk, dtype=torch.int32, device=DEV), torch.empty(T, topk, device=DEV)
        dlogits, p = torch.empty(T, E, device=DEV), torch.randn(n, generator=gen, device=DEV)
        m, v = (torch.zeros(n, dtype=torch.uint8, device=DEV) for _ in range(2))
        ms, vs = (torch.zeros(-(-n // 32), dtype=torch.uint8, device=DEV) for _ in range(2))
        g = dlogits.view(-1)[:n]
        grads, tensors = ft.make_grad_list([g]), ft.make_adamw_list([p], [g], [m], [v], [ms], [vs])
        norm, ws = torch.empty(2, device=DEV), torch.empty(ft.ftmoe_grad_norm_workspace_bytes(grads), dtype=torch.uint8, device=DEV)
        torch.cuda.synchronize()
        for t in range(1, 31):
            ft.ftmoe_route_tokens(logits, router, ids, weights, bias=bias, stream=stream)
            ft.ftmoe_route_tokens_backward(logits, router, ids, weights, weights, dlogits, stream=stream)
            ft.ftmoe_grad_norm(grads, norm, ws, max_norm=0.1, stream=stream)
            ft.ftmoe_adamw_step(tensors, step=t, seed=seed, grad_scale=norm[1:], stream=stream)
        stream.synchronize()
        return ids, weights, dlogits, norm, p, m, v, ms, vs

    streams = [torch.cuda.Stream() for _ in range(4)]
    alone = [work(seed, streams[0]) for seed in range(4)]
    got = [None] * 4

    def run(i):
        got[i] = work(i, streams[i])
    threads = [threading.Thread(target=run, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for a, b in zip(alone, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("moments", ["fp32", "8bit"])
def test_example_runs(moments, monkeypatch):
    import sys

    from examples import train_layer
    monkeypatch.setattr(sys, "argv", ["train_layer.py", "--steps", "3", "--tokens", "200", "--hidden", "256", "--inter", "96",
                                      "--moments", moments])
    assert math.isfinite(train_layer.main())
