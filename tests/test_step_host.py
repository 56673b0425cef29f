"""Refusals of the routing, gradient-norm and AdamW entry points: answered on the host, without a GPU.
The addresses are made up: a call that reached a kernel would fault on a GPU."""
import ctypes

import pytest

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def ft():
    from block_quantized_moe_gb300 import build_lib
    build_lib.build()
    import block_quantized_moe_gb300 as ft
    ft.lib()
    return ft


ROUTER = dict(num_experts=16, topk=2, score=0, renormalize=1, groups=4, group_topk=2, group_best=1, scale=1.0)
# router fields that are no router, and routers beyond what the kernels hold
BAD_ROUTERS = [dict(num_experts=0), dict(num_experts=-1), dict(topk=0), dict(topk=9), dict(score=2), dict(score=-1),
               dict(renormalize=2), dict(groups=0), dict(groups=3), dict(group_topk=0), dict(group_topk=5),
               dict(group_best=0), dict(group_best=3), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("inf")),
               dict(scale=float("nan")), dict(scale=1e-31), dict(scale=1e31)]
LARGE_ROUTERS = [dict(num_experts=1028), dict(num_experts=256, topk=33), dict(num_experts=128, groups=64, group_topk=8)]


def test_route_refusals(ft):
    f = ft.lib().ftmoe_route_tokens
    bad = ft.FTMOE_INVALID_ARG

    def call(x=256, dtype=2, tokens=4, ld=16, bias=256, dev=256, ids=256, w=256, **router):
        return f(P(x), dtype, tokens, ld, ft.Router(**{**ROUTER, **router}), P(bias), P(dev), P(ids), P(w), None)
    assert call(tokens=0) == ft.FTMOE_OK and call(tokens=0, x=None) == ft.FTMOE_OK
    for kw in [dict(x=None), dict(ids=None), dict(w=None), dict(dtype=3), dict(dtype=-1), dict(tokens=-1),
               dict(tokens=1 << 31), dict(ld=15), dict(ld=1 << 31), dict(x=258), dict(x=257, dtype=0), dict(bias=258),
               dict(dev=257), dict(ids=258), dict(w=257)] + BAD_ROUTERS:
        assert call(**kw) == bad, kw
    for kw in LARGE_ROUTERS:
        assert call(ld=2048, **kw) == ft.FTMOE_UNSUPPORTED, kw
    assert f(P(256), 2, 4, 16, None, None, None, P(256), P(256), None) == bad


def test_route_backward_refusals(ft):
    f = ft.lib().ftmoe_route_tokens_backward
    bad = ft.FTMOE_INVALID_ARG

    def call(x=256, dtype=2, tokens=4, ld=16, ids=256, w=256, dw=256, d=256, dd=2, ldd=16, **router):
        return f(P(x), dtype, tokens, ld, ft.Router(**{**ROUTER, **router}), P(ids), P(w), P(dw), P(d), dd, ldd, None)
    assert call(tokens=0) == ft.FTMOE_OK
    for kw in [dict(x=None), dict(ids=None), dict(w=None), dict(dw=None), dict(d=None), dict(dtype=3), dict(dd=3),
               dict(tokens=-1), dict(tokens=1 << 31), dict(ld=15), dict(ldd=15), dict(ldd=1 << 31), dict(x=258),
               dict(ids=257), dict(w=258), dict(dw=258), dict(d=258), dict(d=257, dd=0)] + BAD_ROUTERS:
        assert call(**kw) == bad, kw
    for kw in LARGE_ROUTERS:
        assert call(ld=2048, ldd=2048, **kw) == ft.FTMOE_UNSUPPORTED, kw


def grad_list(ft, entries, dtype=2, count=None):
    a = (ft.Grad * max(1, len(entries)))(*[ft.Grad(n, p) for n, p in entries])
    return ft.GradList(dtype, len(entries) if count is None else count, a)


def test_grad_norm_refusals(ft):
    f, size = ft.lib().ftmoe_grad_norm, ft.lib().ftmoe_grad_norm_workspace_bytes
    bad = ft.FTMOE_INVALID_ARG
    good = grad_list(ft, [(8, 256), (0, None)])
    need = size(good)
    assert need > 0 and need % 8 == 0 and size(grad_list(ft, [])) > 0
    for wrong in (grad_list(ft, [(8, None)]), grad_list(ft, [(-1, 256)]), grad_list(ft, [(8, 258)]),
                  grad_list(ft, [(8, 257)], dtype=0), grad_list(ft, [(8, 256)], dtype=3), grad_list(ft, [], count=-1),
                  grad_list(ft, [(1 << 42, 256)]), ft.GradList(2, 1, None)):
        assert size(wrong) == 0
        assert f(wrong, 1.0, 1.0, P(256), 1 << 30, P(256), None) == bad
    assert f(good, 1.0, 1.0, P(256), need - 1, P(256), None) == ft.FTMOE_WORKSPACE_TOO_SMALL
    for scale, most, ws, result in ((0.0, 1.0, 256, 256), (-1.0, 1.0, 256, 256), (float("inf"), 1.0, 256, 256),
                                    (float("nan"), 1.0, 256, 256), (1.0, 0.0, 256, 256), (1.0, float("nan"), 256, 256),
                                    (1.0, 1.0, None, 256), (1.0, 1.0, 260, 256), (1.0, 1.0, 256, None),
                                    (1.0, 1.0, 256, 258)):
        assert f(good, scale, most, P(ws), need, P(result), None) == bad
    assert f(None, 1.0, 1.0, P(256), need, P(256), None) == bad and size(None) == 0


def test_adamw_refusals(ft):
    f = ft.lib().ftmoe_adamw_step
    bad = ft.FTMOE_INVALID_ARG

    def call(moments=0, pd=2, gd=0, cd=-1, count=1, n=8, tensors=True, opt=None, **at):
        place = dict(param=256, grad=256, m=256, v=256, m_scales=256 if moments == 1 else None,
                     v_scales=256 if moments == 1 else None, copy=None if cd == -1 else 256)
        entries = (ft.AdamwTensor * 1)(ft.AdamwTensor(n, **{**place, **at}))
        o = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.1, step=1, seed=0)
        opt = ft.Adamw(**{**o, **(opt or {})})
        return f(ft.AdamwList(pd, gd, cd, moments, count, entries if tensors else None), ctypes.addressof(opt), None)
    # nothing to do: no launch
    assert call(count=0) == ft.FTMOE_OK and call(n=0) == ft.FTMOE_OK and call(n=0, param=None) == ft.FTMOE_OK
    assert call(count=0, tensors=False) == ft.FTMOE_OK
    for kw in (dict(moments=2), dict(moments=-1), dict(pd=3), dict(gd=-1), dict(cd=2), dict(cd=-2), dict(count=-1),
               dict(tensors=False), dict(n=-1), dict(n=1 << 42), dict(param=None), dict(grad=None), dict(m=None), dict(v=None),
               dict(moments=1, m_scales=None), dict(moments=1, v_scales=None), dict(m_scales=256), dict(v_scales=256),
               dict(copy=256), dict(cd=0, copy=None), dict(param=258), dict(param=257, pd=0), dict(grad=257),
               dict(grad=258, gd=2), dict(m=258), dict(v=258), dict(cd=1, copy=257)):
        assert call(**kw) == bad, kw
    nan, inf = float("nan"), float("inf")
    for opt in (dict(lr=nan), dict(lr=inf), dict(weight_decay=nan), dict(eps=0.0), dict(eps=-1.0), dict(eps=nan),
                dict(eps=inf), dict(beta1=1.0), dict(beta1=-0.1), dict(beta1=nan), dict(beta2=1.0), dict(beta2=nan),
                dict(step=0), dict(lr_dev=258), dict(step_dev=260), dict(grad_scale=257)):
        assert call(opt=opt) == bad, opt
    assert f(None, None, None) == bad


def test_adamw_constants_beyond_fp32_are_refused(ft):
    """The step is computed in fp32: a rate or decay that is infinite there is an error, not NaN parameters."""
    no_tensors = ft.AdamwList(2, 0, -1, 0, 0, None)
    for kw, want in ((dict(lr=3e38), ft.FTMOE_OK), (dict(weight_decay=-3e38), ft.FTMOE_OK), (dict(lr=1e39), ft.FTMOE_INVALID_ARG),
                     (dict(lr=-1e39), ft.FTMOE_INVALID_ARG), (dict(weight_decay=1e300), ft.FTMOE_INVALID_ARG)):
        opt = ft.Adamw(**{**dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.1, step=1, seed=0), **kw})
        assert ft.lib().ftmoe_adamw_step(no_tensors, ctypes.addressof(opt), None) == want, kw


def test_packed_options_are_the_structure(ft):
    packed = ft._pack_adamw(1.0, 2.0, 3.0, 4.0, 5.0, 6, 7, 8, 9, 10)
    o = ft.Adamw.from_buffer_copy(packed)
    assert len(packed) == ctypes.sizeof(ft.Adamw)
    assert (o.lr, o.beta1, o.beta2, o.eps, o.weight_decay, o.step, o.seed, o.lr_dev, o.step_dev, o.grad_scale) == \
        (1.0, 2.0, 3.0, 4.0, 5.0, 6, 7, 8, 9, 10)
