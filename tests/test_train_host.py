"""Refusals of the training and 16-bit entry points: answered on the host, without a GPU."""
import ctypes

import pytest
import torch

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def ft():
    from block_quantized_moe_gb300 import build_lib
    build_lib.build()
    import block_quantized_moe_gb300 as ft
    ft.lib()
    return ft


def bank(ft, dtype=0, E=2, n=16, k=32, ld=32, es=512, w=256):
    return ft.MatrixBank(dtype, E, n, k, ld, es, P(w))


def test_product_refusals(ft):
    f = ft.lib().ftmoe_grouped_matmul

    def call(a=256, rows=4, ld_a=32, off=256, w=None, grad=0, out=256, ld_out=16, od=0):
        return f(P(a), rows, ld_a, P(off), ctypes.byref(w or bank(ft)), grad, P(out), ld_out, od, None)
    bad = ft.FTMOE_INVALID_ARG
    assert call(rows=0) == ft.FTMOE_OK                     # nothing to do
    assert call(rows=-1) == bad and call(rows=1 << 31) == bad
    assert call(ld_a=31) == bad and call(ld_out=15) == bad and call(ld_a=0) == bad
    assert call(a=None) == bad and call(off=None) == bad and call(out=None) == bad
    assert call(a=257) == bad and call(out=257) == bad and call(out=258, od=2) == bad
    assert call(od=3) == bad and call(grad=2) == bad
    assert call(grad=1, ld_a=15) == bad and call(grad=1, ld_a=16, ld_out=31) == bad
    for w in (bank(ft, dtype=2), bank(ft, dtype=5), bank(ft, E=0), bank(ft, n=0), bank(ft, k=-1), bank(ft, ld=31),
              bank(ft, es=511), bank(ft, w=None), bank(ft, w=257), bank(ft, es=1 << 62)):
        assert call(w=w) == bad
    assert f(P(256), 4, 32, P(256), None, 0, P(256), 16, 0, None) == bad


def test_weight_gradient_refusals(ft):
    f, g = ft.lib().ftmoe_grouped_matmul_wgrad, ft.lib().ftmoe_grouped_matmul_wgrad_saved
    bad = ft.FTMOE_INVALID_ARG

    def call(dy=256, ld_dy=16, x=256, ld_x=32, rows=4, dt=0, off=256, w=None, acc=0):
        return f(P(dy), ld_dy, P(x), ld_x, rows, dt, P(off), ctypes.byref(w or bank(ft)), acc, None)
    assert call(rows=-1) == bad and call(dt=2) == bad and call(acc=2) == bad and call(off=None) == bad
    assert call(dy=None) == bad and call(x=None) == bad and call(ld_dy=15) == bad and call(ld_x=31) == bad
    assert call(dy=257) == bad and call(x=257) == bad and call(w=bank(ft, dtype=2, w=258)) == bad
    assert call(w=bank(ft, dtype=3)) == bad and call(w=bank(ft, w=None)) == bad

    def saved(fmt=ft.FMT_MXFP8, rows=4, k=32, q=256, s=256, w=None, gs=None, dt=0):
        act = ft.Act(fmt, 0, rows, k, P(q), P(s), P(gs))
        return g(P(256), 16, dt, ctypes.byref(act), P(256), ctypes.byref(w or bank(ft)), 0, None)
    # an fp32 scale per group would be rounded, e2m1 rows are not taken
    assert saved(fmt=ft.FMT_FP8) == ft.FTMOE_UNSUPPORTED and saved(fmt=ft.FMT_NVFP4) == ft.FTMOE_UNSUPPORTED
    assert saved(fmt=9) == bad and saved(k=64) == bad and saved(q=None) == bad and saved(s=None) == bad
    assert saved(rows=-1) == bad and saved(gs=256) == bad and saved(dt=2) == bad
    assert saved(k=40, w=bank(ft, k=40, ld=40, es=640)) == bad
    assert g(P(256), 16, 0, None, P(256), ctypes.byref(bank(ft)), 0, None) == bad


def test_silu_refusals(ft):
    f, g = ft.lib().ftmoe_silu_mul_save, ft.lib().ftmoe_silu_mul_backward
    bad = ft.FTMOE_INVALID_ARG

    def save(gu=256, gd=0, rows=4, inter=64, ld=128, h=256, ld_h=64, hd=0, fmt=ft.FMT_MXFP8, q=256, s=256):
        return f(P(gu), gd, rows, inter, ld, None, P(h), ld_h, hd, fmt, P(q), P(s), None)
    assert save(rows=0) == ft.FTMOE_OK and save(fmt=ft.FMT_NVFP4) == ft.FTMOE_UNSUPPORTED
    for kw in (dict(gu=None), dict(h=None), dict(q=None), dict(s=None), dict(ld=127), dict(ld_h=63), dict(inter=0),
               dict(inter=40, ld=80), dict(gd=3), dict(hd=-1), dict(fmt=7), dict(rows=-2), dict(gu=257),
               dict(s=258, fmt=ft.FMT_FP8)):
        assert save(**kw) == bad, kw

    def back(q=256, s=256, fmt=ft.FMT_MXFP8, rows=4, inter=64, dh=256, ld_dh=64, dt=0, w=256, dgu=256, ld=128, hw=256,
             ld_hw=64, dw=256):
        return g(P(q), P(s), fmt, rows, inter, None, P(dh), ld_dh, dt, P(w), P(dgu), ld, P(hw), ld_hw, P(dw), None)
    assert back(rows=0) == ft.FTMOE_OK and back(fmt=ft.FMT_NVFP4) == ft.FTMOE_UNSUPPORTED
    for kw in (dict(q=None), dict(s=None), dict(dh=None), dict(dgu=None), dict(ld_dh=63), dict(ld=127), dict(ld_hw=63),
               dict(dt=4), dict(inter=33, ld_dh=64), dict(w=257), dict(dw=258), dict(hw=257), dict(fmt=-1)):
        assert back(**kw) == bad, kw


def test_binding_checks_shapes_types_and_devices(ft):
    w = torch.zeros(2, 16, 32, dtype=torch.bfloat16)
    off = torch.zeros(3, dtype=torch.int32)
    a, out = torch.zeros(4, 32, dtype=torch.bfloat16), torch.zeros(4, 16, dtype=torch.bfloat16)
    for args in ((a, off, w, out), (a[:, :16], off, w, out), (a.half(), off, w, out), (a, off[:2], w, out),
                 (a, off.long(), w, out), (a, off, w, out[:3]), (a, off, w.transpose(1, 2), out)):
        with pytest.raises(ValueError):
            ft.ftmoe_grouped_matmul(*args)
    with pytest.raises(ValueError):
        ft.ftmoe_grouped_matmul_wgrad(out, a[:2], off, w)
    q, s = torch.zeros(4, 128, dtype=torch.uint8), torch.zeros(4, 4, dtype=torch.uint8)
    h, gu = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(4, 128, dtype=torch.bfloat16)
    for kw in (dict(gu=gu), dict(gu=gu[:, :64]), dict(q=q[:, ::2]), dict(s=s[:, :2]), dict(h=h.int())):
        v = {"gu": gu, "h": h, "q": q, "s": s, **kw}
        with pytest.raises(ValueError):
            ft.ftmoe_silu_mul_save(v["gu"], v["h"], v["q"], v["s"])
    with pytest.raises(ValueError):
        ft.ftmoe_silu_mul_backward(q, s, h, gu, dweights=torch.zeros(4, dtype=torch.float16))
