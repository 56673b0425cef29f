"""What the binding of the routing, gradient-norm and AdamW entry points refuses before it calls the
library, and what it hands over. Runs without a GPU: the tensors say that they are on one, and the
library is a list of calls."""
import pytest
import torch

import block_quantized_moe_gb300 as ft
from test_train_binding import OnDevice, calls  # noqa: F401 - the fixture

T, E, K = 4, 8, 2
F32, I32 = torch.float32, torch.int32
ROUTE = dict(logits=((T, E), F32), expert_ids=((T, K), I32), weights=((T, K), F32))
OPERANDS = {"ftmoe_route_tokens": {**ROUTE, "bias": ((E,), F32), "tokens_dev": ((1,), I32)},
            "ftmoe_route_tokens_backward": {**ROUTE, "dweights": ((T, K), F32), "dlogits": ((T, E), F32)}}
EACH = [(f, name) for f, operands in OPERANDS.items() for name in operands]
ANY_TYPE = ("logits", "dlogits")  # of the three


def dev(*shape, dtype=F32, device=0):
    return OnDevice(torch.zeros(shape, dtype=dtype), device)


def operands(f):
    return {"router": ft.make_router(E, K), **{name: dev(*s, dtype=d) for name, (s, d) in OPERANDS[f].items()}}


def refused(calls, f, args, match):  # noqa: F811
    with pytest.raises(ValueError, match=match):
        getattr(ft, f)(**args)
    assert not calls


@pytest.mark.parametrize("f", OPERANDS)
def test_good_operands_reach_the_library(calls, f):  # noqa: F811
    args = operands(f)
    getattr(ft, f)(**args)
    (name, got), = calls
    assert name == f and got[-1] == 77  # the device's current stream
    for operand, t in args.items():
        if operand != "router":
            assert t.data_ptr() in [g for g in got if isinstance(g, int)], operand


@pytest.mark.parametrize("f,name", EACH)
def test_operands_that_are_refused(calls, f, name):  # noqa: F811
    shape, dtype = OPERANDS[f][name]
    off = dev(*shape, dtype=dtype, device=-1)
    refused(calls, f, {**operands(f), name: off}, f"^{name} is not on a CUDA device")
    if not ft._one_device:
        refused(calls, f, {**operands(f), name: dev(*shape, dtype=dtype, device=1)}, "cuda:1, ")
    wrong = (0,) if name == "tokens_dev" else shape[:-1] + (shape[-1] + 1,)
    refused(calls, f, {**operands(f), name: dev(*wrong, dtype=dtype)}, "has shape")
    refused(calls, f, {**operands(f), name: dev(*shape, dtype=torch.int64)}, "expected|is not one of")
    if name != "tokens_dev":
        wide = torch.zeros(*shape[:-1], 2 * shape[-1], dtype=dtype)[..., ::2]
        refused(calls, f, {**operands(f), name: OnDevice(wide)}, "not contiguous")


def test_logits_of_any_row_stride_and_type(calls):  # noqa: F811
    args = operands("ftmoe_route_tokens")
    args["logits"] = OnDevice(torch.zeros(T, 3 * E, dtype=torch.bfloat16)[:, E:2 * E])
    ft.ftmoe_route_tokens(**args)
    assert calls[0][1][1:4] == (ft.OUT_BF16, T, 3 * E)


def adamw_operands(narrow=False, copies=True):
    sizes = (5, 64, 0)
    kinds = {"params": F32, "grads": torch.bfloat16, "m": torch.uint8 if narrow else F32, "v": torch.uint8 if narrow else F32}
    got = {k: [dev(n, dtype=d) for n in sizes] for k, d in kinds.items()}
    if narrow:
        got |= {k: [dev(-(-n // 32), dtype=torch.uint8) for n in sizes] for k in ("m_scales", "v_scales")}
    if copies:
        got["copies"] = [dev(n, dtype=torch.float16) for n in sizes]
    return got


@pytest.mark.parametrize("narrow", [False, True])
def test_adamw_list(calls, narrow):  # noqa: F811
    args = adamw_operands(narrow)
    made = ft.make_adamw_list(**args)
    c = made.c_list
    assert (c.param_dtype, c.grad_dtype, c.copy_dtype, c.moments, c.count) == (ft.OUT_FP32, ft.OUT_BF16, ft.OUT_FP16, int(narrow), 3)
    for i in range(2):
        t = c.tensors[i]
        assert t.n == args["params"][i].numel() and t.grad == args["grads"][i].data_ptr() and t.copy == args["copies"][i].data_ptr()
        assert t.m_scales == (args["m_scales"][i].data_ptr() if narrow else None)
    ft.ftmoe_adamw_step(made, grad_scale=dev(1))
    assert calls[0][0] == "ftmoe_adamw_step" and calls[0][1][-1] == 77
    assert ft.make_adamw_list([], [], [], []).c_list.count == 0


def test_adamw_lists_that_are_refused(calls):  # noqa: F811
    good = adamw_operands(True)

    def bad(match, **kw):
        with pytest.raises(ValueError, match=match):
            ft.make_adamw_list(**{**good, **kw})
    bad("2 grads for 3 params", grads=good["grads"][:2])
    bad("belong together", m_scales=None)
    bad(r"m\[0\] is torch.uint8", m_scales=None, v_scales=None)
    bad(r"v_scales\[1\] has 1 elements, expected 2", v_scales=[dev(1, dtype=torch.uint8)] * 3)
    bad(r"grads\[1\] is torch.float32", grads=[good["grads"][0], dev(64), good["grads"][2]])
    bad(r"grads\[1\] has 63", grads=[good["grads"][0], dev(63, dtype=torch.bfloat16), good["grads"][2]])
    bad(r"copies\[0\] is torch.float32", copies=[dev(5), dev(64), dev(0)])
    bad(r"m\[0\] is torch.float8_e5m2", m=[dev(n, dtype=torch.float8_e5m2) for n in (5, 64, 0)])
    bad("is not on a CUDA device", params=[dev(5, device=-1), *good["params"][1:]])
    bad("not contiguous", params=[good["params"][0], OnDevice(torch.zeros(8, 16).T[:, ::2]), good["params"][2]])
    bad("is not one of", params=[dev(n, dtype=torch.int32) for n in (5, 64, 0)])
    bad("occurs twice", v=[good["v"][0], good["m"][1], good["v"][2]])
    bad("occurs twice", params=[good["params"][0]] * 3, **{k: [good[k][0]] * 3 for k in good if k != "params"})
    made = ft.make_adamw_list(**good)
    for kw in (dict(grad_scale=dev(2)), dict(grad_scale=dev(1, dtype=torch.float16)), dict(lr_dev=dev(1, device=-1)),
               dict(step_dev=dev(1, dtype=torch.int32))):
        with pytest.raises(ValueError):
            ft.ftmoe_adamw_step(made, **kw)
    assert not calls


def test_grad_lists(calls):  # noqa: F811
    made = ft.make_grad_list([dev(3, 4, dtype=torch.float16), dev(0, dtype=torch.float16)])
    assert made.c_list.dtype == ft.OUT_FP16 and made.c_list.grads[0].n == 12 and made.c_list.count == 2
    assert ft.make_grad_list([]).c_list.count == 0
    for wrong, match in (([dev(3), dev(3, dtype=torch.float16)], "is torch.float16"), ([dev(3, dtype=torch.int8)], "is not one of"),
                         ([dev(3, device=-1)], "not on a CUDA device"), ([OnDevice(torch.zeros(6)[::2])], "not contiguous")):
        with pytest.raises(ValueError, match=match):
            ft.make_grad_list(wrong)
    with pytest.raises(ValueError, match="result"):
        ft.ftmoe_grad_norm(made, dev(1), dev(64, dtype=torch.uint8))
    with pytest.raises(ValueError, match="workspace"):
        ft.ftmoe_grad_norm(made, dev(2), dev(64, dtype=torch.int32))
    assert not calls
    ft.ftmoe_grad_norm(made, dev(2), dev(64, dtype=torch.uint8))
    assert calls[0][1][4] == 64


def test_a_list_is_used_on_its_device(calls, monkeypatch):  # noqa: F811
    grads, tensors = ft.make_grad_list([dev(3)]), ft.make_adamw_list(**adamw_operands())
    monkeypatch.setattr(ft, "_current_device", lambda: 1)
    with pytest.raises(ValueError, match="current device is cuda:1"):
        ft.ftmoe_grad_norm(grads, dev(2), dev(64, dtype=torch.uint8))
    with pytest.raises(ValueError, match="current device is cuda:1"):
        ft.ftmoe_adamw_step(tensors)
    assert not calls
