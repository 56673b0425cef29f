"""What the binding of the training and 16-bit entry points refuses before it calls the library, and
what it hands over where nothing is wrong. Runs without a GPU: the tensors say that they are on one,
and the library is a list of calls."""
import pytest
import torch

import block_quantized_moe_gb300 as ft


class OnDevice:
    """A CPU tensor that says it is on cuda:`device`."""

    def __init__(self, t, device=0):
        self.t, self.device = t, device

    def __getattr__(self, name):
        return getattr(self.t, name)

    def get_device(self):
        return self.device

    @property
    def is_cuda(self):
        return self.device >= 0


# whether the process sees one device only, for what does not depend on it
@pytest.fixture(params=[False, True])
def calls(monkeypatch, request):
    made = []

    class Library:
        def __getattr__(self, name):
            return lambda *args: made.append((name, args)) or 0
    monkeypatch.setattr(ft, "lib", Library)
    monkeypatch.setattr(ft, "_one_device", request.param)
    monkeypatch.setattr(ft, "_current_device", lambda: 0)
    monkeypatch.setattr(ft, "_current_raw_stream", lambda device: 77 + device)
    return made


def dev(*shape, dtype=torch.bfloat16, device=0):
    return OnDevice(torch.zeros(shape, dtype=dtype), device)


E, N, K, R = 2, 16, 32, 4
SAVED = dict(q=(dict(shape=(R, 2 * K), dtype=torch.uint8)), scales=dict(shape=(R, 2), dtype=torch.uint8))
OPERANDS = {
    "ftmoe_grouped_matmul": dict(a=dict(shape=(R, K)), offsets=dict(shape=(E + 1,), dtype=torch.int32),
                                 w=dict(shape=(E, N, K)), out=dict(shape=(R, N))),
    "ftmoe_grouped_matmul_wgrad": dict(dy=dict(shape=(R, N)), x=dict(shape=(R, K)),
                                       offsets=dict(shape=(E + 1,), dtype=torch.int32), dw=dict(shape=(E, N, K))),
    "ftmoe_grouped_matmul_wgrad_saved": dict(dy=dict(shape=(R, N)), q=dict(shape=(R, K), dtype=torch.uint8),
                                             scales=dict(shape=(R, 1), dtype=torch.uint8),
                                             offsets=dict(shape=(E + 1,), dtype=torch.int32),
                                             dw=dict(shape=(E, N, K))),
    "ftmoe_silu_mul_save": dict(gu=dict(shape=(R, 2 * K)), h=dict(shape=(R, K)), **SAVED,
                                rows_dev=dict(shape=(1,), dtype=torch.int32)),
    "ftmoe_silu_mul_backward": dict(**SAVED, dh=dict(shape=(R, K)), dgu=dict(shape=(R, 2 * K)), hw=dict(shape=(R, K)),
                                    row_weights=dict(shape=(R,), dtype=torch.float32),
                                    dweights=dict(shape=(R,), dtype=torch.float32),
                                    rows_dev=dict(shape=(1,), dtype=torch.int32)),
}
EACH = [(f, name) for f, operands in OPERANDS.items() for name in operands]
# operands whose type is free: another one of the three is no mistake there
ANY_TYPE = {("ftmoe_grouped_matmul", "out"), ("ftmoe_grouped_matmul_wgrad", "dw"),
            ("ftmoe_grouped_matmul_wgrad_saved", "dw"), ("ftmoe_grouped_matmul_wgrad_saved", "dy"),
            ("ftmoe_silu_mul_save", "gu"), ("ftmoe_silu_mul_save", "h")}


def operands(f):
    return {name: dev(*v["shape"], dtype=v.get("dtype", torch.bfloat16)) for name, v in OPERANDS[f].items()}


def refused(calls, f, args, match):
    with pytest.raises(ValueError, match=match):
        getattr(ft, f)(**args)
    assert not calls


@pytest.mark.parametrize("f", OPERANDS)
def test_good_operands_reach_the_library(calls, f):
    args = operands(f)
    getattr(ft, f)(**args)
    (name, got), = calls
    assert name == f and got[-1] == 77  # the device's current stream
    flat = [g for g in got if isinstance(g, int)]
    for operand, t in args.items():
        if operand not in ("w", "dw") and not (f.endswith("_saved") and operand in ("q", "scales")):
            assert t.data_ptr() in flat, operand


@pytest.mark.parametrize("f,name", EACH)
def test_every_operand_is_on_the_device_of_the_call(calls, f, name):
    args = operands(f)
    args[name] = OnDevice(args[name].t, -1)
    refused(calls, f, args, f"^{name} is not on a CUDA device")
    if not ft._one_device:
        args[name] = OnDevice(args[name].t, 1)
        refused(calls, f, args, "cuda:1, ")


@pytest.mark.parametrize("f", OPERANDS)
def test_the_device_is_the_current_one(calls, f, monkeypatch):
    monkeypatch.setattr(ft, "_one_device", None)
    monkeypatch.setattr(torch.cuda, "device_count", lambda: 2)
    refused(calls, f, {name: OnDevice(t.t, 1) for name, t in operands(f).items()}, "the current device is cuda:0")


@pytest.mark.parametrize("f,name", EACH)
def test_every_operand_has_its_shape(calls, f, name):
    shape = OPERANDS[f][name]["shape"]
    dtype = OPERANDS[f][name].get("dtype", torch.bfloat16)
    wrong = [shape[:-1] + (shape[-1] - 1,)]
    if name == "rows_dev":
        wrong = [(0,)]
    elif len(shape) > 1:
        wrong.append((shape[0] - 1,) + shape[1:])
    for s in wrong:
        args = operands(f)
        args[name] = dev(*s, dtype=dtype)
        refused(calls, f, args, "has shape")


@pytest.mark.parametrize("f,name", EACH)
def test_every_operand_has_its_type(calls, f, name):
    v = OPERANDS[f][name]
    for dtype in (torch.int64, torch.float16):
        args = operands(f)
        args[name] = dev(*v["shape"], dtype=dtype)
        if dtype == torch.float16 and (f, name) in ANY_TYPE:
            continue
        refused(calls, f, args, "expected|is not one of")


@pytest.mark.parametrize("f,name", [e for e in EACH if e[1] != "rows_dev"])
def test_rows_are_contiguous(calls, f, name):
    v = OPERANDS[f][name]
    args = operands(f)
    wide = torch.zeros(*v["shape"][:-1], max(2, v["shape"][-1]) * 2, dtype=v.get("dtype", torch.bfloat16))
    t = wide[..., ::2][..., :v["shape"][-1]]
    if v["shape"][-1] == 1:
        t = torch.zeros(v["shape"][-1], 2 * v["shape"][0], dtype=t.dtype).T[::2]
    args[name] = OnDevice(t)
    refused(calls, f, args, "not contiguous")


def test_row_strides_and_single_rows_are_taken(calls):
    args = operands("ftmoe_grouped_matmul")
    args["a"] = OnDevice(torch.zeros(R, 2 * K, dtype=torch.bfloat16)[:, :K])
    args["w"] = OnDevice(torch.zeros(E, N, 2 * K, dtype=torch.bfloat16)[:, :, K:])
    ft.ftmoe_grouped_matmul(**args)
    assert calls[0][1][2] == 2 * K
    ft.ftmoe_silu_mul_save(**{**operands("ftmoe_silu_mul_save"), "rows_dev": dev(5, dtype=torch.int32)})
    ft.ftmoe_silu_mul_save(**{**operands("ftmoe_silu_mul_save"), "rows_dev": dev(dtype=torch.int32)})
    ft.ftmoe_silu_mul_save(**{**operands("ftmoe_silu_mul_save"), "rows_dev": None})
    assert len(calls) == 4


def test_one_device_is_asked_for_once(calls, monkeypatch):
    monkeypatch.setattr(ft, "_one_device", None)
    monkeypatch.setattr(torch.cuda, "device_count", lambda: 1)
    ft.ftmoe_grouped_matmul(**operands("ftmoe_grouped_matmul"))
    assert ft._one_device is True and len(calls) == 1


def test_banks_of_matrices(calls):
    assert ft.make_matrix_bank(dev(E, N, K)).ld == K
    assert ft.make_matrix_bank(dev(E, N, K, device=1)).n == N  # no launch: any CUDA device
    for t in (dev(E, N, K, device=-1), OnDevice(torch.zeros(E, K, N, dtype=torch.bfloat16).transpose(1, 2)),
              dev(E, N, K, dtype=torch.int64)):
        with pytest.raises(ValueError):
            ft.make_matrix_bank(t)


def test_counts_and_bounds_off_their_alignment_are_refused():
    """The C entries answer an offsets or rows_dev address off 4 bytes with an error, on the host."""
    import ctypes

    from block_quantized_moe_gb300 import build_lib
    build_lib.build()
    P, bad = ctypes.c_void_p, ft.FTMOE_INVALID_ARG
    bank = ctypes.byref(ft.MatrixBank(0, E, N, K, K, N * K, P(256)))
    act = ctypes.byref(ft.Act(ft.FMT_MXFP8, 0, R, K, P(256), P(256), None))
    lib = ft.lib()
    for off in (257, 258, 259):
        assert lib.ftmoe_grouped_matmul(P(256), R, K, P(off), bank, 0, P(256), N, 0, None) == bad
        assert lib.ftmoe_grouped_matmul_wgrad(P(256), N, P(256), K, R, 0, P(off), bank, 0, None) == bad
        assert lib.ftmoe_grouped_matmul_wgrad_saved(P(256), N, 0, act, P(off), bank, 0, None) == bad
        assert lib.ftmoe_silu_mul_save(P(256), 0, R, K, 2 * K, P(off), P(256), K, 0, ft.FMT_MXFP8, P(256), P(256),
                                       None) == bad
        assert lib.ftmoe_silu_mul_backward(P(256), P(256), ft.FMT_MXFP8, R, K, P(off), P(256), K, 0, None, P(256), 2 * K,
                                           None, 0, None, None) == bad
