"""Python binding of libftmoe, the GB300 (sm_103a) block-quantized MoE FFN library.

Argument marshalling only: every function here forwards torch tensors' device
pointers, sizes and the current CUDA stream to the C entry point of the same name
declared in include/ftmoe.h. All arithmetic runs in the library's CUDA kernels;
there is no host or PyTorch fallback. If libftmoe.so is missing or cannot be
loaded, every call raises.
"""
import ctypes
import os
import struct

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libftmoe.so")

FTMOE_OK, FTMOE_INVALID_ARG, FTMOE_UNSUPPORTED, FTMOE_CUDA_ERROR, FTMOE_WORKSPACE_TOO_SMALL, FTMOE_CHECK_FAILED = range(6)
FMT_FP8, FMT_NVFP4, FMT_MXFP8 = 0, 1, 2
ROUTES_GROUPED, ROUTES_SLOTS = 0, 1
ERR_EXPERT_ID_RANGE, ERR_MAP_RANGE, ERR_WAIT_TIMEOUT = 0x1, 0x2, 0x4
OUT_BF16, OUT_FP16, OUT_FP32 = 0, 1, 2
_OUT_DTYPES = {torch.bfloat16: OUT_BF16, torch.float16: OUT_FP16, torch.float32: OUT_FP32}

c_i32, c_i64, c_ptr, c_size = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t


class FtmoeError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        super().__init__(f"{fn} failed: {status} ({_status_string(status)})")


class ExpertBank(ctypes.Structure):
    _fields_ = [("format", c_i32), ("num_experts", c_i32), ("n", c_i64), ("k", c_i64),
                ("q", c_ptr), ("scales", c_ptr), ("global_scale", c_ptr)]


class Act(ctypes.Structure):
    _fields_ = [("format", c_i32), ("reserved", c_i32), ("rows", c_i64), ("k", c_i64),
                ("q", c_ptr), ("scales", c_ptr), ("global_scale", c_ptr)]


class Routes(ctypes.Structure):
    _fields_ = [("kind", c_i32), ("topk", c_i32), ("tokens", c_i64), ("offsets", c_ptr), ("slots", c_ptr)]


class Tile(ctypes.Structure):
    _fields_ = [("tok_tile", c_i32), ("variant", c_i32), ("wblocks", c_i32), ("ctas", c_i32)]


class MoeShape(ctypes.Structure):
    _fields_ = [("tokens", c_i64), ("hidden", c_i64), ("inter", c_i64), ("topk", c_i32),
                ("num_experts", c_i32), ("format", c_i32), ("tok_tile", c_i32), ("path", c_i32),
                ("out_dtype", c_i32)]


class MoeArgs(ctypes.Structure):
    _fields_ = [("shape", MoeShape), ("x", c_ptr), ("ld_x", c_i64), ("expert_ids", c_ptr),
                ("route_weights", c_ptr), ("w_gateup", ExpertBank), ("w_down", ExpertBank),
                ("out", c_ptr), ("ld_out", c_i64)]


class MatrixBank(ctypes.Structure):
    _fields_ = [("dtype", c_i32), ("num_experts", c_i32), ("n", c_i64), ("k", c_i64), ("ld", c_i64),
                ("expert_stride", c_i64), ("w", c_ptr)]


_LAYOUT_FIELDS = ["x_q", "x_scales", "x_gscale", "counts", "offsets", "dst2src", "route2dst",
                  "rows_q", "rows_scales", "gateup", "gateup_bytes", "act_q", "act_q_bytes",
                  "act_scales", "act_scales_bytes", "act_gscale", "down", "down_bytes", "partials",
                  "partials_bytes", "counters", "counters_bytes", "total"]


class WorkspaceLayout(ctypes.Structure):
    _fields_ = [(n, c_size) for n in _LAYOUT_FIELDS]


# (name, restype, argtypes) of every exported entry point (a matrix bank is passed by address: a
# MatrixBank by reference, or the bytes of one)
_SIGNATURES = [
    ("ftmoe_status_string", ctypes.c_char_p, [c_i32]),
    ("ftmoe_pick_tile", c_i32, [c_i64, c_i32, ctypes.POINTER(Tile)]),
    ("ftmoe_quantize_act", c_i32, [c_ptr, c_i64, c_i64, c_i64, c_i32, c_ptr, c_ptr, c_ptr, c_ptr]),
    ("ftmoe_quantize_weights", c_i32, [c_ptr, c_i32, c_i64, c_i64, c_i32, c_ptr, c_ptr, c_ptr, c_ptr]),
    ("ftmoe_segment_routes", c_i32, [c_ptr, c_i64, c_i32, c_i32, c_ptr, c_ptr, c_ptr, c_ptr, c_ptr]),
    ("ftmoe_gather_rows_scales", c_i32, [c_ptr, c_ptr, c_i64, c_i64, c_i64, c_ptr, c_i64, c_ptr,
                                         c_ptr, c_ptr, c_ptr]),
    ("ftmoe_gather_quantize_act", c_i32, [c_ptr, c_i64, c_i64, c_i64, c_ptr, c_i64, c_ptr, c_i32, c_ptr, c_ptr,
                                          c_ptr]),
    ("ftmoe_grouped_gemm_gateup", c_i32, [ctypes.POINTER(Act), ctypes.POINTER(Routes),
                                          ctypes.POINTER(ExpertBank), c_ptr, c_i64,
                                          ctypes.POINTER(Tile), c_ptr]),
    ("ftmoe_grouped_gemm_gateup_silu", c_i32, [ctypes.POINTER(Act), ctypes.POINTER(Routes),
                                               ctypes.POINTER(ExpertBank), c_ptr, c_ptr,
                                               ctypes.POINTER(Tile), c_ptr]),
    ("ftmoe_silu_mul", c_i32, [c_ptr, c_i64, c_i64, c_i64, c_ptr, c_i32, c_ptr, c_ptr, c_ptr, c_ptr]),
    ("ftmoe_grouped_gemm_down", c_i32, [ctypes.POINTER(Act), ctypes.POINTER(Routes),
                                        ctypes.POINTER(ExpertBank), c_ptr, c_i64,
                                        ctypes.POINTER(Tile), c_ptr]),
    ("ftmoe_combine", c_i32, [c_ptr, c_i64, c_ptr, c_ptr, c_ptr, c_i64, c_i32, c_i64, c_i32, c_ptr, c_i64,
                              c_ptr]),
    ("ftmoe_forward_workspace_bytes", c_size, [ctypes.POINTER(MoeShape)]),
    ("ftmoe_forward_workspace_layout", c_i32, [ctypes.POINTER(MoeShape), ctypes.POINTER(WorkspaceLayout)]),
    ("ftmoe_moe_forward", c_i32, [ctypes.POINTER(MoeArgs), c_ptr, c_size, c_ptr]),
    ("ftmoe_moe_forward_noalloc", c_i32, [ctypes.POINTER(MoeArgs), c_ptr]),
    ("ftmoe_grouped_matmul", c_i32, [c_ptr, c_i64, c_i64, c_ptr, c_ptr, c_i32, c_ptr, c_i64,
                                     c_i32, c_ptr]),
    ("ftmoe_grouped_matmul_wgrad", c_i32, [c_ptr, c_i64, c_ptr, c_i64, c_i64, c_i32, c_ptr,
                                           c_ptr, c_i32, c_ptr]),
    ("ftmoe_grouped_matmul_wgrad_saved", c_i32, [c_ptr, c_i64, c_i32, ctypes.POINTER(Act), c_ptr,
                                                 c_ptr, c_i32, c_ptr]),
    ("ftmoe_silu_mul_save", c_i32, [c_ptr, c_i32, c_i64, c_i64, c_i64, c_ptr, c_ptr, c_i64, c_i32, c_i32, c_ptr,
                                    c_ptr, c_ptr]),
    ("ftmoe_silu_mul_backward", c_i32, [c_ptr, c_ptr, c_i32, c_i64, c_i64, c_ptr, c_ptr, c_i64, c_i32, c_ptr, c_ptr,
                                        c_i64, c_ptr, c_i64, c_ptr, c_ptr]),
    ("ftmoe_selftest_wait_timeout", c_i32, [ctypes.c_uint64, c_ptr, c_ptr]),
    ("ftmoe_selftest_shared_division", c_i32, [c_ptr, c_ptr]),
    ("ftmoe_expert_slots", c_i32, [c_ptr, c_i64, c_ptr, c_ptr, c_i32, c_ptr, c_i32, c_i64, c_i32, c_ptr, c_ptr,
                                   c_ptr]),
    ("ftmoe_read_error_flags", c_i32, [ctypes.POINTER(ctypes.c_uint32)]),
]

_lib_handle = None


def lib():
    """The loaded libftmoe (ctypes.CDLL). Raises if it was not built."""
    global _lib_handle
    if _lib_handle is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libftmoe.so not found at {LIB_PATH}; build it first "
                               "(python -c 'import __graft_entry__ as g; g.build()')")
        h = ctypes.CDLL(LIB_PATH)
        for name, res, args in _SIGNATURES:
            fn = getattr(h, name)
            fn.restype, fn.argtypes = res, args
        _lib_handle = h
    return _lib_handle


def _status_string(s):
    try:
        return lib().ftmoe_status_string(s).decode()
    except Exception:  # noqa: BLE001 - message only
        return "?"


def _check(fn, status):
    if status != FTMOE_OK:
        raise FtmoeError(fn, status)


def _p(t):
    """Device (or host) pointer of a tensor, None for None."""
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


# ---------------------------------------------------------------------------------
# entry points (same names as the C ABI)
# ---------------------------------------------------------------------------------

def ftmoe_pick_tile(routes, num_experts):
    t = Tile()
    _check("ftmoe_pick_tile", lib().ftmoe_pick_tile(int(routes), int(num_experts), ctypes.byref(t)))
    return t.tok_tile


def ftmoe_quantize_act(x, q, scales, global_scale=None, fmt=FMT_FP8, rows=None, k=None, stream=None):
    rows = x.shape[0] if rows is None else rows
    k = x.shape[1] if k is None else k
    ld = x.stride(0) if x.dim() == 2 else k
    _check("ftmoe_quantize_act", lib().ftmoe_quantize_act(
        _p(x), rows, k, ld, fmt, _p(q), _p(scales), _p(global_scale), _stream(stream)))


def ftmoe_quantize_weights(w, q, scales, global_scale=None, fmt=FMT_FP8, stream=None):
    E, n, k = w.shape
    _check("ftmoe_quantize_weights", lib().ftmoe_quantize_weights(
        _p(w), E, n, k, fmt, _p(q), _p(scales), _p(global_scale), _stream(stream)))


def ftmoe_segment_routes(expert_ids, num_experts, counts, offsets, dst2src, route2dst, stream=None):
    T, topk = expert_ids.shape
    _check("ftmoe_segment_routes", lib().ftmoe_segment_routes(
        _p(expert_ids), T, topk, num_experts, _p(counts), _p(offsets), _p(dst2src), _p(route2dst),
        _stream(stream)))


def ftmoe_gather_rows_scales(src, src_scales, dst2src, dst, dst_scales, n_dst=None, n_dst_dev=None,
                             stream=None):
    n_src = src.shape[0]
    row_bytes = src.shape[1] * src.element_size()
    scale_bytes = src_scales.shape[1] * src_scales.element_size() if src_scales is not None else 0
    n_dst = dst2src.shape[0] if n_dst is None else n_dst
    _check("ftmoe_gather_rows_scales", lib().ftmoe_gather_rows_scales(
        _p(src), _p(src_scales), n_src, row_bytes, scale_bytes, _p(dst2src), n_dst, _p(n_dst_dev),
        _p(dst), _p(dst_scales), _stream(stream)))


def ftmoe_gather_quantize_act(x, dst2src, q, scales, fmt=FMT_MXFP8, n_dst=None, n_dst_dev=None, stream=None):
    """bf16 rows x[dst2src[d]] quantized into q [n_dst, k] and scales (MXFP8: [n_dst, k/32])."""
    n_src, k = x.shape
    n_dst = dst2src.shape[0] if n_dst is None else n_dst
    _check("ftmoe_gather_quantize_act", lib().ftmoe_gather_quantize_act(
        _p(x), n_src, k, x.stride(0), _p(dst2src), n_dst, _p(n_dst_dev), fmt, _p(q), _p(scales), _stream(stream)))


def make_bank(q, scales, global_scale=None, fmt=FMT_FP8):
    """ExpertBank view of tensors q [E, n, k(/2)], scales, global_scale."""
    E, n, kk = q.shape
    k = 2 * kk if fmt == FMT_NVFP4 else kk
    return ExpertBank(fmt, E, n, k, _p(q), _p(scales), _p(global_scale))


def make_act(q, scales, global_scale=None, fmt=FMT_FP8):
    rows, kk = q.shape
    k = 2 * kk if fmt == FMT_NVFP4 else kk
    return Act(fmt, 0, rows, k, _p(q), _p(scales), _p(global_scale))


def grouped_routes(offsets):
    return Routes(ROUTES_GROUPED, 0, 0, _p(offsets), None)


def slot_routes(expert_ids):
    T, topk = expert_ids.shape
    return Routes(ROUTES_SLOTS, topk, T, None, _p(expert_ids))


def _tile(tok_tile=0, variant=0, wblocks=0, ctas=0):
    return Tile(tok_tile, variant, wblocks, ctas)


def ftmoe_grouped_gemm_gateup(act, routes, bank, out, tok_tile=0, variant=0, wblocks=0, ctas=0, stream=None):
    t = _tile(tok_tile, variant, wblocks, ctas)
    _check("ftmoe_grouped_gemm_gateup", lib().ftmoe_grouped_gemm_gateup(
        ctypes.byref(act), ctypes.byref(routes), ctypes.byref(bank), _p(out), out.stride(0),
        ctypes.byref(t), _stream(stream)))


def ftmoe_grouped_gemm_gateup_silu(act, routes, bank, q, scales, tok_tile=0, stream=None):
    t = _tile(tok_tile)
    _check("ftmoe_grouped_gemm_gateup_silu", lib().ftmoe_grouped_gemm_gateup_silu(
        ctypes.byref(act), ctypes.byref(routes), ctypes.byref(bank), _p(q), _p(scales),
        ctypes.byref(t), _stream(stream)))


def ftmoe_grouped_gemm_down(act, routes, bank, out, tok_tile=0, variant=0, wblocks=0, ctas=0, stream=None):
    t = _tile(tok_tile, variant, wblocks, ctas)
    _check("ftmoe_grouped_gemm_down", lib().ftmoe_grouped_gemm_down(
        ctypes.byref(act), ctypes.byref(routes), ctypes.byref(bank), _p(out), out.stride(0),
        ctypes.byref(t), _stream(stream)))


def ftmoe_silu_mul(gu, q, scales, global_scale=None, fmt=FMT_FP8, rows=None, rows_dev=None, stream=None):
    rows = gu.shape[0] if rows is None else rows
    inter = gu.shape[1] // 2
    _check("ftmoe_silu_mul", lib().ftmoe_silu_mul(
        _p(gu), rows, inter, gu.stride(0), _p(rows_dev), fmt, _p(q), _p(scales), _p(global_scale),
        _stream(stream)))


def out_dtype_code(out):
    """ftmoe_out_dtype of an output tensor (bf16, fp16 or fp32)."""
    if out.dtype not in _OUT_DTYPES:
        raise ValueError(f"output dtype {out.dtype} is not one of bf16, fp16, fp32")
    return _OUT_DTYPES[out.dtype]


def ftmoe_combine(y, expert_ids, weights, out, route2dst=None, stream=None):
    T, topk = expert_ids.shape
    H = out.shape[1]
    _check("ftmoe_combine", lib().ftmoe_combine(
        _p(y), y.stride(0), _p(route2dst), _p(expert_ids), _p(weights), T, topk, H, out_dtype_code(out),
        _p(out), out.stride(0), _stream(stream)))


def moe_shape(tokens, hidden, inter, topk, num_experts, fmt=FMT_FP8, tok_tile=0, path=0, out_dtype=OUT_BF16):
    return MoeShape(tokens, hidden, inter, topk, num_experts, fmt, tok_tile, path, out_dtype)


def _check_out(shape, out):
    if out_dtype_code(out) != shape.out_dtype:
        raise ValueError(f"output tensor is {out.dtype}, the shape says out_dtype {shape.out_dtype}")


def ftmoe_forward_workspace_bytes(shape):
    return int(lib().ftmoe_forward_workspace_bytes(ctypes.byref(shape)))


def ftmoe_forward_workspace_layout(shape):
    lay = WorkspaceLayout()
    _check("ftmoe_forward_workspace_layout",
           lib().ftmoe_forward_workspace_layout(ctypes.byref(shape), ctypes.byref(lay)))
    return {n: int(getattr(lay, n)) for n in _LAYOUT_FIELDS}


def ftmoe_moe_forward(shape, x, expert_ids, route_weights, bank_gateup, bank_down, out, workspace,
                      stream=None):
    _check_out(shape, out)
    args = MoeArgs(shape, _p(x), x.stride(0), _p(expert_ids), _p(route_weights), bank_gateup,
                   bank_down, _p(out), out.stride(0))
    _check("ftmoe_moe_forward", lib().ftmoe_moe_forward(
        ctypes.byref(args), _p(workspace), workspace.numel() * workspace.element_size(),
        _stream(stream)))


def ftmoe_moe_forward_noalloc(shape, x, expert_ids, route_weights, bank_gateup, bank_down, out, stream=None):
    """The fused forward with its intermediates in the library's own device array (no workspace)."""
    _check_out(shape, out)
    args = MoeArgs(shape, _p(x), x.stride(0), _p(expert_ids), _p(route_weights), bank_gateup,
                   bank_down, _p(out), out.stride(0))
    _check("ftmoe_moe_forward_noalloc", lib().ftmoe_moe_forward_noalloc(ctypes.byref(args), _stream(stream)))


def ftmoe_expert_slots(expert_ids, slot_expert, slot_usage, expert_slot, step, max_fetch, fetch_plan, n_fetch,
                       stream=None):
    """One step of the device-side expert-slot pool: expert_ids (int32, any shape) become slot
    ids in place; the pool state tensors are updated in place."""
    _check("ftmoe_expert_slots", lib().ftmoe_expert_slots(
        _p(expert_ids), expert_ids.numel(), _p(slot_expert), _p(slot_usage), slot_expert.numel(),
        _p(expert_slot), expert_slot.numel(), int(step), int(max_fetch), _p(fetch_plan), _p(n_fetch),
        _stream(stream)))


# The training entry points check what the C entry cannot see (devices, shapes, dtypes, contiguous
# rows) in as few tensor queries as that takes: at decode sizes the binding costs more than the
# kernel, and each query of a tensor costs about as much as a Python call. The kernels launch on
# the current device, so all tensors of a call have to be there; where the process sees one device,
# being on a CUDA device says that (asking every tensor for its index made a call 0.3 to 0.4 us longer).

_one_device = None  # whether the process sees one device only; None until a call has asked

def _dtype_code(t, name):
    code = _OUT_DTYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} dtype {t.dtype} is not one of bf16, fp16, fp32")
    return code


def _device_of(t, name):
    """Index of the device that a call runs on: the tensor's, which has to be the current one."""
    global _one_device
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} is not on a CUDA device")
    if _one_device is None:
        _one_device = torch.cuda.device_count() == 1
    if dev != _current_device():
        raise ValueError(f"{name} is on cuda:{dev}, the current device is cuda:{_current_device()}")
    return dev


def _refuse(t, name, shape, dtype, dev):
    """Says what is wrong with a tensor that failed a check."""
    if t.get_device() < 0:
        raise ValueError(f"{name} is not on a CUDA device")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on cuda:{t.get_device()}, other tensors of the call on cuda:{dev}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} is {t.dtype}, expected {dtype}")
    raise ValueError(f"the rows of {name} are not contiguous")


def _rows_of(t, name, rows, cols, dev, dtype=None):
    """Row stride of a [rows, cols] tensor with contiguous rows (any stride where there is one row)."""
    if not t.is_cuda or (not _one_device and t.get_device() != dev) or t.shape != (rows, cols) or (dtype is not None and t.dtype != dtype):
        _refuse(t, name, (rows, cols), dtype, dev)
    ld, one = t.stride()
    if one != 1 and cols > 1 and rows:
        _refuse(t, name, (rows, cols), dtype, dev)
    return ld if rows > 1 else max(cols, ld)


def _dense_of(t, name, shape, dtype, dev):
    """Address of a contiguous tensor of this shape."""
    if not t.is_cuda or (not _one_device and t.get_device() != dev) or t.shape != shape or t.dtype != dtype or not t.is_contiguous():
        _refuse(t, name, shape, dtype, dev)
    return t.data_ptr()


def _count_of(t, name, dev):
    """Address of a row count, the first element of an int32 tensor (None for None)."""
    if t is None:
        return None
    if not t.is_cuda or (not _one_device and t.get_device() != dev) or t.dtype != torch.int32 or t.numel() < 1:
        _refuse(t, name, tuple(t.shape) if t.numel() else (1,), torch.int32, dev)
    return t.data_ptr()


def _raw_stream(stream, dev):
    """The stream handle as an int: the given one, or the current one of the device."""
    if stream is None:
        return _current_raw_stream(dev)
    if isinstance(stream, torch.cuda.Stream):
        if stream.device_index != dev:
            raise ValueError(f"the stream is on cuda:{stream.device_index}, the call's tensors on cuda:{dev}")
        return stream.cuda_stream
    return int(stream)


try:
    _current_raw_stream, _current_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
except AttributeError:  # a torch without CUDA
    def _current_raw_stream(device):
        return torch.cuda.current_stream(device).cuda_stream

    def _current_device():
        return torch.cuda.current_device()


_pack_bank = struct.Struct("@iiqqqqP").pack  # the fields of MatrixBank, about three times as fast to fill


def _bank_of(w, name, dev):
    """(bytes of a MatrixBank, E, n, k) of a [E, n, k] tensor on CUDA device dev."""
    E, n, k = w.shape
    es, ld, one = w.stride()
    if not w.is_cuda or (one != 1 and k > 1):
        _refuse(w, name, (E, n, k), None, dev)
    if n <= 1:
        ld = max(k, ld)
    if E <= 1:
        es = max((n - 1) * ld + k, es)
    return _pack_bank(_dtype_code(w, name), E, n, k, ld, es, w.data_ptr()), E, n, k


def make_matrix_bank(w):
    """MatrixBank view of a [E, n, k] tensor of bf16, fp16 or fp32 matrices (any expert and row
    strides, contiguous rows)."""
    return MatrixBank.from_buffer_copy(_bank_of(w, "w", w.get_device())[0])


def ftmoe_grouped_matmul(a, offsets, w, out, input_grad=False, stream=None):
    """out rows = a rows times the transposed matrix of their expert (input_grad: times the
    matrix itself). a [rows, k] (input_grad: [rows, n]), w [E, n, k], both bf16 or fp16; out
    [rows, n] (input_grad: [rows, k]) bf16, fp16 or fp32; offsets int32 [E + 1]."""
    dev = 0 if _one_device else _device_of(w, "w")
    bank, E, wide_out, wide_in = _bank_of(w, "w", dev)
    rows = a.shape[0]
    if input_grad:
        wide_in, wide_out = wide_out, wide_in
    off = _dense_of(offsets, "offsets", (E + 1,), torch.int32, dev)
    ld_a, ld_out = _rows_of(a, "a", rows, wide_in, dev, w.dtype), _rows_of(out, "out", rows, wide_out, dev)
    st = lib().ftmoe_grouped_matmul(a.data_ptr(), rows, ld_a, off, bank, 1 if input_grad else 0, out.data_ptr(), ld_out,
                                    _dtype_code(out, "out"), _raw_stream(stream, dev))
    if st:
        raise FtmoeError("ftmoe_grouped_matmul", st)


def ftmoe_grouped_matmul_wgrad(dy, x, offsets, dw, accumulate=False, stream=None):
    """dw[e] = dy_e^T x_e over the rows of expert e (accumulate: added to dw). dy [rows, n] and
    x [rows, k] bf16 or fp16, dw [E, n, k] bf16, fp16 or fp32."""
    dev = 0 if _one_device else _device_of(dw, "dw")
    bank, E, n, k = _bank_of(dw, "dw", dev)
    rows, dt = dy.shape[0], dy.dtype
    off = _dense_of(offsets, "offsets", (E + 1,), torch.int32, dev)
    ld_dy, ld_x = _rows_of(dy, "dy", rows, n, dev), _rows_of(x, "x", rows, k, dev, dt)
    st = lib().ftmoe_grouped_matmul_wgrad(dy.data_ptr(), ld_dy, x.data_ptr(), ld_x, rows, _dtype_code(dy, "dy"), off,
                                          bank, 1 if accumulate else 0, _raw_stream(stream, dev))
    if st:
        raise FtmoeError("ftmoe_grouped_matmul_wgrad", st)


def ftmoe_grouped_matmul_wgrad_saved(dy, q, scales, offsets, dw, fmt=FMT_MXFP8, accumulate=False, stream=None):
    """The same with x as MXFP8 rows: q uint8 [rows, k], scales uint8 [rows, k / 32]."""
    dev = 0 if _one_device else _device_of(dw, "dw")
    bank, E, n, k = _bank_of(dw, "dw", dev)
    rows = dy.shape[0]
    off = _dense_of(offsets, "offsets", (E + 1,), torch.int32, dev)
    ld_dy = _rows_of(dy, "dy", rows, n, dev)
    qp = _dense_of(q, "q", (rows, k), torch.uint8, dev)
    sp = _dense_of(scales, "scales", (rows, k // 32), torch.uint8, dev) if fmt == FMT_MXFP8 else scales.data_ptr()
    act = Act(fmt, 0, rows, k, qp, sp, None)
    st = lib().ftmoe_grouped_matmul_wgrad_saved(dy.data_ptr(), ld_dy, _dtype_code(dy, "dy"), act, off, bank,
                                                1 if accumulate else 0, _raw_stream(stream, dev))
    if st:
        raise FtmoeError("ftmoe_grouped_matmul_wgrad_saved", st)


def _saved_of(q, scales, rows, inter, fmt, dev):
    """Addresses of q uint8 [rows, 2 * inter] and scales [rows, 2 * groups] of kept gate/up rows."""
    qp = _dense_of(q, "q", (rows, 2 * inter), torch.uint8, dev)
    if fmt == FMT_FP8:
        return qp, _dense_of(scales, "scales", (rows, 2 * cdiv(inter, 128)), torch.float32, dev)
    if fmt == FMT_MXFP8:
        return qp, _dense_of(scales, "scales", (rows, 2 * (inter // 32)), torch.uint8, dev)
    return qp, scales.data_ptr()


def ftmoe_silu_mul_save(gu, h, q, scales, fmt=FMT_MXFP8, rows_dev=None, stream=None):
    """h = silu(gate) * up from gu [rows, 2 * inter], and both halves kept in 8 bits: q uint8
    [rows, 2 * inter], scales [rows, 2 * groups] (FP8: fp32 per 128, MXFP8: uint8 per 32)."""
    rows, inter = h.shape
    dev = 0 if _one_device else _device_of(gu, "gu")
    ld_gu, ld_h = _rows_of(gu, "gu", rows, 2 * inter, dev), _rows_of(h, "h", rows, inter, dev)
    qp, sp = _saved_of(q, scales, rows, inter, fmt, dev)
    st = lib().ftmoe_silu_mul_save(gu.data_ptr(), _dtype_code(gu, "gu"), rows, inter, ld_gu,
                                   _count_of(rows_dev, "rows_dev", dev), h.data_ptr(), ld_h,
                                   _dtype_code(h, "h"), fmt, qp, sp, _raw_stream(stream, dev))
    if st:
        raise FtmoeError("ftmoe_silu_mul_save", st)


def ftmoe_silu_mul_backward(q, scales, dh, dgu, hw=None, row_weights=None, dweights=None, fmt=FMT_MXFP8,
                            rows_dev=None, stream=None):
    """Gradients from the kept gate/up rows: dgu [rows, 2 * inter], hw = weight * h [rows, inter]
    and dweights fp32 [rows], for the gradient dh [rows, inter] of the unweighted h."""
    rows, inter = dh.shape
    dev, dt = 0 if _one_device else _device_of(dh, "dh"), dh.dtype
    ld_dh, ld_dgu = _rows_of(dh, "dh", rows, inter, dev), _rows_of(dgu, "dgu", rows, 2 * inter, dev, dt)
    hp, ld_hw = (None, 0) if hw is None else (hw.data_ptr(), _rows_of(hw, "hw", rows, inter, dev, dt))
    wp = None if row_weights is None else _dense_of(row_weights, "row_weights", (rows,), torch.float32, dev)
    dp = None if dweights is None else _dense_of(dweights, "dweights", (rows,), torch.float32, dev)
    qp, sp = _saved_of(q, scales, rows, inter, fmt, dev)
    st = lib().ftmoe_silu_mul_backward(qp, sp, fmt, rows, inter, _count_of(rows_dev, "rows_dev", dev),
                                       dh.data_ptr(), ld_dh, _dtype_code(dh, "dh"), wp, dgu.data_ptr(), ld_dgu, hp,
                                       ld_hw, dp, _raw_stream(stream, dev))
    if st:
        raise FtmoeError("ftmoe_silu_mul_backward", st)


def ftmoe_selftest_wait_timeout(timeout_ns, elapsed_ns=None, stream=None):
    """One bounded pipeline wait that nothing completes, given up after timeout_ns."""
    _check("ftmoe_selftest_wait_timeout", lib().ftmoe_selftest_wait_timeout(
        int(timeout_ns), _p(elapsed_ns), _stream(stream)))


def ftmoe_selftest_shared_division(counts, stream=None):
    """The quantizers' division by a shared group scale against IEEE division on the device;
    counts (int64 tensor [2]) receives {quotients checked, quotients that differ}."""
    _check("ftmoe_selftest_shared_division", lib().ftmoe_selftest_shared_division(_p(counts), _stream(stream)))


def ftmoe_read_error_flags():
    v = ctypes.c_uint32(0)
    _check("ftmoe_read_error_flags", lib().ftmoe_read_error_flags(ctypes.byref(v)))
    return int(v.value)


# ---------------------------------------------------------------------------------
# allocation helpers (torch allocates; the library computes)
# ---------------------------------------------------------------------------------

def cdiv(a, b):
    return -(-a // b)


def quantize_act(x, fmt=FMT_FP8, stream=None):
    """bf16 [rows, k] -> (q, scales, global_scale) allocated with torch on x's device."""
    rows, k = x.shape
    dev = x.device
    if fmt == FMT_FP8:
        q = torch.empty(rows, k, dtype=torch.uint8, device=dev)
        s = torch.empty(rows, cdiv(k, 128), dtype=torch.float32, device=dev)
        ftmoe_quantize_act(x, q, s, None, fmt, stream=stream)
        return q, s, None
    if fmt == FMT_MXFP8:
        q = torch.empty(rows, k, dtype=torch.uint8, device=dev)
        s = torch.empty(rows, k // 32, dtype=torch.uint8, device=dev)
        ftmoe_quantize_act(x, q, s, None, fmt, stream=stream)
        return q, s, None
    q = torch.empty(rows, k // 2, dtype=torch.uint8, device=dev)
    s = torch.empty(rows, k // 16, dtype=torch.uint8, device=dev)
    g = torch.empty(1, dtype=torch.float32, device=dev)
    ftmoe_quantize_act(x, q, s, g, fmt, stream=stream)
    return q, s, g


def quantize_weights(w, fmt=FMT_FP8, stream=None):
    """float32 [E, n, k] -> (q, scales, global_scale) in the ExpertBank layout."""
    E, n, k = w.shape
    dev = w.device
    if fmt == FMT_FP8:
        q = torch.empty(E, n, k, dtype=torch.uint8, device=dev)
        s = torch.empty(E, cdiv(n, 128), cdiv(k, 128), dtype=torch.float32, device=dev)
        ftmoe_quantize_weights(w, q, s, None, fmt, stream=stream)
        return q, s, None
    if fmt == FMT_MXFP8:
        q = torch.empty(E, n, k, dtype=torch.uint8, device=dev)
        s = torch.empty(E, n, k // 32, dtype=torch.uint8, device=dev)
        ftmoe_quantize_weights(w, q, s, None, fmt, stream=stream)
        return q, s, None
    q = torch.empty(E, n, k // 2, dtype=torch.uint8, device=dev)
    s = torch.empty(E, n, k // 16, dtype=torch.uint8, device=dev)
    g = torch.empty(E, dtype=torch.float32, device=dev)
    ftmoe_quantize_weights(w, q, s, g, fmt, stream=stream)
    return q, s, g
