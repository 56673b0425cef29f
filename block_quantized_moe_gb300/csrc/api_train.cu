// C ABI of the training and 16-bit entry points: argument checks on the host, then launches on
// the caller's stream (no allocation, no synchronisation).
#include "common.cuh"
#include "internal.h"

using namespace ftmoe;

namespace {

inline cudaStream_t as_stream(void* s) { return reinterpret_cast<cudaStream_t>(s); }
inline ftmoe_status from_cuda(cudaError_t e) { return e == cudaSuccess ? FTMOE_OK : FTMOE_CUDA_ERROR; }

bool half_dtype(int32_t d) { return d == FTMOE_OUT_BF16 || d == FTMOE_OUT_FP16; }
bool any_dtype(int32_t d) { return half_dtype(d) || d == FTMOE_OUT_FP32; }

// sizes are checked against limits that keep every product of them in 64 bits
constexpr int64_t kMaxDim = (int64_t)1 << 31;

ftmoe_status check_matrix_bank(const ftmoe_matrix_bank* w, bool half_only) {
  if (!w || w->num_experts <= 0 || w->n <= 0 || w->k <= 0 || w->n >= kMaxDim || w->k >= kMaxDim) return FTMOE_INVALID_ARG;
  if (half_only ? !half_dtype(w->dtype) : !any_dtype(w->dtype)) return FTMOE_INVALID_ARG;
  if (w->ld < w->k || w->ld >= kMaxDim || w->expert_stride < (w->n - 1) * w->ld + w->k ||
      w->expert_stride > ((int64_t)1 << 60) / w->num_experts)
    return FTMOE_INVALID_ARG;
  return w->w ? FTMOE_OK : FTMOE_INVALID_ARG;
}

// element addresses have to be multiples of the element
bool aligned(const void* p, int32_t dtype) { return (uintptr_t)p % (dtype == FTMOE_OUT_FP32 ? 4 : 2) == 0; }
bool aligned4(const void* p) { return (uintptr_t)p % 4 == 0; }

}  // namespace

extern "C" {

ftmoe_status ftmoe_grouped_matmul(const void* a, int64_t rows, int64_t ld_a, const int32_t* offsets,
                                  const ftmoe_matrix_bank* w, int32_t input_grad, void* out, int64_t ld_out,
                                  int32_t out_dtype, void* stream) {
  if (rows < 0 || rows >= kMaxDim || !any_dtype(out_dtype) || (input_grad != 0 && input_grad != 1)) return FTMOE_INVALID_ARG;
  const ftmoe_status st = check_matrix_bank(w, true);
  if (st != FTMOE_OK) return st;
  const int64_t in = input_grad ? w->n : w->k, outw = input_grad ? w->k : w->n;
  if (ld_a < in || ld_out < outw || ld_a >= kMaxDim || ld_out >= kMaxDim) return FTMOE_INVALID_ARG;
  if (rows == 0) return FTMOE_OK;
  if (!a || !offsets || !out) return FTMOE_INVALID_ARG;
  if (!aligned(a, w->dtype) || !aligned(w->w, w->dtype) || !aligned(out, out_dtype) || !aligned4(offsets))
    return FTMOE_INVALID_ARG;
  Matmul16Args g = {};
  g.a = a;
  g.ld_a = ld_a;
  g.rows = rows;
  g.dtype = w->dtype;
  g.offsets = offsets;
  g.w = *w;
  g.input_grad = input_grad;
  g.out = out;
  g.ld_out = ld_out;
  g.out_dtype = out_dtype;
  return from_cuda(launch_matmul16(g, as_stream(stream)));
}

static ftmoe_status wgrad(const void* dy, int64_t ld_dy, const void* x, int64_t ld_x, const uint8_t* x_scales,
                          int64_t rows, int32_t dtype, const int32_t* offsets, const ftmoe_matrix_bank* dw,
                          int32_t accumulate, void* stream) {
  if (rows < 0 || rows >= kMaxDim || !half_dtype(dtype) || (accumulate != 0 && accumulate != 1)) return FTMOE_INVALID_ARG;
  const ftmoe_status st = check_matrix_bank(dw, false);
  if (st != FTMOE_OK) return st;
  if (ld_dy < dw->n || ld_x < dw->k || ld_dy >= kMaxDim || ld_x >= kMaxDim || !offsets) return FTMOE_INVALID_ARG;
  if (rows > 0 && (!dy || !x)) return FTMOE_INVALID_ARG;
  if (!aligned(dy, dtype) || (!x_scales && !aligned(x, dtype)) || !aligned(dw->w, dw->dtype) ||
      !aligned4(offsets))
    return FTMOE_INVALID_ARG;
  Matmul16Args g = {};
  g.a = dy;
  g.ld_a = ld_dy;
  g.rows = rows;
  g.dtype = dtype;
  g.offsets = offsets;
  g.w = *dw;
  g.wgrad = 1;
  g.x = x;
  g.ld_x = ld_x;
  g.x_scales = x_scales;
  g.accumulate = accumulate;
  return from_cuda(launch_matmul16(g, as_stream(stream)));
}

ftmoe_status ftmoe_grouped_matmul_wgrad(const void* dy, int64_t ld_dy, const void* x, int64_t ld_x, int64_t rows,
                                        int32_t dtype, const int32_t* offsets, const ftmoe_matrix_bank* dw,
                                        int32_t accumulate, void* stream) {
  return wgrad(dy, ld_dy, x, ld_x, nullptr, rows, dtype, offsets, dw, accumulate, stream);
}

ftmoe_status ftmoe_grouped_matmul_wgrad_saved(const void* dy, int64_t ld_dy, int32_t dtype, const ftmoe_act* x,
                                              const int32_t* offsets, const ftmoe_matrix_bank* dw,
                                              int32_t accumulate, void* stream) {
  if (!x || !dw || x->rows < 0 || x->k != dw->k) return FTMOE_INVALID_ARG;
  if (x->format == FTMOE_FMT_FP8 || x->format == FTMOE_FMT_NVFP4) return FTMOE_UNSUPPORTED;
  if (x->format != FTMOE_FMT_MXFP8 || x->k % kMxBlock != 0 || x->global_scale) return FTMOE_INVALID_ARG;
  if (x->rows > 0 && (!x->q || !x->scales)) return FTMOE_INVALID_ARG;
  if (x->rows == 0) return wgrad(dy, ld_dy, nullptr, dw->k, nullptr, 0, dtype, offsets, dw, accumulate, stream);
  return wgrad(dy, ld_dy, x->q, x->k, static_cast<const uint8_t*>(x->scales), x->rows, dtype, offsets, dw, accumulate,
               stream);
}

ftmoe_status ftmoe_silu_mul_save(const void* gu, int32_t gu_dtype, int64_t rows, int64_t inter, int64_t ld_gu,
                                 const int32_t* rows_dev, void* h, int64_t ld_h, int32_t h_dtype, int32_t format,
                                 uint8_t* q, void* scales, void* stream) {
  if (rows < 0 || rows >= kMaxDim || inter <= 0 || inter >= kMaxDim / 2 || ld_gu < 2 * inter || ld_h < inter ||
      ld_gu >= kMaxDim || ld_h >= kMaxDim || !any_dtype(gu_dtype) || !any_dtype(h_dtype))
    return FTMOE_INVALID_ARG;
  if (format == FTMOE_FMT_NVFP4) return FTMOE_UNSUPPORTED;
  if (format != FTMOE_FMT_FP8 && format != FTMOE_FMT_MXFP8) return FTMOE_INVALID_ARG;
  if (format == FTMOE_FMT_MXFP8 && inter % kMxBlock != 0) return FTMOE_INVALID_ARG;
  if (rows == 0) return FTMOE_OK;
  if (!gu || !h || !q || !scales) return FTMOE_INVALID_ARG;
  if (!aligned(gu, gu_dtype) || !aligned(h, h_dtype) || (format == FTMOE_FMT_FP8 && !aligned4(scales)) || !aligned4(rows_dev))
    return FTMOE_INVALID_ARG;
  SiluSaveArgs s = {gu, gu_dtype, rows, inter, ld_gu, rows_dev, h, ld_h, h_dtype, format == FTMOE_FMT_MXFP8, q, scales};
  return from_cuda(launch_silu_save(s, as_stream(stream)));
}

ftmoe_status ftmoe_silu_mul_backward(const uint8_t* q, const void* scales, int32_t format, int64_t rows,
                                     int64_t inter, const int32_t* rows_dev, const void* dh, int64_t ld_dh,
                                     int32_t dtype, const float* row_weights, void* dgu, int64_t ld_dgu, void* hw,
                                     int64_t ld_hw, float* dweights, void* stream) {
  if (rows < 0 || rows >= kMaxDim || inter <= 0 || inter >= kMaxDim / 2 || ld_dh < inter || ld_dgu < 2 * inter ||
      ld_dh >= kMaxDim || ld_dgu >= kMaxDim || (hw && (ld_hw < inter || ld_hw >= kMaxDim)) || !any_dtype(dtype))
    return FTMOE_INVALID_ARG;
  if (format == FTMOE_FMT_NVFP4) return FTMOE_UNSUPPORTED;
  if (format != FTMOE_FMT_FP8 && format != FTMOE_FMT_MXFP8) return FTMOE_INVALID_ARG;
  if (format == FTMOE_FMT_MXFP8 && inter % kMxBlock != 0) return FTMOE_INVALID_ARG;
  if (rows == 0) return FTMOE_OK;
  if (!q || !scales || !dh || !dgu) return FTMOE_INVALID_ARG;
  if (!aligned(dh, dtype) || !aligned(dgu, dtype) || !aligned(hw, dtype) ||
      (format == FTMOE_FMT_FP8 && !aligned4(scales)) || !aligned4(row_weights) || !aligned4(dweights) || !aligned4(rows_dev))
    return FTMOE_INVALID_ARG;
  SiluBackwardArgs s = {q,   scales, format == FTMOE_FMT_MXFP8, rows, inter, rows_dev, dh, ld_dh, dtype, row_weights,
                        dgu, ld_dgu, hw, ld_hw, dweights};
  return from_cuda(launch_silu_backward(s, as_stream(stream)));
}

}  // extern "C"
