// tmoe_norm_host.cpp -- C ABI of the RMS norm and of MXFP8 quantisation: argument checks and launches. Every argument is
// checked before the first launch; nothing is allocated and nothing synchronizes.
#include <cmath>
#include <cstdint>
#include <cstring>

#include <hip/hip_runtime.h>

#include "tmoe.h"
#include "tmoe_mxfp8.hpp"
#include "tmoe_norm.hpp"

using namespace tmoe;

namespace {

constexpr int kMaxHidden = 16384;
constexpr int kMaxTokens = (1 << 22) - 1;        // a row has up to 1024 threads, a launch fewer than 2^32

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

size_t size_of(int dtype) { return dtype == TMOE_F32 ? 4 : 2; }

bool dtype_ok(int d) { return d == TMOE_F32 || d == TMOE_BF16 || d == TMOE_F16; }

tmoe_status launched() { return hipGetLastError() == hipSuccess ? TMOE_OK : TMOE_ERR_HIP; }

tmoe_status check_config(const tmoe_norm_config* c, bool mxfp8) {
  if (!c || c->hidden <= 0 || !dtype_ok(c->dtype) || !dtype_ok(c->weight_dtype)) return TMOE_ERR_INVALID_ARG;
  if (c->weight_dtype != TMOE_F32 && c->weight_dtype != c->dtype) return TMOE_ERR_INVALID_ARG;
  if (!std::isfinite(c->eps) || c->eps < 0.0f) return TMOE_ERR_INVALID_ARG;
  if (c->hidden > kMaxHidden || (mxfp8 && c->hidden % 32 != 0)) return TMOE_ERR_UNSUPPORTED;
  return TMOE_OK;
}

tmoe_status check_tokens(int32_t T) {
  return T < 0 ? TMOE_ERR_INVALID_ARG : T > kMaxTokens ? TMOE_ERR_UNSUPPORTED : TMOE_OK;
}

bool stride_ok(int64_t stride, int hidden) { return stride >= hidden && stride <= (int64_t{1} << 32); }

tmoe_status norm(const tmoe_norm_config* c, const void* x, int64_t x_stride, const void* residual, int64_t residual_stride,
                 const void* weight, int32_t T, void* y, uint8_t* scales, void* h, float* rstd, bool mxfp8, void* stream) {
  tmoe_status st = check_config(c, mxfp8);
  if (st != TMOE_OK) return st;
  st = check_tokens(T);
  if (st != TMOE_OK || T == 0) return st;
  if (!x || !weight || !y || (mxfp8 && !scales) || (residual == nullptr) != (h == nullptr)) return TMOE_ERR_INVALID_ARG;
  if (!stride_ok(x_stride, c->hidden) || (residual && !stride_ok(residual_stride, c->hidden))) return TMOE_ERR_INVALID_ARG;
  const size_t es = size_of(c->dtype);
  if (!aligned(x, es) || !aligned(residual, es) || !aligned(h, es) || !aligned(weight, size_of(c->weight_dtype)) ||
      !aligned(y, mxfp8 ? 16 : es) || !aligned(rstd, 4))
    return TMOE_ERR_ALIGNMENT;
  NormArgs a;
  a.x = x;
  a.residual = residual;
  a.x_stride = x_stride;
  a.residual_stride = residual ? residual_stride : 0;
  a.weight = weight;
  a.eps = c->eps;
  a.tokens = T;
  a.hidden = c->hidden;
  a.y = y;
  a.scales = scales;
  a.h = h;
  a.rstd = rstd;
  (void)hipGetLastError();
  launch_rms_norm(a, c->dtype, c->weight_dtype == TMOE_F32, mxfp8, static_cast<hipStream_t>(stream));
  return launched();
}

size_t grad_scratch(const tmoe_norm_config* c, int32_t T) {
  if (T == 0) return 0;
  return 4ull * norm_grad_groups(T, c->hidden, c->dtype) * c->hidden;
}

tmoe_status check_blocks(const void* x, int32_t dtype, int64_t rows, int32_t cols, const void* codes,
                         const void* scales) {
  if (!dtype_ok(dtype) || rows < 0 || cols <= 0) return TMOE_ERR_INVALID_ARG;
  if (cols % 32 != 0 || rows > (int64_t{1} << 40) / cols) return TMOE_ERR_UNSUPPORTED;
  if (rows == 0) return TMOE_OK;
  if (!x || !codes || !scales) return TMOE_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(codes, 16)) return TMOE_ERR_ALIGNMENT;
  return TMOE_OK;
}

}  // namespace

extern "C" {

tmoe_status tmoe_rms_norm(const tmoe_norm_config* c, const void* x, int64_t x_stride, const void* residual,
                          int64_t residual_stride, const void* weight, int32_t T, void* y, void* h, float* rstd,
                          void* stream) {
  return norm(c, x, x_stride, residual, residual_stride, weight, T, y, nullptr, h, rstd, false, stream);
}

tmoe_status tmoe_rms_norm_mxfp8(const tmoe_norm_config* c, const void* x, int64_t x_stride, const void* residual,
                                int64_t residual_stride, const void* weight, int32_t T, uint8_t* codes, uint8_t* scales,
                                void* h, void* stream) {
  return norm(c, x, x_stride, residual, residual_stride, weight, T, codes, scales, h, nullptr, true, stream);
}

tmoe_status tmoe_rms_norm_backward_scratch(const tmoe_norm_config* c, int32_t T, size_t* bytes) {
  tmoe_status st = check_config(c, false);
  if (st != TMOE_OK) return st;
  st = check_tokens(T);
  if (st != TMOE_OK) return st;
  if (!bytes) return TMOE_ERR_INVALID_ARG;
  *bytes = grad_scratch(c, T);
  return TMOE_OK;
}

tmoe_status tmoe_rms_norm_backward(const tmoe_norm_config* c, const void* h, int64_t h_stride, const void* weight,
                                   const float* rstd, const void* dy, const void* dh, int32_t T, void* dx, void* dweight,
                                   void* scratch, size_t bytes, void* stream) {
  tmoe_status st = check_config(c, false);
  if (st != TMOE_OK) return st;
  st = check_tokens(T);
  if (st != TMOE_OK) return st;
  const size_t es = size_of(c->dtype), ws = size_of(c->weight_dtype), need = grad_scratch(c, T);
  if (!dweight || (T > 0 && (!h || !weight || !rstd || !dy || !dx || !stride_ok(h_stride, c->hidden))))
    return TMOE_ERR_INVALID_ARG;
  if (!aligned(h, es) || !aligned(weight, ws) || !aligned(rstd, 4) || !aligned(dy, es) || !aligned(dh, es) ||
      !aligned(dx, es) || !aligned(dweight, ws))
    return TMOE_ERR_ALIGNMENT;
  if (need > 0 && (!scratch || !aligned(scratch, 16) || bytes < need)) return TMOE_ERR_SCRATCH;
  NormGradArgs a;
  a.h = h;
  a.h_stride = h_stride;
  a.weight = weight;
  a.rstd = rstd;
  a.dy = dy;
  a.dh = dh;
  a.tokens = T;
  a.hidden = c->hidden;
  a.groups = T > 0 ? norm_grad_groups(T, c->hidden, c->dtype) : 0;
  a.dx = dx;
  a.part = static_cast<float*>(scratch);
  a.dweight = dweight;
  (void)hipGetLastError();
  launch_rms_norm_grad(a, c->dtype, c->weight_dtype == TMOE_F32, static_cast<hipStream_t>(stream));
  return launched();
}

tmoe_status tmoe_mxfp8_quantize(const void* x, int32_t dtype, int64_t rows, int32_t cols, uint8_t* codes,
                                uint8_t* scales, void* stream) {
  const tmoe_status st = check_blocks(x, dtype, rows, cols, codes, scales);
  if (st != TMOE_OK || rows == 0) return st;
  Mxfp4QuantArgs a;
  a.x = x;
  a.groups = rows * cols / 8;
  a.codes = codes;
  a.scales = scales;
  (void)hipGetLastError();
  launch_mxfp8_quantize(a, dtype, static_cast<hipStream_t>(stream));
  return launched();
}

tmoe_status tmoe_mxfp8_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int32_t cols,
                                  int32_t dtype, void* x, void* stream) {
  const tmoe_status st = check_blocks(x, dtype, rows, cols, codes, scales);
  if (st != TMOE_OK || rows == 0) return st;
  Mxfp4DequantArgs a;
  a.codes = codes;
  a.scales = scales;
  a.groups = rows * cols / 8;
  a.x = x;
  (void)hipGetLastError();
  launch_mxfp8_dequantize(a, dtype, static_cast<hipStream_t>(stream));
  return launched();
}

}  // extern "C"
