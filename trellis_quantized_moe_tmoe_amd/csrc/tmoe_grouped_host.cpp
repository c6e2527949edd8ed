// tmoe_grouped_host.cpp -- C ABI of the products grouped by expert: argument checks and launches. Every argument is
// checked before the launch; nothing is allocated and nothing synchronizes.
#include <cstdint>
#include <cstring>

#include <hip/hip_runtime.h>

#include "tmoe.h"
#include "tmoe_grouped.hpp"

using namespace tmoe;

namespace {

constexpr int kMaxExperts = 512;                 // eight a lane in the kernels' search
constexpr int kMaxDim = 1 << 16;
constexpr int kMaxRows = 1 << 26;

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

tmoe_status check_config(const tmoe_grouped_config* c, bool mxfp8) {
  if (!c || c->num_experts <= 0 || c->in_features <= 0 || c->out_features <= 0) return TMOE_ERR_INVALID_ARG;
  if (!mxfp8 && c->dtype != TMOE_BF16 && c->dtype != TMOE_F16) return TMOE_ERR_INVALID_ARG;
  if (c->out_dtype != TMOE_F32 && c->out_dtype != (mxfp8 ? static_cast<int32_t>(TMOE_BF16) : c->dtype))
    return TMOE_ERR_INVALID_ARG;
  if (c->offsets_dtype != TMOE_IDS_I32 && c->offsets_dtype != TMOE_IDS_I64) return TMOE_ERR_INVALID_ARG;
  if (c->num_experts > kMaxExperts || c->in_features > kMaxDim || c->out_features > kMaxDim) return TMOE_ERR_UNSUPPORTED;
  if (c->in_features % (mxfp8 ? 32 : 8) != 0 || c->out_features % 8 != 0) return TMOE_ERR_UNSUPPORTED;
  return TMOE_OK;
}

tmoe_status check_call(const tmoe_grouped_config* c, const void* r, const void* cc, const void* offsets, int32_t R,
                       const void* y) {
  if (R < 0) return TMOE_ERR_INVALID_ARG;
  if (R > kMaxRows) return TMOE_ERR_UNSUPPORTED;
  if (!aligned(r, 16) || !aligned(cc, 16) || !aligned(y, 16) || !aligned(offsets, c->offsets_dtype == TMOE_IDS_I64 ? 8 : 4))
    return TMOE_ERR_ALIGNMENT;
  return TMOE_OK;
}

GroupedArgs args(const tmoe_grouped_config* c, const void* r, const void* cc, const void* offsets, int32_t R, int depth,
                 int cols, void* y) {
  GroupedArgs a;
  std::memset(&a, 0, sizeof(a));
  a.r = r;
  a.c = cc;
  a.offsets = offsets;
  a.off64 = c->offsets_dtype == TMOE_IDS_I64;
  a.experts = c->num_experts;
  a.rows = R;
  a.depth = depth;
  a.cols = cols;
  a.y = y;
  return a;
}

tmoe_status launch(const tmoe_grouped_config* c, const GroupedArgs& a, int op, void* stream) {
  (void)hipGetLastError();
  const bool f32 = c->out_dtype == TMOE_F32;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const bool fits = c->dtype == TMOE_BF16 ? launch_grouped_bf16(a, op, f32, s) : launch_grouped_f16(a, op, f32, s);
  if (!fits) return TMOE_ERR_UNSUPPORTED;
  return hipGetLastError() == hipSuccess ? TMOE_OK : TMOE_ERR_HIP;
}

}  // namespace

extern "C" {

tmoe_status tmoe_grouped_linear(const tmoe_grouped_config* c, const void* x, const void* w, const void* offsets, int32_t R,
                                void* y, void* stream) {
  tmoe_status st = check_config(c, false);
  if (st == TMOE_OK) st = check_call(c, x, w, offsets, R, y);
  if (st != TMOE_OK || R == 0) return st;
  if (!x || !w || !offsets || !y) return TMOE_ERR_INVALID_ARG;
  return launch(c, args(c, x, w, offsets, R, c->in_features, c->out_features, y), kGroupedLinear, stream);
}

tmoe_status tmoe_grouped_grad_x(const tmoe_grouped_config* c, const void* dy, const void* w, const void* offsets, int32_t R,
                                void* dx, void* stream) {
  tmoe_status st = check_config(c, false);
  if (st == TMOE_OK) st = check_call(c, dy, w, offsets, R, dx);
  if (st != TMOE_OK || R == 0) return st;
  if (!dy || !w || !offsets || !dx) return TMOE_ERR_INVALID_ARG;
  return launch(c, args(c, dy, w, offsets, R, c->out_features, c->in_features, dx), kGroupedGradX, stream);
}

tmoe_status tmoe_grouped_grad_w(const tmoe_grouped_config* c, const void* dy, const void* x, const void* offsets, int32_t R,
                                void* dw, void* stream) {
  tmoe_status st = check_config(c, false);
  if (st == TMOE_OK) st = check_call(c, dy, x, offsets, R, dw);
  if (st != TMOE_OK) return st;
  if (!offsets || !dw || (R > 0 && (!dy || !x))) return TMOE_ERR_INVALID_ARG;
  GroupedArgs a = args(c, dy, x, offsets, R, 0, c->in_features, dw);
  a.out_rows = c->out_features;
  return launch(c, a, kGroupedGradW, stream);
}

tmoe_status tmoe_grouped_linear_mxfp8(const tmoe_grouped_config* c, const uint8_t* xq, const uint8_t* xs, const uint8_t* wq,
                                      const uint8_t* ws, const void* offsets, int32_t R, void* y, void* stream) {
  tmoe_status st = check_config(c, true);
  if (st == TMOE_OK) st = check_call(c, xq, wq, offsets, R, y);
  if (st != TMOE_OK || R == 0) return st;
  if (!xq || !xs || !wq || !ws || !offsets || !y) return TMOE_ERR_INVALID_ARG;
  GroupedArgs a = args(c, xq, wq, offsets, R, c->in_features, c->out_features, y);
  a.rs = xs;
  a.cs = ws;
  (void)hipGetLastError();
  if (!launch_grouped_mxfp8(a, c->out_dtype == TMOE_F32, static_cast<hipStream_t>(stream))) return TMOE_ERR_UNSUPPORTED;
  return hipGetLastError() == hipSuccess ? TMOE_OK : TMOE_ERR_HIP;
}

}  // extern "C"
