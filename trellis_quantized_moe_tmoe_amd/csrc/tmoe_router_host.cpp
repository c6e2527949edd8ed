// tmoe_router_host.cpp -- C ABI of the router: argument checks and launches. Every argument is
// checked before the first launch; nothing is allocated and nothing synchronizes.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include <hip/hip_runtime.h>

#include "tmoe.h"
#include "tmoe_router.hpp"

using namespace tmoe;

namespace {

constexpr int kMaxExperts = 512;
constexpr int kMaxTopK = 32;
constexpr int kMaxTokens = 1 << 24;

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

tmoe_status check_config(const tmoe_router_config* c) {
  if (!c || c->num_experts <= 0 || c->top_k <= 0) return TMOE_ERR_INVALID_ARG;
  if (c->logits_dtype < TMOE_F32 || c->logits_dtype > TMOE_F16) return TMOE_ERR_INVALID_ARG;
  if (c->ids_dtype != TMOE_IDS_I32 && c->ids_dtype != TMOE_IDS_I64) return TMOE_ERR_INVALID_ARG;
  if (c->renormalize != 0 && c->renormalize != 1) return TMOE_ERR_INVALID_ARG;
  if (c->num_experts > kMaxExperts || c->top_k > kMaxTopK) return TMOE_ERR_UNSUPPORTED;
  if (c->top_k > c->num_experts) return TMOE_ERR_INVALID_ARG;
  return TMOE_OK;
}

tmoe_status check_rows(const tmoe_router_config* c, const void* logits, int64_t stride, const void* ids, int32_t T) {
  if (T < 0) return TMOE_ERR_INVALID_ARG;
  if (T > kMaxTokens) return TMOE_ERR_UNSUPPORTED;
  if (T == 0) return TMOE_OK;
  if (!logits || !ids || stride < c->num_experts) return TMOE_ERR_INVALID_ARG;
  if (stride > (int64_t{1} << 32)) return TMOE_ERR_UNSUPPORTED;
  if (!aligned(logits, c->logits_dtype == TMOE_F32 ? 4 : 2) || !aligned(ids, c->ids_dtype == TMOE_IDS_I64 ? 8 : 4))
    return TMOE_ERR_ALIGNMENT;
  return TMOE_OK;
}

struct BalanceShape {
  int groups, rows, pitch;
  size_t psum, csum, nsum, done, part, total;    // arena offsets
};

BalanceShape balance_shape(int T, int E) {
  BalanceShape b;
  // at least 16 rows (one a wavefront) per workgroup, at most kBalanceMaxGroups workgroups
  b.pitch = (E + 3) / 4 * 4;
  b.rows = std::max(16, (T + kBalanceMaxGroups - 1) / kBalanceMaxGroups);
  b.groups = (T + b.rows - 1) / b.rows;
  auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  b.psum = 0;
  b.csum = up(4ull * b.groups * b.pitch);
  b.nsum = b.csum + up(4ull * b.groups * b.pitch);
  b.done = b.nsum + up(8ull * b.groups);
  b.part = b.done + up(4);
  b.total = b.groups ? b.part + up(8ull * ((E + 31) / 32)) : 0;
  return b;
}

tmoe_status launched() { return hipGetLastError() == hipSuccess ? TMOE_OK : TMOE_ERR_HIP; }

}  // namespace

extern "C" {

tmoe_status tmoe_router_topk(const tmoe_router_config* c, const void* logits, int64_t stride, const uint8_t* mask,
                             int32_t T, void* ids, float* w, float* lse, void* stream) {
  tmoe_status st = check_config(c);
  if (st != TMOE_OK) return st;
  st = check_rows(c, logits, stride, ids, T);
  if (st != TMOE_OK || T == 0) return st;
  if (!w || !lse) return TMOE_ERR_INVALID_ARG;
  if (!aligned(w, 4) || !aligned(lse, 4)) return TMOE_ERR_ALIGNMENT;
  RouterTopkArgs a;
  a.logits = logits;
  a.stride = stride;
  a.mask = mask;
  a.tokens = T;
  a.experts = c->num_experts;
  a.top_k = c->top_k;
  a.renormalize = c->renormalize;
  a.ids64 = c->ids_dtype == TMOE_IDS_I64;
  a.ids = ids;
  a.w = w;
  a.lse = lse;
  (void)hipGetLastError();
  launch_router_topk(a, c->logits_dtype, static_cast<hipStream_t>(stream));
  return launched();
}

tmoe_status tmoe_balance_loss_scratch(const tmoe_router_config* c, int32_t T, size_t* bytes) {
  const tmoe_status st = check_config(c);
  if (st != TMOE_OK) return st;
  if (!bytes || T < 0) return TMOE_ERR_INVALID_ARG;
  if (T > kMaxTokens) return TMOE_ERR_UNSUPPORTED;
  *bytes = balance_shape(T, c->num_experts).total;
  return TMOE_OK;
}

tmoe_status tmoe_balance_loss(const tmoe_router_config* c, const void* logits, int64_t stride, const float* lse,
                              const void* ids, int32_t T, float coefficient, float* loss, int32_t* counts,
                              float* slope, void* scratch, size_t bytes, void* stream) {
  tmoe_status st = check_config(c);
  if (st != TMOE_OK) return st;
  st = check_rows(c, logits, stride, ids, T);
  if (st != TMOE_OK) return st;
  if (!std::isfinite(coefficient) || !loss || !counts || !slope || (T > 0 && !lse)) return TMOE_ERR_INVALID_ARG;
  if (!aligned(lse, 4) || !aligned(loss, 4) || !aligned(counts, 4) || !aligned(slope, 4)) return TMOE_ERR_ALIGNMENT;
  const BalanceShape b = balance_shape(T, c->num_experts);
  if (b.total > 0 && (!scratch || !aligned(scratch, 16) || bytes < b.total)) return TMOE_ERR_SCRATCH;
  BalanceArgs a;
  a.logits = logits;
  a.stride = stride;
  a.lse = lse;
  a.ids = ids;
  a.tokens = T;
  a.experts = c->num_experts;
  a.top_k = c->top_k;
  a.ids64 = c->ids_dtype == TMOE_IDS_I64;
  a.groups = b.groups;
  a.rows_per_group = b.rows;
  a.pitch = b.pitch;
  a.coefficient = coefficient;
  char* base = static_cast<char*>(scratch);
  a.psum = reinterpret_cast<float*>(base + b.psum);
  a.csum = reinterpret_cast<int32_t*>(base + b.csum);
  a.nsum = reinterpret_cast<int32_t*>(base + b.nsum);
  a.done = reinterpret_cast<int32_t*>(base + b.done);
  a.part = reinterpret_cast<double*>(base + b.part);
  a.loss = loss;
  a.counts = counts;
  a.slope = slope;
  (void)hipGetLastError();
  launch_balance(a, c->logits_dtype, static_cast<hipStream_t>(stream));
  return launched();
}

tmoe_status tmoe_router_backward(const tmoe_router_config* c, const void* logits, int64_t stride, const float* lse,
                                 const void* ids, const float* w, const float* dw, const float* slope,
                                 const float* dloss, int32_t T, void* dlogits, void* stream) {
  tmoe_status st = check_config(c);
  if (st != TMOE_OK) return st;
  st = check_rows(c, logits, stride, ids, T);
  if (st != TMOE_OK) return st;
  if ((w == nullptr) != (dw == nullptr) || (slope == nullptr) != (dloss == nullptr) || (!dw && !dloss))
    return TMOE_ERR_INVALID_ARG;
  if (T == 0) return TMOE_OK;
  if (!lse || !dlogits) return TMOE_ERR_INVALID_ARG;
  if (!aligned(lse, 4) || !aligned(w, 4) || !aligned(dw, 4) || !aligned(slope, 4) || !aligned(dloss, 4) ||
      !aligned(dlogits, c->logits_dtype == TMOE_F32 ? 4 : 2))
    return TMOE_ERR_ALIGNMENT;
  RouterGradArgs a;
  a.logits = logits;
  a.stride = stride;
  a.lse = lse;
  a.ids = ids;
  a.w = w;
  a.dw = dw;
  a.slope = slope;
  a.dloss = dloss;
  a.tokens = T;
  a.experts = c->num_experts;
  a.top_k = c->top_k;
  a.renormalize = c->renormalize;
  a.ids64 = c->ids_dtype == TMOE_IDS_I64;
  a.dlogits = dlogits;
  (void)hipGetLastError();
  launch_router_grad(a, c->logits_dtype, static_cast<hipStream_t>(stream));
  return launched();
}

}  // extern "C"
