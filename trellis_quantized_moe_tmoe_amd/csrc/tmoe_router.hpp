// tmoe_router.hpp -- launch arguments of the router kernels (top-k, balance loss, their gradients).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace tmoe {

struct RouterTopkArgs {
  const void* logits;        // [T][E], row stride `stride` elements
  long long stride;
  const uint8_t* mask;       // [T] 0 = the row is left out, or null
  int tokens, experts, top_k, renormalize, ids64;
  void* ids;                 // [T][k]
  float* w;                  // [T][k]
  float* lse;                // [T]
};

struct BalanceArgs {
  const void* logits;
  long long stride;
  const float* lse;          // [T], -inf leaves the row out
  const void* ids;           // [T][k]
  int tokens, experts, top_k, ids64;
  int groups;                // workgroups of the first launch
  int rows_per_group;
  float coefficient;
  int pitch;                 // E rounded up to a multiple of 4
  float* psum;               // [groups][pitch] sums of probabilities
  int32_t* csum;             // [groups][pitch] routes per expert
  int32_t* nsum;             // [groups][2] rows that count, and routes
  int32_t* done;             // workgroups of the second launch that have ended (cleared by the first)
  double* part;              // [ceil(E / 32)] their parts of the loss
  float* loss;               // [1]
  int32_t* counts;           // [E]
  float* slope;              // [E] dloss/dp_te = coefficient * E * f_e / n
};

struct RouterGradArgs {
  const void* logits;
  long long stride;
  const float* lse;
  const void* ids;
  const float* w;            // top-k part: [T][k] with dw, or null
  const float* dw;
  const float* slope;        // balance part: [E] with dloss [1], or null
  const float* dloss;
  int tokens, experts, top_k, renormalize, ids64;
  void* dlogits;             // [T][E], the logits' type
};

constexpr int kBalanceMaxGroups = 256;   // one workgroup of 16 wavefronts a CU

// dtype: TMOE_F32, TMOE_BF16 or TMOE_F16
void launch_router_topk(const RouterTopkArgs& a, int dtype, hipStream_t s);
void launch_balance(const BalanceArgs& a, int dtype, hipStream_t s);
void launch_router_grad(const RouterGradArgs& a, int dtype, hipStream_t s);

}  // namespace tmoe
