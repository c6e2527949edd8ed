// tmoe_norm.hpp -- launch arguments of the RMS norm and its backward.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace tmoe {

struct NormArgs {
  const void* x;             // [T][H], row stride x_stride elements
  const void* residual;      // or null
  long long x_stride, residual_stride;
  const void* weight;        // [H]
  float eps;
  int tokens, hidden;
  void* y;                   // [T][H], or MXFP8 codes
  uint8_t* scales;           // MXFP8: [T][H / 32]
  void* h;                   // [T][H] x + residual; null without a residual
  float* rstd;               // [T] or null
};

struct NormGradArgs {
  const void* h;             // [T][H], row stride h_stride elements
  long long h_stride;
  const void* weight;
  const float* rstd;         // [T]
  const void* dy;            // [T][H]
  const void* dh;            // [T][H] or null
  int tokens, hidden;
  int groups;                // partial sums of dweight
  void* dx;                  // [T][H]
  float* part;               // [groups][H]
  void* dweight;             // [H]
};

// Vectors of a lane's 16 bytes of x in a row, and the shape they run on: wavefronts that share a row, rows a workgroup,
// vectors a lane.
struct NormShape {
  int threads, rows, nv;     // threads a row (64 .. 1024), rows a workgroup, vectors a lane (1, 2 or 4)
};
NormShape norm_shape(int hidden, int dtype);
int norm_grad_groups(int tokens, int hidden, int dtype);

// dtype: TMOE_F32, TMOE_BF16, TMOE_F16 of x (and y, h); weight_f32: the weight is fp32, else of dtype
void launch_rms_norm(const NormArgs& a, int dtype, bool weight_f32, bool mxfp8, hipStream_t s);
void launch_rms_norm_grad(const NormGradArgs& a, int dtype, bool weight_f32, hipStream_t s);

}  // namespace tmoe
