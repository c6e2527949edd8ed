// k_mxfp4_quant.hip -- MXFP4 quantisation of fp32, bf16 or fp16 rows, and back.
//
// Both are one pass over the data and bound by HBM. A lane holds eight neighbouring values (16 or 32
// bytes of input, 4 bytes of codes); the four lanes of a block exchange their largest magnitude (as
// integer bits, so infinities and NaNs win) by quad permutes.
#include "tmoe.h"
#include "tmoe_mxfp4.hpp"

namespace tmoe {

namespace {

constexpr int kThreads = 256;

template <int DT>
__global__ __launch_bounds__(kThreads) void k_mxfp4_quantize(Mxfp4QuantArgs a) {
  // whole quads are in range together: the group count is a multiple of four
  for (long long g = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x; g < a.groups;
       g += static_cast<long long>(gridDim.x) * kThreads)
    mxfp4_quantize_group<DT>(a, g);
}

__device__ __forceinline__ uint16_t bf16_rne(float f) {
  const uint32_t u = __float_as_uint(f);
  if ((u & 0x7fffffffu) > 0x7f800000u) return static_cast<uint16_t>((u >> 16) | 0x40u);
  return static_cast<uint16_t>((u + 0x7fffu + ((u >> 16) & 1u)) >> 16);
}

template <int DT>
__global__ __launch_bounds__(kThreads) void k_mxfp4_dequantize(Mxfp4DequantArgs a) {
  typedef float f2 __attribute__((ext_vector_type(2)));
  for (long long g = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x; g < a.groups;
       g += static_cast<long long>(gridDim.x) * kThreads) {
    const uint32_t c = reinterpret_cast<const uint32_t*>(a.codes)[g];
    const float s = mxfp4_scale(a.scales[g >> 2]);
    const f2 p[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 0),
                     __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 1),
                     __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 2),
                     __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 3)};
    if constexpr (DT == TMOE_F32) {
      float4* o = static_cast<float4*>(a.x) + 2 * g;
      o[0] = make_float4(p[0][0] * s, p[0][1] * s, p[1][0] * s, p[1][1] * s);
      o[1] = make_float4(p[2][0] * s, p[2][1] * s, p[3][0] * s, p[3][1] * s);
    } else {
      uint32_t u[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float lo = p[i][0] * s, hi = p[i][1] * s;
        if constexpr (DT == TMOE_BF16) {
          u[i] = static_cast<uint32_t>(bf16_rne(lo)) | (static_cast<uint32_t>(bf16_rne(hi)) << 16);
        } else {
          u[i] = static_cast<uint32_t>(__builtin_bit_cast(uint16_t, static_cast<_Float16>(lo))) |
                 (static_cast<uint32_t>(__builtin_bit_cast(uint16_t, static_cast<_Float16>(hi))) << 16);
        }
      }
      static_cast<uint4*>(a.x)[g] = make_uint4(u[0], u[1], u[2], u[3]);
    }
  }
}

unsigned grid_of(long long groups) {
  const long long g = (groups + kThreads - 1) / kThreads;
  return static_cast<unsigned>(g < 1048576 ? g : 1048576);
}

}  // namespace

void launch_mxfp4_quantize(const Mxfp4QuantArgs& a, int dtype, hipStream_t s) {
  const dim3 g(grid_of(a.groups)), b(kThreads);
  if (dtype == TMOE_F32) hipLaunchKernelGGL(k_mxfp4_quantize<TMOE_F32>, g, b, 0, s, a);
  else if (dtype == TMOE_BF16) hipLaunchKernelGGL(k_mxfp4_quantize<TMOE_BF16>, g, b, 0, s, a);
  else hipLaunchKernelGGL(k_mxfp4_quantize<TMOE_F16>, g, b, 0, s, a);
}

void launch_mxfp4_dequantize(const Mxfp4DequantArgs& a, int dtype, hipStream_t s) {
  const dim3 g(grid_of(a.groups)), b(kThreads);
  if (dtype == TMOE_F32) hipLaunchKernelGGL(k_mxfp4_dequantize<TMOE_F32>, g, b, 0, s, a);
  else if (dtype == TMOE_BF16) hipLaunchKernelGGL(k_mxfp4_dequantize<TMOE_BF16>, g, b, 0, s, a);
  else hipLaunchKernelGGL(k_mxfp4_dequantize<TMOE_F16>, g, b, 0, s, a);
}

}  // namespace tmoe
