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

__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  uint32_t o = __builtin_amdgcn_update_dpp(0, v, 0xB1, 0xF, 0xF, true);   // quad_perm 1,0,3,2
  v = o > v ? o : v;
  o = __builtin_amdgcn_update_dpp(0, v, 0x4E, 0xF, 0xF, true);            // quad_perm 2,3,0,1
  return o > v ? o : v;
}

template <int DT>
__device__ __forceinline__ void load8(const void* x, long long g, float (&v)[8]) {
  if constexpr (DT == TMOE_F32) {
    const float4* p = static_cast<const float4*>(x) + 2 * g;
    const float4 a = p[0], b = p[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    const uint4 q = static_cast<const uint4*>(x)[g];
    const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (DT == TMOE_BF16) {
        v[2 * i] = __uint_as_float(u[i] << 16);
        v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
      } else {
        v[2 * i] = h2f(static_cast<uint16_t>(u[i] & 0xffffu));
        v[2 * i + 1] = h2f(static_cast<uint16_t>(u[i] >> 16));
      }
    }
  }
}

template <int DT>
__global__ __launch_bounds__(kThreads) void k_mxfp4_quantize(Mxfp4QuantArgs a) {
  // whole quads are in range together: the group count is a multiple of four
  for (long long g = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x; g < a.groups;
       g += static_cast<long long>(gridDim.x) * kThreads) {
    float v[8];
    load8<DT>(a.x, g, v);
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t b = __float_as_uint(v[i]) & 0x7fffffffu;
      m = b > m ? b : m;
    }
    const uint32_t byte = mxfp4_scale_byte(quad_max(m));
    const float inv = mxfp4_inverse_scale(byte);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= inv;
    reinterpret_cast<uint32_t*>(a.codes)[g] = byte == 255u ? 0u : mxfp4_codes8(v);
    if ((threadIdx.x & 3) == 0) a.scales[g >> 2] = static_cast<uint8_t>(byte);
  }
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
