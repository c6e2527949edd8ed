// k_mxfp8_quant.hip -- MXFP8 quantisation of fp32, bf16 or fp16 rows, and back.
//
// Both are one pass over the data and bound by HBM. A lane holds eight neighbouring values (16 or 32 bytes of input, 8
// bytes of codes); the four lanes of a block exchange their largest magnitude (as integer bits, so infinities and NaNs
// win) by quad permutes. Passes over more than the caches hold read past them (65536 x 1024 fp32, quantised and read back:
// 115 us instead of 134). Stores that do so cost more than they give: a lane's two of fp32 fill a line only together (60 us
// of dequantisation become 99).
#include <type_traits>

#include "tmoe.h"
#include "tmoe_mxfp8.hpp"

namespace tmoe {

namespace {

constexpr int kThreads = 256;

typedef uint32_t u2v __attribute__((ext_vector_type(2)));
typedef uint32_t u4v __attribute__((ext_vector_type(4)));

// PAST: what is read does not stay in the caches.
template <int DT, bool PAST>
__global__ __launch_bounds__(kThreads) void k_mxfp8_quantize(Mxfp4QuantArgs a) {
  // whole quads are in range together: the group count is a multiple of four
  for (long long g = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x; g < a.groups;
       g += static_cast<long long>(gridDim.x) * kThreads) {
    float v[8];
    if constexpr (PAST) {
      constexpr int N = DT == TMOE_F32 ? 2 : 1;
      u4v q[N];
#pragma unroll
      for (int i = 0; i < N; ++i) q[i] = __builtin_nontemporal_load(static_cast<const u4v*>(a.x) + N * g + i);
      mxfp4_load8<DT>(q, 0, v);
    } else {
      mxfp4_load8<DT>(a.x, g, v);
    }
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t b = __float_as_uint(v[i]) & 0x7fffffffu;
      m = b > m ? b : m;
    }
    const uint32_t byte = mxfp8_scale_byte(mxfp4_quad_max(m));
    const float inv = mxfp4_inverse_scale(byte);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= inv;
    reinterpret_cast<uint2*>(a.codes)[g] =
        byte == 255u ? make_uint2(0u, 0u) : make_uint2(mxfp8_codes4(v[0], v[1], v[2], v[3]), mxfp8_codes4(v[4], v[5], v[6], v[7]));
    if ((threadIdx.x & 3) == 0) a.scales[g >> 2] = static_cast<uint8_t>(byte);
  }
}

template <int DT, bool PAST>
__global__ __launch_bounds__(kThreads) void k_mxfp8_dequantize(Mxfp4DequantArgs a) {
  typedef float f2 __attribute__((ext_vector_type(2)));
  for (long long g = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x; g < a.groups;
       g += static_cast<long long>(gridDim.x) * kThreads) {
    const u2v* const codes = reinterpret_cast<const u2v*>(a.codes) + g;
    u2v c;
    if constexpr (PAST) c = __builtin_nontemporal_load(codes);
    else c = *codes;
    const float s = mxfp4_scale(a.scales[g >> 2]);
    const f2 p[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c.x, 1.0f, false),
                     __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c.x, 1.0f, true),
                     __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c.y, 1.0f, false),
                     __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c.y, 1.0f, true)};
    if constexpr (DT == TMOE_F32) {
      float4* o = static_cast<float4*>(a.x) + 2 * g;
      o[0] = make_float4(p[0][0] * s, p[0][1] * s, p[1][0] * s, p[1][1] * s);
      o[1] = make_float4(p[2][0] * s, p[2][1] * s, p[3][0] * s, p[3][1] * s);
    } else {
      typedef __bf16 b2 __attribute__((ext_vector_type(2)));
      uint32_t u[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f2 v = {p[i][0] * s, p[i][1] * s};
        if constexpr (DT == TMOE_BF16) u[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(v, b2));
        else u[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(v, half2v));
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

void launch_mxfp8_quantize(const Mxfp4QuantArgs& a, int dtype, hipStream_t s) {
  const dim3 g(grid_of(a.groups)), b(kThreads);
  const bool past = passes_caches(8 * a.groups * ((dtype == TMOE_F32 ? 4 : 2) + 1));
  auto go = [&](auto dt) {
    if (past) hipLaunchKernelGGL((k_mxfp8_quantize<dt.value, true>), g, b, 0, s, a);
    else hipLaunchKernelGGL((k_mxfp8_quantize<dt.value, false>), g, b, 0, s, a);
  };
  if (dtype == TMOE_F32) go(std::integral_constant<int, TMOE_F32>{});
  else if (dtype == TMOE_BF16) go(std::integral_constant<int, TMOE_BF16>{});
  else go(std::integral_constant<int, TMOE_F16>{});
}

void launch_mxfp8_dequantize(const Mxfp4DequantArgs& a, int dtype, hipStream_t s) {
  const dim3 g(grid_of(a.groups)), b(kThreads);
  const bool past = passes_caches(8 * a.groups * ((dtype == TMOE_F32 ? 4 : 2) + 1));
  auto go = [&](auto dt) {
    if (past) hipLaunchKernelGGL((k_mxfp8_dequantize<dt.value, true>), g, b, 0, s, a);
    else hipLaunchKernelGGL((k_mxfp8_dequantize<dt.value, false>), g, b, 0, s, a);
  };
  if (dtype == TMOE_F32) go(std::integral_constant<int, TMOE_F32>{});
  else if (dtype == TMOE_BF16) go(std::integral_constant<int, TMOE_BF16>{});
  else go(std::integral_constant<int, TMOE_F16>{});
}

}  // namespace tmoe
