// tmoe_mxfp8.hpp -- MXFP8 pieces: the block format on the device, launch arguments and launchers.
//
// MXFP8 (OCP Microscaling Formats, version 1.0): blocks of 32 values along the contraction axis, E4M3 elements (up to
// 448) and one E8M0 scale byte (2^(byte - 127), 255 = NaN) per block.
#pragma once
#include "tmoe.h"
#include "tmoe_device.hpp"
#include "tmoe_mxfp4.hpp"

namespace tmoe {

// Scale byte of a block with the largest magnitude amax, given as the bits of |amax|: the smallest power of two 2^e with
// amax / 2^e <= 448 (so nothing saturates), e >= -127. amax = 2^x * 1.m lies in (448 * 2^(e-1), 448 * 2^e] with
// 448 = 1.75 * 2^8, so e = x - 8, plus 1 where 1.m > 1.75. An infinity or a NaN in the block gives 255.
__device__ __forceinline__ uint32_t mxfp8_scale_byte(uint32_t amax_bits) {
  if (amax_bits >= 0x7f800000u) return 255u;
  const int byte = static_cast<int>(amax_bits >> 23) - 8 + ((amax_bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return static_cast<uint32_t>(byte > 0 ? byte : 0);
}

// Four values already divided by their block's scale -> four E4M3 bytes, round to nearest even.
__device__ __forceinline__ uint32_t mxfp8_codes4(float a, float b, float c, float d) {
  return fp8x2_from_f32(a, b) | (fp8x2_from_f32(c, d) << 16);
}

// Largest of the values of 8 neighbouring lanes: of each 4 (mxfp4_quad_max), then of the two, by mirroring the 8.
__device__ __forceinline__ uint32_t mxfp8_oct_max(uint32_t v) {
  v = mxfp4_quad_max(v);
  const uint32_t o = __builtin_amdgcn_update_dpp(0, v, 0x141, 0xF, 0xF, true);   // row_half_mirror
  return o > v ? o : v;
}

// launches: the arguments of the MXFP4 calls, codes of one byte a value
void launch_mxfp8_quantize(const Mxfp4QuantArgs& a, int dtype, hipStream_t s);
void launch_mxfp8_dequantize(const Mxfp4DequantArgs& a, int dtype, hipStream_t s);

}  // namespace tmoe
