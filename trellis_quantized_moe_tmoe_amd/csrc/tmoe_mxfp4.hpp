// tmoe_mxfp4.hpp -- MXFP4 pieces: the block format on the device, launch arguments and launchers.
//
// MXFP4 (OCP Microscaling Formats, version 1.0): blocks of 32 values along the contraction axis, E2M1
// elements (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives) and one E8M0 scale byte (2^(byte - 127),
// 255 = NaN) per block. Element 2i of a row is the low nibble of byte i.
#pragma once
#include "tmoe.h"
#include "tmoe_device.hpp"

namespace tmoe {

struct RouteMapArgs;

// Scale byte of a block with the largest magnitude amax, given as the bits of |amax|: the smallest
// power of two 2^e with amax / 2^e <= 6 (so nothing saturates), e >= -127. amax = 2^x * 1.m lies in
// (6 * 2^(e-1), 6 * 2^e] with 6 = 1.5 * 2^2, so e = x - 2, plus 1 where 1.m > 1.5; subnormal amax
// gives -127. An infinity or a NaN in the block gives 255.
__device__ __forceinline__ uint32_t mxfp4_scale_byte(uint32_t amax_bits) {
  if (amax_bits >= 0x7f800000u) return 255u;
  const int byte = static_cast<int>(amax_bits >> 23) - 2 + ((amax_bits & 0x7fffffu) > 0x400000u ? 1 : 0);
  return static_cast<uint32_t>(byte > 0 ? byte : 0);
}

// 2^-(byte - 127), exact for the bytes above (0..253); for 255 the caller puts zeros in place of the codes.
__device__ __forceinline__ float mxfp4_inverse_scale(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// 2^(byte - 127); NaN for 255.
__device__ __forceinline__ float mxfp4_scale(uint32_t byte) {
  if (byte == 255u) return __uint_as_float(0x7fc00000u);
  return __uint_as_float(byte == 0u ? 0x00400000u : byte << 23);
}

// Eight values already divided by their block's scale -> eight codes, round to nearest even.
__device__ __forceinline__ uint32_t mxfp4_codes8(const float (&v)[8]) {
  uint32_t r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, v[0], v[1], 1.0f, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[2], v[3], 1.0f, 1);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[4], v[5], 1.0f, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[6], v[7], 1.0f, 3);
}

struct Mxfp4QuantArgs {
  const void* x;             // [rows][cols], contiguous
  long long groups;          // rows * cols / 8
  uint8_t* codes;            // [rows][cols / 2]
  uint8_t* scales;           // [rows][cols / 32]
};

// Largest of a quad's four values, by quad permutes.
__device__ __forceinline__ uint32_t mxfp4_quad_max(uint32_t v) {
  uint32_t o = __builtin_amdgcn_update_dpp(0, v, 0xB1, 0xF, 0xF, true);   // quad_perm 1,0,3,2
  v = o > v ? o : v;
  o = __builtin_amdgcn_update_dpp(0, v, 0x4E, 0xF, 0xF, true);            // quad_perm 2,3,0,1
  return o > v ? o : v;
}

template <int DT>
__device__ __forceinline__ void mxfp4_load8(const void* x, long long g, float (&v)[8]) {
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

// Quantises eight neighbouring values (group g); the four lanes of a block exchange their largest magnitude (as
// integer bits, so infinities and NaNs win): whole quads call it together.
template <int DT>
__device__ __forceinline__ void mxfp4_quantize_group(const Mxfp4QuantArgs& a, long long g) {
  float v[8];
  mxfp4_load8<DT>(a.x, g, v);
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t b = __float_as_uint(v[i]) & 0x7fffffffu;
    m = b > m ? b : m;
  }
  const uint32_t byte = mxfp4_scale_byte(mxfp4_quad_max(m));
  const float inv = mxfp4_inverse_scale(byte);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] *= inv;
  reinterpret_cast<uint32_t*>(a.codes)[g] = byte == 255u ? 0u : mxfp4_codes8(v);
  if ((threadIdx.x & 3) == 0) a.scales[g >> 2] = static_cast<uint8_t>(byte);
}

struct Mxfp4DequantArgs {
  const uint8_t* codes;
  const uint8_t* scales;
  long long groups;
  void* x;
};

// out[row][n] = sum_k X[row][k] W[n][k] over MXFP4 rows of K values. Dense: row tiles of the T rows.
// Grouped: tile i of the list holds rows [y, y + z) (slots) of expert x; X row of a slot:
// sorted[slot] / top_k (first product) or the slot itself (second).
struct Mxfp4GemmArgs {
  const uint16_t* x;         // first product of few routes, K <= kQuantizeInPlaceMax: bf16 [T][K] instead of xq, xs
  const uint8_t* xq;         // [rows][K / 2]
  const uint8_t* xs;         // [rows][K / 32]
  const uint8_t* wq;         // [N][K / 2] (times experts)
  const uint8_t* ws;         // [N][K / 32]
  int K, N;
  int rows;                  // dense: T
  const int4* gtiles;
  const int32_t* num_gtiles;
  int max_gtiles;
  const int32_t* sorted;     // first product: slot -> route
  const void* ids;           // few routes: [R] expert ids instead of a tile list (a slot is its route)
  int ids64, routes, experts;
  int top_k;
  void* y;                   // dense: [T][N] fp32 or bf16; second product: fp32 [slots][N]
  uint8_t* bq;               // first product: [slots][N / 4] codes of silu(gate) * up (N = 2I)
  uint8_t* bs;               // [slots][N / 64]
};

struct Mxfp4CombineArgs {
  const float* v;            // [slots][H]
  const int32_t* route_slot; // [T][k], -1 = dropped; null: a route's slot is the route itself, and
  const void* ids;           //   ids outside [0, experts) are dropped
  int ids64, experts;
  const float* w;            // [T][k]
  int tokens, top_k, H;
  void* y;                   // [T][H] fp32 or bf16
};

// dtype: TMOE_F32, TMOE_BF16 or TMOE_F16
void launch_mxfp4_quantize(const Mxfp4QuantArgs& a, int dtype, hipStream_t s);
// the route map and, in the same launch (extra workgroups, independent work), the bf16 input's quantisation
void launch_route_map_mxfp4(const RouteMapArgs& a, const Mxfp4QuantArgs& q, hipStream_t s);
void launch_mxfp4_dequantize(const Mxfp4DequantArgs& a, int dtype, hipStream_t s);
void launch_mxfp4_dense(const Mxfp4GemmArgs& a, int y_dtype, hipStream_t s);
// tile_rows: rows of the tile list's tiles, as mxfp4_tile_rows chose them; kFewRoutes: no list
void launch_mxfp4_fc1(const Mxfp4GemmArgs& a, int tile_rows, hipStream_t s);
void launch_mxfp4_fc2(const Mxfp4GemmArgs& a, int tile_rows, hipStream_t s);
void launch_mxfp4_combine(const Mxfp4CombineArgs& a, int y_dtype, hipStream_t s);
int mxfp4_tile_rows(long long routes, int experts);
constexpr int kFewRoutes = 1;
constexpr int kFewRoutesMax = 256;               // one id a thread
constexpr int kQuantizeInPlaceMax = 1024;

}  // namespace tmoe
