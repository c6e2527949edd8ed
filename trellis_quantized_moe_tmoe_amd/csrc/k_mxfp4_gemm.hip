// k_mxfp4_gemm.hip -- products of MXFP4 rows: the dense linear, the two grouped products of the
// expert layer, and the layer's weighted sum.
//
// v_mfma_scale_f32_16x16x128_f8f6f4 with both operands E2M1 takes one whole 32-value block a lane: lane
// l holds row (or column) l % 16, block l / 16 of the 128-deep step (16 bytes, as stored) and its scale
// byte. The weights are the first operand, so a lane's four results are four neighbouring output columns
// (4 (l / 16) + i) of one token (l % 16). Products are exact; sums are fp32.
#include <type_traits>

#include "tmoe.h"
#include "tmoe_mxfp4.hpp"

namespace tmoe {

namespace {

typedef int i4v __attribute__((ext_vector_type(4)));
typedef __bf16 bf4 __attribute__((ext_vector_type(4)));

enum { kDenseF32 = 0, kDenseBf16 = 1, kFc1 = 2, kFc2 = 3, kFc1Few = 4, kFc2Few = 5, kFc1FewX = 6 };

// One 128-deep product; byte BYTE of the scale words holds this lane's scales.
template <int BYTE>
__device__ __forceinline__ f4 mma_byte(i4v w, int ws, i4v x, int xs, f4 c) {
  const i8v a = __builtin_shufflevector(w, w, 0, 1, 2, 3, -1, -1, -1, -1);
  const i8v b = __builtin_shufflevector(x, x, 0, 1, 2, 3, -1, -1, -1, -1);
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 4, 4, BYTE, ws, BYTE, xs);
}
__device__ __forceinline__ f4 mma(int byte, i4v w, int ws, i4v x, int xs, f4 c) {   // byte: known once unrolled
  return byte == 0 ? mma_byte<0>(w, ws, x, xs, c)
       : byte == 1 ? mma_byte<1>(w, ws, x, xs, c)
       : byte == 2 ? mma_byte<2>(w, ws, x, xs, c) : mma_byte<3>(w, ws, x, xs, c);
}

// N (1, 2 or 4) neighbouring scale bytes, first one in byte 0.
template <int N>
__device__ __forceinline__ int load_scale_bytes(const uint8_t* p) {
  if constexpr (N == 1) {
    return *p;
  } else if constexpr (N == 2) {
    uint16_t v;
    __builtin_memcpy(&v, p, 2);
    return v;
  } else {
    uint32_t v;
    __builtin_memcpy(&v, p, 4);
    return static_cast<int>(v);
  }
}

// A block of 32 bf16 values in one lane -> its 32 codes; returns the scale byte.
__device__ __forceinline__ int quantize_block(const uint4 (&raw)[4], i4v& codes) {
  uint32_t w[16], m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w[4 * i] = raw[i].x;
    w[4 * i + 1] = raw[i].y;
    w[4 * i + 2] = raw[i].z;
    w[4 * i + 3] = raw[i].w;
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint32_t lo = (w[i] << 16) & 0x7fffffffu, hi = w[i] & 0x7fff0000u;
    m = max(m, max(lo, hi));
  }
  const uint32_t byte = mxfp4_scale_byte(m);
  const float inv = mxfp4_inverse_scale(byte);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float v[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = __uint_as_float(w[4 * i + j] << 16) * inv;
      v[2 * j + 1] = __uint_as_float(w[4 * i + j] & 0xffff0000u) * inv;
    }
    codes[i] = byte == 255u ? 0 : static_cast<int>(mxfp4_codes8(v));
  }
  return static_cast<int>(byte);
}

// Four neighbouring columns col.. of a row of N, at element `at` of y; columns past N are dropped. QUADS: N
// is a multiple of four, so a quad is whole and aligned.
template <bool BF16, bool QUADS>
__device__ __forceinline__ void store4(void* y, long long at, int col, int N, f4 v) {
  if constexpr (BF16) {
    uint16_t* o = static_cast<uint16_t*>(y) + at;
    if constexpr (QUADS) {                                 // both round to nearest even
      if (col < N) *reinterpret_cast<bf4*>(o) = __builtin_convertvector(v, bf4);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (col + i < N) o[i] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(v[i]));
    }
  } else {
    float* o = static_cast<float*>(y) + at;
    if constexpr (QUADS) {
      if (col < N) *reinterpret_cast<f4*>(o) = v;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (col + i < N) o[i] = v[i];
    }
  }
}

// x / (1 + exp(-x)) with the hardware's 2^y and reciprocal: off by one unit in the last place each, and for negative x by
// up to |x| half steps (2^-24) from the exponent's product, 17 of them at x = -20. The codes that follow are rounded by
// up to 2^-2 of their value, so this can only move a value that lies on the border of two codes.
__device__ __forceinline__ float silu(float x) {
  return x * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x * -1.44269504f));
}

// silu(g) * u, then the MXFP4 block of 32 neighbouring columns: a lane holds four of them in each of two
// fragments, the lanes 16 apart the others.
__device__ __forceinline__ void store_swiglu(const f4 (&g)[2], const f4 (&u)[2], uint8_t* bq, uint8_t* bs, int lane,
                                             bool store) {
  float h[8];
  uint32_t m = 0;
#pragma unroll
  for (int f = 0; f < 2; ++f)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      h[4 * f + i] = silu(g[f][i]) * u[f][i];
      const uint32_t b = __float_as_uint(h[4 * f + i]) & 0x7fffffffu;
      m = b > m ? b : m;
    }
  uint32_t o = __shfl_xor(m, 16, 64);
  m = o > m ? o : m;
  o = __shfl_xor(m, 32, 64);
  m = o > m ? o : m;
  const uint32_t byte = mxfp4_scale_byte(m);
  const float inv = mxfp4_inverse_scale(byte);
#pragma unroll
  for (int i = 0; i < 8; ++i) h[i] *= inv;
  const uint32_t c = byte == 255u ? 0u : mxfp4_codes8(h);
  if (store) {
    const int at = lane >> 4;
    reinterpret_cast<uint16_t*>(bq)[at] = static_cast<uint16_t>(c & 0xffffu);          // columns 4 at ..
    reinterpret_cast<uint16_t*>(bq)[4 + at] = static_cast<uint16_t>(c >> 16);          // columns 16 + 4 at ..
    if (at == 0) *bs = static_cast<uint8_t>(byte);
  }
}

// Few rows: a workgroup of KW wavefronts computes 16 MT rows by 16 NT columns straight from global memory,
// each wavefront every KW-th batch of K, their sums joined in LDS in a fixed order. What bounds it is the
// latency of a wavefront's loads, so they are issued AH 128-deep steps at a time (the weights first: they do not wait
// for the tile's routes) and, with TWO, the next batch before the products of the one before; the expert
// layer's products have many workgroups a CU instead, and few registers keep them there. A batch is 4 AH
// neighbouring blocks of every row; lane group q takes AH of them in a row, so that their scales are one
// load (a byte load for each block took a third of the first product's time at T = 16). Blocks past K repeat
// the last one with the scale 2^-127 on both sides (see the tiles below).
//
// kFc1Few, kFc2Few (up to kFewRoutesMax routes): there is no tile list. A workgroup stands for a route, finds
// the routes of that route's expert itself, one id a thread, and goes on if it is the 1st, 17th, ... of them,
// with the 16 from there on; slots are the routes. That saves the route map's launch (5.8 us of 35 at T = 16,
// k = 8, E = 96, H = 1024, I = 512).
//
// kFc1FewX: the input is bf16 and each workgroup quantises its tokens' rows itself, a block a lane, while the
// weights are on their way: another launch less (2.5 us), for rows of one batch (kQuantizeInPlaceMax).
template <int MODE, int MT, int NT, int KW, int AH, bool TWO>
__global__ __launch_bounds__(64 * KW, TWO ? 2 : MODE == kFc1FewX ? 4 : 5) void k_mxfp4_rows(Mxfp4GemmArgs a) {
  constexpr bool QX = MODE == kFc1FewX, FC1 = MODE == kFc1 || MODE == kFc1Few || QX;
  constexpr bool FEW = MODE == kFc1Few || MODE == kFc2Few || QX;
  static_assert(!FC1 || (NT == 4 && MT == 1), "first product: two gate and two up fragments");
  static_assert(!FEW || (KW * 64 == kFewRoutesMax && MT == 1), "one id a thread, tiles of 16 routes");
  __shared__ int list[FEW ? kFewRoutesMax : 1];
  __shared__ int first[FEW ? KW : 1], my_rank;
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, q = lane >> 4;
  // workgroups in x only (a tile's column groups next to each other): y and z are limited to 65535
  const int ngroups = FC1 ? a.N / 64 : (a.N + 16 * NT - 1) / (16 * NT);
  const int tile = blockIdx.x / ngroups, group = blockIdx.x % ngroups;
  int row0 = 0, nrows;
  long long expert = 0;
  if constexpr (FEW) {
    const int tid = threadIdx.x;
    long long id = -1;
    if (tid < a.routes) id = a.ids64 ? static_cast<const long long*>(a.ids)[tid] : static_cast<const int*>(a.ids)[tid];
    expert = a.ids64 ? static_cast<const long long*>(a.ids)[tile] : static_cast<const int*>(a.ids)[tile];
    if (expert < 0 || expert >= a.experts) return;           // the same for the whole workgroup
    const unsigned long long mine = __ballot(id == expert);
    if (lane == 0) first[wv] = __popcll(mine);
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int p = 0; p < KW; ++p) {
      if (p < wv) before += first[p];
      all += first[p];
    }
    const int rank = before + __popcll(mine & ((1ull << lane) - 1));
    if (id == expert) list[rank] = tid;
    if (tid == tile) my_rank = rank;
    __syncthreads();
    row0 = my_rank;                              // a tile's rows: list[row0 ..]
    nrows = min(16, all - row0);
    if (row0 % 16 != 0) return;
  } else if constexpr (MODE == kFc1 || MODE == kFc2) {
    const int count = *a.num_gtiles;
    const int4 t = a.gtiles[tile];               // tile < max_gtiles: inside the list, also past its count
    if (tile >= count) return;
    expert = t.x & 0xffffff;
    row0 = t.y;
    nrows = t.z;
  } else {
    row0 = tile * 16 * MT;
    nrows = min(16 * MT, a.rows - row0);
  }
  const int nblk = a.K / 32, batches = (nblk + 4 * AH - 1) / (4 * AH);
  const uint8_t* wq = a.wq + expert * a.N * (a.K / 2);
  const uint8_t* ws = a.ws + expert * a.N * nblk;

  const uint8_t *pq[NT], *ps[NT], *xq[MT], *xs[MT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    long long col;
    if constexpr (FC1) col = (n >> 1) * (a.N / 2) + 32 * group + 16 * (n & 1) + r;
    else col = min(16 * NT * group + 16 * n + r, a.N - 1);
    pq[n] = wq + col * (a.K / 2);
    ps[n] = ws + col * nblk;
  }
  struct Batch {
    i4v w[AH][NT], x[AH][MT];
    int ws[NT], xs[MT];
  };
  auto scale_word = [&](const uint8_t* p, int blk) -> int {   // K / 32 >= AH; bytes past K are 0
    const int from = min(blk, nblk - AH);
    const uint32_t v = static_cast<uint32_t>(load_scale_bytes<AH>(p + from)) >> (8 * min(blk - from, AH - 1));
    return blk < nblk ? static_cast<int>(v) : 0;
  };
  auto load_w = [&](int batch, Batch& b) {
    const int blk = 4 * AH * batch + AH * q;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int u = 0; u < AH; ++u) b.w[u][n] = reinterpret_cast<const i4v*>(pq[n])[min(blk + u, nblk - 1)];
      b.ws[n] = scale_word(ps[n], blk);
    }
  };
  auto load_x = [&](int batch, Batch& b) {
    const int blk = 4 * AH * batch + AH * q;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
#pragma unroll
      for (int u = 0; u < AH; ++u) b.x[u][m] = reinterpret_cast<const i4v*>(xq[m])[min(blk + u, nblk - 1)];
      b.xs[m] = scale_word(xs[m], blk);
    }
  };
  __shared__ f4 part[KW][MT * NT][64];
  Batch b0, b1;
  uint4 raw[QX ? AH : 1][4];                     // kFc1FewX: the lane's blocks of its token's row, in flight
  if constexpr (QX) {
    const int blk = 4 * AH * wv + AH * q;
    const uint16_t* row = a.x + static_cast<long long>(list[row0 + min(r, nrows - 1)] / a.top_k) * a.K;
#pragma unroll
    for (int u = 0; u < AH; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i) raw[u][i] = reinterpret_cast<const uint4*>(row)[4 * min(blk + u, nblk - 1) + i];
  }
  load_w(wv, b0);
  long long slot[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    slot[m] = FEW ? list[row0 + min(r, nrows - 1)] : row0 + min(16 * m + r, nrows - 1);
    long long row = slot[m];
    if constexpr (MODE == kFc1) row = a.sorted[row] / a.top_k;
    if constexpr (MODE == kFc1Few) row = row / a.top_k;
    xq[m] = a.xq + row * (a.K / 2);
    xs[m] = a.xs + row * nblk;
  }
  if constexpr (QX) {
    b0.xs[0] = 0;
#pragma unroll
    for (int u = 0; u < AH; ++u) {
      const int byte = quantize_block(raw[u], b0.x[u][0]);
      b0.xs[0] |= 4 * AH * wv + AH * q + u < nblk ? byte << (8 * u) : 0;
    }
  } else {
    load_x(wv, b0);
  }
  f4 acc[MT][NT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[m][n] = f4{0, 0, 0, 0};
  auto multiply = [&](const Batch& b) {
#pragma unroll
    for (int u = 0; u < AH; ++u)
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[m][n] = mma(u, b.w[u][n], b.ws[n], b.x[u][m], b.xs[m], acc[m][n]);
  };
  int at = wv;                                   // the batch in b0
  if constexpr (QX) {
    if (at < batches) multiply(b0);              // K <= 128 AH KW: there is no other batch
  } else if constexpr (TWO) {
    for (; at + KW < batches; at += 2 * KW) {
      load_w(at + KW, b1);
      load_x(at + KW, b1);
      multiply(b0);
      if (at + 2 * KW < batches) {
        load_w(at + 2 * KW, b0);
        load_x(at + 2 * KW, b0);
      }
      multiply(b1);
    }
    if (at < batches) multiply(b0);
  } else {
    while (at < batches) {
      multiply(b0);
      at += KW;
      if (at < batches) {
        load_w(at, b0);
        load_x(at, b0);
      }
    }
  }

  // join: fragment f of MT * NT belongs to wavefront f % KW (first product: all of them to wavefront 0)
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n) part[wv][m * NT + n][lane] = acc[m][n];
  __syncthreads();
  auto total = [&](int f) {
    f4 s = part[0][f][lane];
#pragma unroll
    for (int p = 1; p < KW; ++p) s += part[p][f][lane];
    return s;
  };
  if constexpr (FC1) {
    if (wv == 0) {
      const f4 g[2] = {total(0), total(1)}, u[2] = {total(2), total(3)};
      const int inter = a.N / 2;
      store_swiglu(g, u, a.bq + slot[0] * (inter / 2) + 16 * group, a.bs + slot[0] * (inter / 32) + group, lane,
                   r < nrows);
    }
  } else {
    for (int f = wv; f < MT * NT; f += KW) {
      const f4 s = total(f);
      const int m = f / NT, n = f % NT;
      const int col = 16 * NT * group + 16 * n + 4 * q;
      const long long to = (FEW ? slot[0] : row0 + 16 * m + r) * a.N + col;
      if (16 * m + r >= nrows) continue;
      if (a.N % 4 == 0) store4<MODE == kDenseBf16, true>(a.y, to, col, a.N, s);
      else store4<MODE == kDenseBf16, false>(a.y, to, col, a.N, s);
    }
  }
}

// ---------------------------------------------------------------- tiles through LDS
// A workgroup of four wavefronts computes 32 MT WT rows by 32 NT WC columns with
// v_mfma_scale_f32_32x32x64_f8f6f4: a lane holds row l % 32 of a fragment and one 16-byte block of it;
// in sub-step s of a 128-deep step the lanes of half h = l / 32 take block 2 h + s (the sum does not
// care which half takes which block), so a lane's two scale bytes of a step are neighbours.
//
// Codes go from global memory straight to LDS, 256 deep (a pair of steps) at a time into one of two slots: 128
// bytes a row, so that L2 is asked for whole lines (64-byte pieces, one step at a time into four slots,
// ran its channels at 60% of their requests: 45.9 us at T = 4096, K = N = 4096). The 16-byte chunk c of row r
// lies at place c ^ swizzle(r), so that the 16-byte reads of any 8 or 16 neighbouring rows touch every bank
// once; the copy writes LDS in lane order, so the swizzle is in the lane's global address. Scales come as 16
// bytes (four steps) a row, two buffers of them. Blocks past K repeat the codes of the last block and get
// the scale 2^-127 in both operands: their products, at most 36 * 2^-254 each, vanish in an fp32 sum.
//
// A step has two sub-steps of 64; each multiplies fragments that were read from LDS during the one
// before. One barrier a pair, in the middle of its second step: by then every wavefront has read all of the
// pair's slot, so the copies of the pair after the next go there.
typedef float f16v __attribute__((ext_vector_type(16)));

__device__ __forceinline__ int swizzle(int r) { return ((r >> 1) & 7) ^ ((r & 1) << 2); }

template <int SUB>
__device__ __forceinline__ f16v mma32(i4v w, int ws, i4v x, int xs, f16v c) {
  const i8v a = __builtin_shufflevector(w, w, 0, 1, 2, 3, -1, -1, -1, -1);
  const i8v b = __builtin_shufflevector(x, x, 0, 1, 2, 3, -1, -1, -1, -1);
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 4, 4, SUB, ws, SUB, xs);
}

template <int MODE, int WT, int WC, int MT, int NT>
struct Tile {
  static constexpr int TR = 32 * MT * WT, TC = 32 * NT * WC;      // rows (tokens) and columns
  static constexpr int kSlot = (TR + TC) * 128;                   // bytes of one slot
  static constexpr int kScales = (TR + TC) * 16;                  // bytes of one scale buffer
  static constexpr int kLds = 2 * kSlot + 2 * kScales;
  static constexpr int LPP = (TR + TC) / 32;                      // copies a wavefront issues a pair
  static constexpr int SPT = (TR + TC + 255) / 256;               // scale rows a thread stages
};

// silu(g) * u of 32 neighbouring columns of one token and their MXFP4 block: a lane holds the columns
// 8 i + 4 h + [0, 4), the lane 32 away the others.
__device__ __forceinline__ void store_swiglu32(const f16v& g, const f16v& u, uint8_t* bq, uint8_t* bs, int h, bool store) {
  float v[16];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    v[i] = silu(g[i]) * u[i];
    const uint32_t b = __float_as_uint(v[i]) & 0x7fffffffu;
    m = b > m ? b : m;
  }
  const uint32_t o = __shfl_xor(m, 32, 64);
  m = o > m ? o : m;
  const uint32_t byte = mxfp4_scale_byte(m);
  const float inv = mxfp4_inverse_scale(byte);
  uint32_t c[2];
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    float w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = v[8 * p + i] * inv;
    c[p] = byte == 255u ? 0u : mxfp4_codes8(w);
  }
  // half 0 stores columns 0..15, half 1 columns 16..31: each gives the other what it holds of them
  const uint32_t other = __shfl_xor(h ? c[0] : c[1], 32, 64);
  const uint32_t own = h ? c[1] : c[0];
  const uint32_t even = h ? other : own, odd = h ? own : other;   // columns 8 i + [0, 4) and 8 i + [4, 8)
  if (store) {
    reinterpret_cast<uint2*>(bq)[h] = make_uint2((even & 0xffffu) | (odd << 16), (even >> 16) | (odd & 0xffff0000u));
    if (h == 0) *bs = static_cast<uint8_t>(byte);
  }
}

// ALIGNED: K is a multiple of 128 and at least 512 and the scales are 4-byte aligned. Their rows are then copied
// straight to LDS like the codes; else they pass through registers, where the compiler's wait for them is one
// for every copy in flight.
//
// next: gives the workgroup's next tile, until there is none (NoNext: at once). The ring does not stop between two
// tiles: the copies of a tile's last group are the first two pairs of the next tile, and land while the results
// are stored.
struct TileAt {
  long long expert;
  int row0, nrows, cg;
};
struct NoNext {
  __device__ bool operator()(TileAt&) const { return false; }
};

template <int MODE, int WT, int WC, int MT, int NT, bool ALIGNED, class Next>
__device__ __forceinline__ void tile_body(const Mxfp4GemmArgs& a, TileAt t, Next next, uint8_t* lds) {
  constexpr bool STREAM = !std::is_same<Next, NoNext>::value;
  static_assert((ALIGNED && MODE == kFc1) || !STREAM, "its scales are copies and its results need no LDS");
  using S = Tile<MODE, WT, WC, MT, NT>;
  static_assert(WT * WC == 4 && (MODE != kFc1 || NT == 2), "four wavefronts; first product: gate and up fragment");
  const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r32 = lane & 31, h = lane >> 5;
  const int wt = wv / WC, wc = wv % WC;
  const int nblk = a.K / 32, steps = (nblk + 3) / 4;
  const int inter = a.N / 2;

  // Rows of a tile: tokens first, then weight rows; rows past the end repeat the last one. A token's row of the first
  // product is behind its route (route_of), which is read apart; route / k by the reciprocal ceil(2^32 / k),
  // exact for routes below 2^27 (k <= 32).
  const uint32_t recip = MODE == kFc1 ? 0xffffffffu / static_cast<uint32_t>(a.top_k) + 1u : 0u;   // k = 1: wraps to 0
  auto route_of = [&](const TileAt& t, int i) -> int {
    if constexpr (MODE == kFc1) return a.sorted[t.row0 + min(i, t.nrows - 1)];
    else return 0;
  };
  auto token_row = [&](const TileAt& t, int i, int route) -> uint32_t {
    if constexpr (MODE == kFc1) return __umulhi(static_cast<uint32_t>(route), recip) + (recip ? 0u : route);
    else return t.row0 + min(i, t.nrows - 1);
  };
  auto weight_row = [&](const TileAt& t, int j) -> uint32_t {          // of all experts: below 2^24
    uint32_t col;
    if constexpr (MODE == kFc1) col = ((j >> 5) & 1) * inter + min(t.cg * (S::TC / 2) + (j >> 6) * 32 + (j & 31), inter - 1);
    else col = min(t.cg * S::TC + j, a.N - 1);
    return static_cast<uint32_t>(t.expert) * a.N + col;
  };
  auto scales_at = [&](const TileAt& t, int i, int route) -> const uint8_t* {
    const bool tok = i < S::TR;
    const uint32_t row = tok ? token_row(t, i, route) : weight_row(t, i - S::TR);
    return (tok ? a.xs : a.ws) + static_cast<unsigned long long>(row) * static_cast<uint32_t>(nblk);
  };
  // copies in the order weights, tokens: a token's address may wait for its route
  const uint8_t* src[S::LPP];
  auto place_of = [&](int i) { return wv + 4 * (i < S::TC / 32 ? S::TR / 32 + i : i - S::TC / 32); };
  auto code_row = [&](int i) { return 8 * place_of(i) + (lane >> 3); };
  auto scale_row = [&](int i) {
    return ALIGNED ? 64 * min(wv + 4 * i, (S::TR + S::TC) / 64 - 1) + lane : min(tid + 256 * i, S::TR + S::TC - 1);
  };
  const uint8_t* ssrc[S::SPT];
  int route[S::LPP], sroute[S::SPT];
  auto read_routes = [&](const TileAt& t) {
#pragma unroll
    for (int i = 0; i < S::LPP; ++i) route[i] = i < S::TC / 32 ? 0 : route_of(t, code_row(i));
#pragma unroll
    for (int i = 0; i < S::SPT; ++i) sroute[i] = route_of(t, scale_row(i));
  };
  auto point_at = [&](const TileAt& t) {
    const uint32_t pitch = a.K / 2;
#pragma unroll
    for (int i = 0; i < S::LPP; ++i) {
      if (i < S::TC / 32) src[i] = a.wq + static_cast<unsigned long long>(weight_row(t, code_row(i) - S::TR)) * pitch;
      else src[i] = a.xq + static_cast<unsigned long long>(token_row(t, code_row(i), route[i])) * pitch;
    }
#pragma unroll
    for (int i = 0; i < S::SPT; ++i) ssrc[i] = ALIGNED || nblk >= 16 ? scales_at(t, scale_row(i), sroute[i]) : a.wq;
  };
  read_routes(t);
  point_at(t);
  const int chunk = (lane & 7) ^ swizzle(8 * (wv & 1) + (lane >> 3));

  auto issue = [&](int pair, int i) {            // one of a wavefront's LPP copies (8 rows) of a pair of steps
    const int blk = min(8 * pair + chunk, nblk - 1);
    __builtin_amdgcn_global_load_lds(
        (const void __attribute__((address_space(1)))*)(src[i] + 16 * blk),
        (void __attribute__((address_space(3)))*)(lds + (pair & 1) * S::kSlot + place_of(i) * 1024), 16, 0, 0);
  };
  // Scales of steps 4 g .. 4 g + 3: bytes 16 g .. of each row. The last group's load starts where it ends with
  // the row and is shifted when it is stored; rows shorter than 16 bytes have one
  // group, read before the loop (the loop's fetches then read 16 bytes of codes for nothing).
  int buffer = 0;                                // scale buffer of group 0
  auto copy_scales = [&](int g, int b) {         // ALIGNED: 64 rows of 16 bytes a copy, repeats at the end
    const int from = min(16 * g, nblk - 16);
#pragma unroll
    for (int i = 0; i < S::SPT; ++i)
      __builtin_amdgcn_global_load_lds(
          (const void __attribute__((address_space(1)))*)(ssrc[i] + from),
          (void __attribute__((address_space(3)))*)(lds + 2 * S::kSlot + (b & 1) * S::kScales +
                                                    min(wv + 4 * i, (S::TR + S::TC) / 64 - 1) * 1024),
          16, 0, 0);
  };
  uint4 sreg[S::SPT];
  auto load_scales = [&](int g) {
    const int from = nblk >= 16 ? min(16 * g, nblk - 16) : 0;
#pragma unroll
    for (int i = 0; i < S::SPT; ++i) __builtin_memcpy(&sreg[i], ssrc[i] + from, 16);
  };
  auto store_scales = [&](int g) {               // no branches: the loop body stays one block
    uint8_t* buf = lds + 2 * S::kSlot + (g & 1) * S::kScales;
    const int by = max(16 * g - (nblk - 16), 0);   // bytes to shift out: 8 and 4 by masks, the rest by alignbyte
    uint32_t keep[2] = {by & 8 ? 0u : ~0u, by & 4 ? 0u : ~0u};
    asm("" : "+v"(keep[0]), "+v"(keep[1]));      // opaque: selects on a known condition become branches
#pragma unroll
    for (int i = 0; i < S::SPT; ++i) {
      uint32_t w[4] = {sreg[i].x, sreg[i].y, sreg[i].z, sreg[i].w};
#pragma unroll
      for (int d = 2; d; d >>= 1)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint32_t m = keep[2 - d];
          w[q] = (w[q] & m) | (q + d < 4 ? w[q + d] & ~m : 0u);
        }
      const uint32_t b = by & 3;
      reinterpret_cast<uint4*>(buf)[min(tid + 256 * i, S::TR + S::TC - 1)] =
          make_uint4(__builtin_amdgcn_alignbyte(w[1], w[0], b), __builtin_amdgcn_alignbyte(w[2], w[1], b),
                     __builtin_amdgcn_alignbyte(w[3], w[2], b), __builtin_amdgcn_alignbyte(0u, w[3], b));
    }
  };
  auto first_scales = [&]() {
    if (nblk >= 16) {
      load_scales(0);
      store_scales(0);
      return;
    }
    // rows of less than 16 bytes: 16 bytes that lie in the array, shifted to the row's first and cut behind its last
    const long long tokens = MODE == kFc1 ? a.routes / a.top_k : MODE == kFc2 ? a.routes : a.rows;
    const uint8_t* x_end = a.xs + tokens * nblk;
    const uint8_t* ws = a.ws + t.expert * a.N * nblk;
    const uint8_t* w_end = ws + static_cast<long long>(a.N) * nblk;    // the expert's own rows
    uint8_t* buf = lds + 2 * S::kSlot;
#pragma unroll
    for (int i = 0; i < S::SPT; ++i) {
      const int at = min(tid + 256 * i, S::TR + S::TC - 1);
      const uint8_t* p = scales_at(t, at, route_of(t, at));
      const uint8_t* end = at < S::TR ? x_end : w_end;
      uint32_t w[4] = {0, 0, 0, 0};
      if (end - (at < S::TR ? a.xs : ws) >= 16) {
        const uint8_t* from = p + 16 <= end ? p : end - 16;
        const int by = static_cast<int>(p - from);
        __builtin_memcpy(w, from, 16);
#pragma unroll
        for (int d = 2; d; d >>= 1)
#pragma unroll
          for (int q = 0; q < 4; ++q) w[q] = by & (4 * d) ? (q + d < 4 ? w[q + d] : 0u) : w[q];
        const uint32_t b = by & 3;
#pragma unroll
        for (int q = 0; q < 4; ++q) w[q] = __builtin_amdgcn_alignbyte(q < 3 ? w[q + 1] : 0u, w[q], b);
      } else {
#pragma unroll
        for (int b = 0; b < 15; ++b) w[b >> 2] |= static_cast<uint32_t>(p[min(b, nblk - 1)]) << (8 * (b & 3));
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int have = max(0, min(4, nblk - 4 * q));
        w[q] = have == 4 ? w[q] : w[q] & ((1u << (8 * have)) - 1u);
      }
      reinterpret_cast<uint4*>(buf)[at] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  };

  struct Frags {                                 // one sub-step
    i4v x[MT], w[NT];
  };
  const int place = swizzle(r32);
  int lane_at[4];                                // chunk 4 (ks & 1) + 2 h + s of a row, by 2 (ks & 1) + s
#pragma unroll
  for (int i = 0; i < 4; ++i) lane_at[i] = 128 * r32 + 16 * ((4 * (i >> 1) + 2 * h + (i & 1)) ^ place);
  // Piece p of MT + NT reads one fragment of sub-step s of step ks (and, with SCALES, its scales): the columns
  // first, which every matrix instruction of the first row needs.
  int xs[MT], ws4[NT], nx[MT], nw[NT];
  auto read_piece = [&](int ks, int s, int p, Frags& f, bool scales) {
    const uint8_t* slot = lds + ((ks >> 1) & 1) * S::kSlot + lane_at[2 * (ks & 1) + s];
    // ALIGNED: the last group's bytes start where they end with the row
    const int at = ALIGNED ? min(4 * ks - min(16 * (ks >> 2), nblk - 16), 12) : 4 * (ks & 3);
    const uint8_t* sc = lds + 2 * S::kSlot + ((buffer + (ks >> 2)) & 1) * S::kScales + 16 * r32 + at + 2 * h;
    if (p < NT) {
      f.w[p] = *reinterpret_cast<const i4v*>(slot + 128 * S::TR + 4096 * (wc * NT + p));
      if (scales) nw[p] = *reinterpret_cast<const uint16_t*>(sc + 16 * S::TR + 512 * (wc * NT + p));
    } else {
      const int m = p - NT;
      f.x[m] = *reinterpret_cast<const i4v*>(slot + 4096 * (wt * MT + m));
      if (scales) nx[m] = *reinterpret_cast<const uint16_t*>(sc + 512 * (wt * MT + m));
    }
  };

  f16v acc[MT][NT];

  if constexpr (ALIGNED) copy_scales(0, 0);
  else first_scales();
#pragma unroll
  for (int d = 0; d < 2; ++d)
#pragma unroll
    for (int i = 0; i < S::LPP; ++i) issue(d, i);
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(S::LPP) : "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  Frags f0, f1;
#pragma unroll
  for (int p = 0; p < MT + NT; ++p) read_piece(0, 0, p, f0, true);

  // Copies past the last step repeat its last block and reads of step `steps` see one of those: neither is
  // used, and every step looks the same. PHASE: ks % 4; the next group's scales are fetched during step 0
  // and stored during step 2. The order within a step is pinned, one or two reads or a copy in front of each
  // matrix instruction: a wavefront has its SIMD to itself and issues in order, so what does not fit under
  // the 32 cycles of the instruction before is lost (four of them behind a bunch of reads and copies: 52.9 us
  // at T = 4096, K = N = 4096; left free, the compiler gathers the matrix instructions of four steps).
  constexpr int MM = MT * NT, RD = MT + NT;
  const int groups = (steps + 3) / 4;            // whole groups of four: steps past K add nothing
  // LAST: the group's copies are those of the next tile (its pairs 0 and 1, its scale group 0), to which src points
  auto step = [&](int ks, auto phase, auto last) {
    constexpr int PHASE = decltype(phase)::value;
    constexpr bool LAST = decltype(last)::value;
    const int mask = !ALIGNED || 4 * ks < nblk ? 0xffff : 0;   // ALIGNED: steps past K read any scale
#pragma unroll
    for (int m = 0; m < MT; ++m) xs[m] = nx[m] & mask;
#pragma unroll
    for (int n = 0; n < NT; ++n) ws4[n] = nw[n] & mask;
    if constexpr (PHASE == 0 && ALIGNED) copy_scales(LAST ? 0 : (ks >> 2) + 1, buffer + (ks >> 2) + 1);
    if constexpr (PHASE == 0 && !ALIGNED) load_scales((ks >> 2) + 1);
    if constexpr (PHASE == 2 && !ALIGNED) store_scales((ks >> 2) + 1);
#pragma unroll
    for (int j = 0; j < MM; ++j) {
      constexpr int per = (RD + MM - 1) / MM;    // reads in front of one instruction
#pragma unroll
      for (int p = j * per; p < (j + 1) * per && p < RD; ++p) read_piece(ks, 1, p, f1, false);
      __builtin_amdgcn_sched_barrier(0);
      acc[j / NT][j % NT] = mma32<0>(f0.w[j % NT], ws4[j % NT], f0.x[j / NT], xs[j / NT], acc[j / NT][j % NT]);
      __builtin_amdgcn_sched_barrier(0);
    }
    // Second step of a pair: the next pair has landed (the only newer copies are those of the scales, issued
    // in step 0 of the group; step 3's wait covers them) and this wavefront's LDS accesses are done. Behind
    // the barrier that holds for all four wavefronts: this pair's slot is free.
    if constexpr (PHASE & 1) {
      asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(ALIGNED && PHASE == 1 ? S::SPT : 0) : "memory");
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
    }
    if constexpr (LAST && PHASE == 3) buffer = (buffer + groups) & 1;
#pragma unroll
    for (int j = 0; j < MM; ++j) {
      constexpr int per = (RD + MM - 1) / MM;
#pragma unroll
      for (int p = j * per; p < (j + 1) * per && p < RD; ++p) {
        if constexpr (LAST && PHASE == 3) read_piece(0, 0, p, f0, true);   // buffer: the next tile's by now
        else read_piece(ks + 1, 0, p, f0, true);
      }
      if constexpr (PHASE & 1) {
#pragma unroll
        for (int i = j * S::LPP / MM; i < (j + 1) * S::LPP / MM; ++i) issue(LAST ? PHASE >> 1 : (ks >> 1) + 2, i);
      }
      __builtin_amdgcn_sched_barrier(0);
      acc[j / NT][j % NT] = mma32<1>(f1.w[j % NT], ws4[j % NT], f1.x[j / NT], xs[j / NT], acc[j / NT][j % NT]);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  auto store_tile = [&](const TileAt& t) {
    if constexpr (MODE == kFc1) {
      const int col = t.cg * (S::TC / 2) + 32 * wc;
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const int i = 32 * (wt * MT + m) + r32;
        const long long row = t.row0 + i;
        if constexpr (STREAM) __builtin_amdgcn_sched_barrier(0);
        store_swiglu32(acc[m][0], acc[m][1], a.bq + row * (inter / 2) + col / 2, a.bs + row * (inter / 32) + col / 32, h,
                       i < t.nrows && col < inter);
      }
    } else {
      // Rows of y are written whole: 32 rows at a time pass through the wavefront's own part of the ring (rows
      // padded by 16 bytes), so that a store covers 256 or 512 neighbouring bytes of a row (8- or 16-byte
      // pieces straight from the registers: 22 us of the 52.9 at T = 4096, K = N = 4096).
      constexpr bool BF = MODE == kDenseBf16;
      constexpr int ES = BF ? 2 : 4, EPL = 16 / ES, PITCH = 32 * NT * ES + 16;
      static_assert(4 * 32 * PITCH <= S::kLds, "four wavefronts' rows fit the ring");
      const int col0 = t.cg * S::TC + 32 * NT * wc;
      if (a.N % EPL == 0) {
        __syncthreads();                           // every wavefront has read its last fragments
        uint8_t* mine = lds + wv * 32 * PITCH;
#pragma unroll
        for (int m = 0; m < MT; ++m) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const f4 v = {acc[m][n][4 * q], acc[m][n][4 * q + 1], acc[m][n][4 * q + 2], acc[m][n][4 * q + 3]};
              uint8_t* to = mine + r32 * PITCH + (32 * n + 8 * q + 4 * h) * ES;
              if constexpr (BF) *reinterpret_cast<bf4*>(to) = __builtin_convertvector(v, bf4);
              else *reinterpret_cast<f4*>(to) = v;
            }
          __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
          constexpr int LPR = 32 * NT / EPL, RPI = 64 / LPR;     // lanes a row, rows a store
          const int c = col0 + (lane % LPR) * EPL;
#pragma unroll
          for (int i = 0; i < 32 / RPI; ++i) {
            const int r = RPI * i + lane / LPR, row = 32 * (wt * MT + m) + r;
            const i4v v = *reinterpret_cast<const i4v*>(mine + r * PITCH + (lane % LPR) * 16);
            if (row < t.nrows && c < a.N)
              *reinterpret_cast<i4v*>(static_cast<uint8_t*>(a.y) + (static_cast<long long>(t.row0 + row) * a.N + c) * ES) = v;
          }
          __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        }
        return;
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const int i = 32 * (wt * MT + m) + r32;
        const long long row = static_cast<long long>(t.row0 + i) * a.N;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int col = col0 + 32 * n + 8 * q + 4 * h;
            const f4 v = {acc[m][n][4 * q], acc[m][n][4 * q + 1], acc[m][n][4 * q + 2], acc[m][n][4 * q + 3]};
            if (i < t.nrows) store4<BF, false>(a.y, row + col, col, a.N, v);
          }
      }
    }
  };
  auto four = [&](int ks, auto last) {
    step(ks, std::integral_constant<int, 0>{}, last);
    step(ks + 1, std::integral_constant<int, 1>{}, last);
    step(ks + 2, std::integral_constant<int, 2>{}, last);
    step(ks + 3, std::integral_constant<int, 3>{}, last);
  };
  for (;;) {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n) acc[m][n] = f16v{};
    bool more = false;
    if constexpr (STREAM) {
      TileAt then = t;
      more = next(then);                         // without a next tile the copies repeat this one's
      read_routes(then);                         // used a group later
      __builtin_amdgcn_sched_barrier(0);
      int g = 0;                                 // K is more than 512: at least two groups
      do four(4 * g, std::false_type{});
      while (++g + 1 < groups);
      point_at(then);
      four(4 * g, std::true_type{});
#pragma unroll
      for (int m = 0; m < MT; ++m)               // opaque: else products sink into the branches of the stores
#pragma unroll
        for (int n = 0; n < NT; ++n) asm volatile("" : "+v"(acc[m][n]));
      store_tile(t);
      __builtin_amdgcn_sched_barrier(0);
      t = then;
    } else {
      for (int g = 0; g < groups; ++g) four(4 * g, std::false_type{});
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // the copies past the end land before LDS is given up
      store_tile(t);
    }
    if (!more) break;
  }
  if constexpr (STREAM) asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

// Dense: row tiles by column tiles in groups of eight row tiles, a contiguous run of them to each of the
// eight XCDs (workgroups are dealt to the XCDs in turn), so that an XCD's L2 holds what its tiles share.
template <int MODE, int WT, int WC, int MT, int NT, bool ALIGNED>
__global__ __launch_bounds__(256, MT * NT > 8 ? 1 : 2) void k_mxfp4_tile_dense(Mxfp4GemmArgs a, int row_tiles, int col_tiles) {
  using S = Tile<MODE, WT, WC, MT, NT>;
  __shared__ __align__(16) uint8_t lds[S::kLds];
  const int total = row_tiles * col_tiles, per = gridDim.x / 8;
  const int t = (blockIdx.x % 8) * per + blockIdx.x / 8;
  if (t >= total) return;
  constexpr int G = 8;
  const int g = t / (G * col_tiles), in = t % (G * col_tiles);
  const int rows_g = min(G, row_tiles - g * G);
  const int rt = g * G + in % rows_g, ct = in / rows_g;
  const int row0 = rt * S::TR;
  tile_body<MODE, WT, WC, MT, NT, ALIGNED>(a, TileAt{0, row0, min(S::TR, a.rows - row0), ct}, NoNext{}, lds);
}

// Grouped: tiles of up to 128 rows of one expert by 128 columns (first product: 64 gate and 64 up). A tile's
// column blocks go to one XCD, which then reads its rows once; fewer than eight tiles therefore keep as few XCDs busy
// (E = 1, H = 4096, I = 8192: 31 us for the layer with 10 routes, without a tile list, 67 with 11). Tiles of at most 64
// rows run with half the row fragments; the tile list holds them last.
template <int MODE, bool ALIGNED>
__global__ __launch_bounds__(256, 2) void k_mxfp4_tile_grouped(Mxfp4GemmArgs a, int col_tiles) {
  using S = Tile<MODE, 2, 2, 2, 2>;
  __shared__ __align__(16) uint8_t lds[S::kLds];
  const int i = blockIdx.x / 8;
  const int tile = i / col_tiles * 8 + blockIdx.x % 8, ct = i % col_tiles;
  const int4 t = a.gtiles[min(tile, a.max_gtiles - 1)];      // read beside the count, not after it
  if (tile >= *a.num_gtiles) return;
  const long long expert = t.x & 0xffffff;
  if (t.z > 64) tile_body<MODE, 2, 2, 2, 2, ALIGNED>(a, TileAt{expert, t.y, t.z, ct}, NoNext{}, lds);
  else tile_body<MODE, 2, 2, 1, 2, ALIGNED>(a, TileAt{expert, t.y, t.z, ct}, NoNext{}, lds);
}

// First product, K > 512, more workgroups in the grouped launch (room for the largest tile list, in whole eights) than
// run at once: the same tiles by a fixed number of workgroups, two a CU, each of which walks over its XCD's tiles
// without stopping the ring (H = 1024, I = 512, E = 96, k = 8: T = 2048 the layer 82.3 -> 77.7 us, T = 8192 this product
// 94.9 -> 74.9, T = 700 18.0 -> 17.2; with 384 tiles, one each, 13.7 -> 15.6). The layer on other geometries, streaming
// and one each: H = 2048, I = 768, E = 16, k = 2, T = 2048 (576 workgroups) 55.4 and 54.5, T = 8192 (1728) 146.7 and
// 149.2; H = 4096, I = 1024, E = 8, k = 2, T = 2048 (640) 96.6 and 95.2, T = 8192 (2176) 322.7 and 325.7. All tiles run
// with all row fragments here, short ones too. The second product's results need the ring's LDS on their way out; with 8 KB of their own instead the layer took 80.6.
constexpr unsigned kStreamGroups = 512;

__global__ __launch_bounds__(256, 2) void k_mxfp4_tile_stream(Mxfp4GemmArgs a, int col_tiles) {
  using S = Tile<kFc1, 2, 2, 2, 2>;
  __shared__ __align__(16) uint8_t lds[S::kLds];
  const int count = *a.num_gtiles, xcd = blockIdx.x % 8;
  const int items = count > xcd ? (count - xcd + 7) / 8 * col_tiles : 0;
  int at = blockIdx.x / 8;
  if (at >= items) return;
  auto tile = [&](int at) {
    // below the count: at < items. Constant address space (the list is of an earlier launch): a scalar load, which
    // waits for no copy in flight.
    const i4v t = reinterpret_cast<const __attribute__((address_space(4))) i4v*>(
        reinterpret_cast<uintptr_t>(a.gtiles))[at / col_tiles * 8 + xcd];
    return TileAt{t[0] & 0xffffff, t[1], t[2], at % col_tiles};
  };
  auto next = [&](TileAt& t) {
    at += gridDim.x / 8;
    if (at >= items) return false;
    t = tile(at);
    return true;
  };
  tile_body<kFc1, 2, 2, 2, 2, true>(a, tile(at), next, lds);
}

// y_t = sum over j ascending of w[t][j] * v[slot of (t, j)], four columns a thread; eight rows' loads in
// flight (one after the other: 6.5 us at T = 16, k = 8).
template <bool BF16>
__global__ __launch_bounds__(256) void k_mxfp4_combine(Mxfp4CombineArgs a) {
  const int quads = a.H / 4;
  const long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= static_cast<long long>(a.tokens) * quads) return;
  const long long t = i / quads;
  const int c = static_cast<int>(i - t * quads);
  f4 s = {0, 0, 0, 0};
  for (int j0 = 0; j0 < a.top_k; j0 += 8) {
    long long slot[8];
    float w[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const long long r = t * a.top_k + min(j0 + u, a.top_k - 1);
      w[u] = a.w[r];
      if (a.route_slot) {
        slot[u] = a.route_slot[r];
      } else {
        const long long id = a.ids64 ? static_cast<const long long*>(a.ids)[r] : static_cast<const int*>(a.ids)[r];
        slot[u] = id >= 0 && id < a.experts ? r : -1;
      }
      if (j0 + u >= a.top_k) slot[u] = -1;
    }
    f4 v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (slot[u] >= 0) v[u] = reinterpret_cast<const f4*>(a.v + slot[u] * a.H)[c];
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (slot[u] >= 0) s += w[u] * v[u];
  }
  if constexpr (BF16)
    static_cast<bf4*>(a.y)[i] = __builtin_convertvector(s, bf4);
  else
    static_cast<f4*>(a.y)[i] = s;
}

}  // namespace

// Rows of a tile of the expert layer: 16 while experts hold a few rows each (straight from global memory; up to
// kFewRoutesMax routes without a tile list), else 128 (through LDS). The layer with a tile list, 16-row and 128-row
// tiles (us), at 6, 10, 12, 16 and 24 routes an expert:
//   H = 1024, I = 512, E = 96, k = 8     32.1 34.6   35.0 35.6   36.6 37.3   40.5 37.3   50.8 40.6
//   H = 1024, I = 512, E = 256, k = 8    67.3 67.4   74.0 71.3   77.3 72.0   90.2 76.3   110.9 79.3
//   H = 2560, I = 320, E = 128, k = 10   54.6 69.4   59.7 72.7   61.8 73.0   72.7 75.3   89.8 80.9
//   H = 2048, I = 768, E = 16, k = 2 (16 and 24)                             27.2 23.8   31.4 24.6
int mxfp4_tile_rows(long long routes, int experts) {
  if (routes > 10LL * experts) return 128;
  return routes <= kFewRoutesMax ? kFewRoutes : 16;
}

bool scales_aligned(const Mxfp4GemmArgs& a) {
  return a.K % 128 == 0 && a.K >= 512 &&
         ((reinterpret_cast<uintptr_t>(a.xs) | reinterpret_cast<uintptr_t>(a.ws)) & 3) == 0;
}

template <int MODE, int MT, int NT>
void launch_tiles(const Mxfp4GemmArgs& a, hipStream_t s) {
  using S = Tile<MODE, 2, 2, MT, NT>;
  const int rt = (a.rows + S::TR - 1) / S::TR, ct = (a.N + S::TC - 1) / S::TC;
  const dim3 g((rt * ct + 7) / 8 * 8);
  if (scales_aligned(a)) hipLaunchKernelGGL((k_mxfp4_tile_dense<MODE, 2, 2, MT, NT, true>), g, dim3(256), 0, s, a, rt, ct);
  else hipLaunchKernelGGL((k_mxfp4_tile_dense<MODE, 2, 2, MT, NT, false>), g, dim3(256), 0, s, a, rt, ct);
}

template <int MODE, int MT, int NT, int AH>
void launch_rows(const Mxfp4GemmArgs& a, hipStream_t s) {
  const int groups = (a.N + 16 * NT - 1) / (16 * NT), tiles = (a.rows + 16 * MT - 1) / (16 * MT);
  hipLaunchKernelGGL((k_mxfp4_rows<MODE, MT, NT, 8, AH, true>), dim3(groups * tiles), dim3(512), 0, s, a);
}

// The shape of the dense product, by the number of 128 x 128 tiles (us; K = 4096 unless said):
//   T <= 64         wavefronts that split K (T = 48, N = 1024: 7.6, 64 x 128 tiles 8.5; K = 2560: 5.1 and 6.4;
//                   T = 17 and 64, N = 4096: 5.2 and 9.1, tiles 8.5 and 9.4). Each 16 columns read all of X again: with
//                   N = 16384 tiles would be faster (T = 17 and 64: 14.2 and 32.2, tiles 12.6 and 13.2)
//   up to 160 tiles 64 x 128, two workgroups a CU (T = 400, N = 4096: 9.5; 128 x 128 11.6, 256 x 256 26.5)
//   up to 512 tiles 128 x 128, two workgroups a CU (T = 1600, N = 4096: 23.4; 64 x 128 33.5, 256 x 256 30.6)
//   more            256 x 256, one workgroup a CU: half the LDS traffic for each product (T = 3200, N = 4096:
//                   36.8; 128 x 128 46.4)
template <int MODE>
void launch_dense(const Mxfp4GemmArgs& a, hipStream_t s) {
  const long long tiles = ((a.rows + 127LL) / 128) * ((a.N + 127) / 128);
  if (a.rows <= 64 && a.K >= 128) {              // they read four or two neighbouring scales
    if (a.rows <= 16) launch_rows<MODE, 1, 1, 4>(a, s);
    else if (a.rows <= 32) launch_rows<MODE, 2, 1, 2>(a, s);
    else launch_rows<MODE, 4, 1, 2>(a, s);
  } else if (tiles <= 160) {
    launch_tiles<MODE, 1, 2>(a, s);
  } else if (tiles <= 512) {
    launch_tiles<MODE, 2, 2>(a, s);
  } else {
    launch_tiles<MODE, 4, 4>(a, s);
  }
}

void launch_mxfp4_dense(const Mxfp4GemmArgs& a, int y_dtype, hipStream_t s) {
  if (y_dtype == TMOE_BF16) launch_dense<kDenseBf16>(a, s);
  else launch_dense<kDenseF32>(a, s);
}

// Few rows an expert: one 128-deep step a wavefront and batch up to K = 512, two up to K = 1024 (one batch), two and
// the next batch ahead beyond (H = 2560, T = 16: 25.6 -> 22.5 us; one batch: 13.5 -> 15.3 with it).
template <int MODE>
void launch_few_rows(const Mxfp4GemmArgs& a, int tiles, hipStream_t s) {
  const dim3 g((a.N + 63) / 64 * tiles), b(256);
  if (a.K <= 512) hipLaunchKernelGGL((k_mxfp4_rows<MODE, 1, 4, 4, 1, false>), g, b, 0, s, a);
  else if (a.K <= 1024) hipLaunchKernelGGL((k_mxfp4_rows<MODE, 1, 4, 4, 2, false>), g, b, 0, s, a);
  else hipLaunchKernelGGL((k_mxfp4_rows<MODE, 1, 4, 4, 2, true>), g, b, 0, s, a);
}

template <int MODE>
void launch_grouped(const Mxfp4GemmArgs& a, int tile_rows, hipStream_t s) {
  if (tile_rows == kFewRoutes) {
    if constexpr (MODE == kFc1) {
      if (a.x) {
        const dim3 g(a.N / 64 * a.routes), b(256);
        if (a.K <= 512) hipLaunchKernelGGL((k_mxfp4_rows<kFc1FewX, 1, 4, 4, 1, false>), g, b, 0, s, a);
        else hipLaunchKernelGGL((k_mxfp4_rows<kFc1FewX, 1, 4, 4, 2, false>), g, b, 0, s, a);
        return;
      }
    }
    return launch_few_rows<MODE == kFc1 ? kFc1Few : kFc2Few>(a, a.routes, s);
  }
  if (tile_rows == 16) return launch_few_rows<MODE>(a, a.max_gtiles, s);
  const int ct = (a.N + 127) / 128;
  const dim3 g((a.max_gtiles + 7) / 8 * 8 * ct);
  if (MODE == kFc1 && a.K > 512 && g.x > kStreamGroups && scales_aligned(a)) {
    hipLaunchKernelGGL(k_mxfp4_tile_stream, dim3(kStreamGroups), dim3(256), 0, s, a, ct);
    return;
  }
  if (scales_aligned(a)) hipLaunchKernelGGL((k_mxfp4_tile_grouped<MODE, true>), g, dim3(256), 0, s, a, ct);
  else hipLaunchKernelGGL((k_mxfp4_tile_grouped<MODE, false>), g, dim3(256), 0, s, a, ct);
}

void launch_mxfp4_fc1(const Mxfp4GemmArgs& a, int tile_rows, hipStream_t s) { launch_grouped<kFc1>(a, tile_rows, s); }
void launch_mxfp4_fc2(const Mxfp4GemmArgs& a, int tile_rows, hipStream_t s) { launch_grouped<kFc2>(a, tile_rows, s); }

void launch_mxfp4_combine(const Mxfp4CombineArgs& a, int y_dtype, hipStream_t s) {
  const long long n = static_cast<long long>(a.tokens) * (a.H / 4);
  const dim3 g(static_cast<unsigned>((n + 255) / 256)), b(256);
  if (y_dtype == TMOE_BF16) hipLaunchKernelGGL(k_mxfp4_combine<true>, g, b, 0, s, a);
  else hipLaunchKernelGGL(k_mxfp4_combine<false>, g, b, 0, s, a);
}

}  // namespace tmoe
