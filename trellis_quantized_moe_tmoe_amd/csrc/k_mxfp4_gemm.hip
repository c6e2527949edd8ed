// k_mxfp4_gemm.hip -- products of MXFP4 rows: the dense linear, the two grouped products of the
// expert layer, and the layer's weighted sum.
//
// v_mfma_scale_f32_16x16x128_f8f6f4 with both operands E2M1 takes one whole 32-value block a lane: lane
// l holds row (or column) l % 16, block l / 16 of the 128-deep step (16 bytes, as stored) and its scale
// byte. The weights are the first operand, so a lane's four results are four neighbouring output columns
// (4 (l / 16) + i) of one token (l % 16). Products are exact; sums are fp32.
#include "tmoe.h"
#include "tmoe_mxfp4.hpp"

namespace tmoe {

namespace {

typedef int i4v __attribute__((ext_vector_type(4)));

enum { kDenseF32 = 0, kDenseBf16 = 1, kFc1 = 2, kFc2 = 3 };

__device__ __forceinline__ uint16_t bf16_rne(float f) {
  const uint32_t u = __float_as_uint(f);
  if ((u & 0x7fffffffu) > 0x7f800000u) return static_cast<uint16_t>((u >> 16) | 0x40u);
  return static_cast<uint16_t>((u + 0x7fffu + ((u >> 16) & 1u)) >> 16);
}

__device__ __forceinline__ f4 mma(i4v w, int ws, i4v x, int xs, f4 c) {
  const i8v a = __builtin_shufflevector(w, w, 0, 1, 2, 3, -1, -1, -1, -1);
  const i8v b = __builtin_shufflevector(x, x, 0, 1, 2, 3, -1, -1, -1, -1);
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 4, 4, 0, ws, 0, xs);
}

struct Frag {
  i4v q;
  int s;
};

// Block `blk` of a row; blocks past the row (the tail of a K that is no multiple of 128) are zeros.
__device__ __forceinline__ Frag load_block(const uint8_t* q, const uint8_t* s, int blk, int nblk) {
  Frag f;
  if (blk < nblk) {
    f.q = reinterpret_cast<const i4v*>(q)[blk];
    f.s = s[blk];
  } else {
    f.q = i4v{0, 0, 0, 0};
    f.s = 127;
  }
  return f;
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
      const float x = g[f][i];
      h[4 * f + i] = x / (1.0f + expf(-x)) * u[f][i];
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

// A wavefront computes 16 MT rows by 16 NT columns straight from global memory. KW = 4: the workgroup's
// wavefronts share one tile and take every fourth 128-deep step each, joined in LDS in a fixed order;
// KW = 1: they take neighbouring column groups.
template <int MODE, int MT, int NT, int KW>
__global__ __launch_bounds__(256) void k_mxfp4_direct(Mxfp4GemmArgs a) {
  static_assert(MODE != kFc1 || NT == 4, "first product: two gate and two up fragments");
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int r = lane & 15, q = lane >> 4;
  // workgroups in x only (a tile's column groups next to each other): y and z are limited to 65535
  const int ngroups = MODE == kFc1 ? a.N / 64 : (a.N + 16 * NT - 1) / (16 * NT);
  const int nwg = KW == 1 ? (ngroups + 3) / 4 : ngroups;
  const int tile = blockIdx.x / nwg, wg = blockIdx.x % nwg;
  int row0, nrows;
  long long expert = 0;
  if constexpr (MODE == kFc1 || MODE == kFc2) {
    if (tile >= *a.num_gtiles) return;
    const int4 t = a.gtiles[tile];
    expert = t.x & 0xffffff;
    row0 = t.y;
    nrows = t.z;
  } else {
    row0 = tile * 16 * MT;
    nrows = min(16 * MT, a.rows - row0);
  }
  const int group = KW == 1 ? wg * 4 + wv : wg;
  if (KW == 1 && group >= ngroups) return;
  const int nblk = a.K / 32, steps = (nblk + 3) / 4;
  const uint8_t* wq = a.wq + expert * a.N * (a.K / 2);
  const uint8_t* ws = a.ws + expert * a.N * nblk;

  const uint8_t *xq[MT], *xs[MT], *pq[NT], *ps[NT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    long long row = row0 + min(16 * m + r, nrows - 1);
    if constexpr (MODE == kFc1) row = a.sorted[row] / a.top_k;
    xq[m] = a.xq + row * (a.K / 2);
    xs[m] = a.xs + row * nblk;
  }
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    long long col;
    if constexpr (MODE == kFc1) col = (n >> 1) * (a.N / 2) + 32 * group + 16 * (n & 1) + r;
    else col = min(16 * NT * group + 16 * n + r, a.N - 1);
    pq[n] = wq + col * (a.K / 2);
    ps[n] = ws + col * nblk;
  }
  f4 acc[MT][NT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[m][n] = f4{0, 0, 0, 0};
  for (int st = KW == 1 ? 0 : wv; st < steps; st += KW) {
    const int blk = 4 * st + q;
    Frag x[MT], w[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) w[n] = load_block(pq[n], ps[n], blk, nblk);
#pragma unroll
    for (int m = 0; m < MT; ++m) x[m] = load_block(xq[m], xs[m], blk, nblk);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n) acc[m][n] = mma(w[n].q, w[n].s, x[m].q, x[m].s, acc[m][n]);
  }
  if constexpr (KW > 1) {
    __shared__ f4 part[KW - 1][MT * NT][64];
    if (wv > 0) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n) part[wv - 1][m * NT + n][lane] = acc[m][n];
    }
    __syncthreads();
    if (wv > 0) return;
#pragma unroll
    for (int p = 0; p < KW - 1; ++p)
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[m][n] += part[p][m * NT + n][lane];
  }
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const bool live = 16 * m + r < nrows;
    const long long row = row0 + 16 * m + r;
    if constexpr (MODE == kFc1) {
      const f4 g[2] = {acc[m][0], acc[m][1]}, u[2] = {acc[m][2], acc[m][3]};
      const int inter = a.N / 2;
      store_swiglu(g, u, a.bq + row * (inter / 2) + 16 * group, a.bs + row * (inter / 32) + group, lane, live);
    } else {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int col = 16 * NT * group + 16 * n + 4 * q;
        if (!live) continue;
        const long long at = row * a.N + col;
        if constexpr (MODE == kDenseBf16) {
          uint16_t* y = static_cast<uint16_t*>(a.y) + at;
          uint16_t b[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) b[i] = bf16_rne(acc[m][n][i]);
          if (a.N % 4 == 0 && col < a.N) {
            *reinterpret_cast<ushort4*>(y) = make_ushort4(b[0], b[1], b[2], b[3]);
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (col + i < a.N) y[i] = b[i];
          }
        } else {
          float* y = static_cast<float*>(a.y) + at;
          if (a.N % 4 == 0 && col < a.N) {
            *reinterpret_cast<f4*>(y) = acc[m][n];
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (col + i < a.N) y[i] = acc[m][n][i];
          }
        }
      }
    }
  }
}

// y_t = sum over j ascending of w[t][j] * v[slot of (t, j)], four columns a thread.
template <bool BF16>
__global__ __launch_bounds__(256) void k_mxfp4_combine(Mxfp4CombineArgs a) {
  const int quads = a.H / 4;
  const long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= static_cast<long long>(a.tokens) * quads) return;
  const long long t = i / quads;
  const int c = static_cast<int>(i - t * quads);
  f4 s = {0, 0, 0, 0};
  for (int j = 0; j < a.top_k; ++j) {
    const int slot = a.route_slot[t * a.top_k + j];
    if (slot < 0) continue;
    s += a.w[t * a.top_k + j] * reinterpret_cast<const f4*>(a.v + static_cast<long long>(slot) * a.H)[c];
  }
  if constexpr (BF16)
    static_cast<ushort4*>(a.y)[i] = make_ushort4(bf16_rne(s[0]), bf16_rne(s[1]), bf16_rne(s[2]), bf16_rne(s[3]));
  else
    static_cast<f4*>(a.y)[i] = s;
}

}  // namespace

int mxfp4_tile_rows(long long routes, int experts) { return routes <= 4LL * experts ? 16 : 64; }

template <int MODE>
void launch_direct(const Mxfp4GemmArgs& a, bool small, int tiles, hipStream_t s) {
  const int cols = MODE == kFc1 ? a.N / 64 : (a.N + 63) / 64;
  if (small) hipLaunchKernelGGL((k_mxfp4_direct<MODE, 1, 4, 4>), dim3(cols * tiles), dim3(256), 0, s, a);
  else hipLaunchKernelGGL((k_mxfp4_direct<MODE, 4, 4, 1>), dim3((cols + 3) / 4 * tiles), dim3(256), 0, s, a);
}

void launch_mxfp4_dense(const Mxfp4GemmArgs& a, int y_dtype, hipStream_t s) {
  const bool small = a.rows <= 16;
  const int tiles = small ? 1 : (a.rows + 63) / 64;
  if (y_dtype == TMOE_BF16) launch_direct<kDenseBf16>(a, small, tiles, s);
  else launch_direct<kDenseF32>(a, small, tiles, s);
}

void launch_mxfp4_fc1(const Mxfp4GemmArgs& a, int tile_rows, hipStream_t s) {
  launch_direct<kFc1>(a, tile_rows == 16, a.max_gtiles, s);
}

void launch_mxfp4_fc2(const Mxfp4GemmArgs& a, int tile_rows, hipStream_t s) {
  launch_direct<kFc2>(a, tile_rows == 16, a.max_gtiles, s);
}

void launch_mxfp4_combine(const Mxfp4CombineArgs& a, int y_dtype, hipStream_t s) {
  const long long n = static_cast<long long>(a.tokens) * (a.H / 4);
  const dim3 g(static_cast<unsigned>((n + 255) / 256)), b(256);
  if (y_dtype == TMOE_BF16) hipLaunchKernelGGL(k_mxfp4_combine<true>, g, b, 0, s, a);
  else hipLaunchKernelGGL(k_mxfp4_combine<false>, g, b, 0, s, a);
}

}  // namespace tmoe
