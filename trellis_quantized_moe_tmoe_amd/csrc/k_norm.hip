// k_norm.hip -- RMS norm with the residual's addition, its MXFP8 form, and the gradients.
//
//   h = x + residual (rounded to their type);  r = 1 / sqrt(mean(h^2) + eps);  y = h r g
//   dx = dh + r (g dy - h r^2 mean(g dy h));   dg = sum over rows of dy h r
// Sums are fp32 whatever the types; every output is rounded once. All of it is one pass over the data and bound by HBM
// for many rows, by one row's latency for few.
//
// A row is held in registers by 64 to 1024 threads, vectors of 16 bytes of x a lane (its last vector may be short), so
// nothing is read twice. Rows may start at any element: the vectors are loaded at the element's alignment. Passes over more
// than the caches hold read past them (16384 rows of 4096 bf16, residual, traced: forward 84 - 96 us, 5.6 - 6.4 TB/s, instead of
// 89 - 98; backward 83 - 85, 6.4 TB/s, instead of 128).
#include <algorithm>

#include "tmoe.h"
#include "tmoe_mxfp8.hpp"
#include "tmoe_norm.hpp"

namespace tmoe {

namespace {

// SMALL: the type holds values whose squares fall below fp32's smallest numbers.
struct F32 {
  typedef float T;
  static constexpr int V = 4;
  static constexpr bool SMALL = true;
  static __device__ __forceinline__ float get(float v) { return v; }
  static __device__ __forceinline__ float put(float v) { return v; }
};
struct BF16 {
  typedef uint16_t T;
  static constexpr int V = 8;
  static constexpr bool SMALL = true;
  static __device__ __forceinline__ float get(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }
  static __device__ __forceinline__ uint16_t put(float v) { return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v)); }
};
struct F16 {
  typedef uint16_t T;
  static constexpr int V = 8;
  static constexpr bool SMALL = false;
  static __device__ __forceinline__ float get(uint16_t v) { return static_cast<float>(__builtin_bit_cast(_Float16, v)); }
  static __device__ __forceinline__ uint16_t put(float v) { return __builtin_bit_cast(uint16_t, static_cast<_Float16>(v)); }
};

template <class T, int V>
struct Raw {
  T v[V];
};
template <class T, int V>
struct Vec {                                     // the same as one vector, at an element's alignment
  typedef T type __attribute__((ext_vector_type(V), aligned(sizeof(T))));
};

// V neighbouring values of a row of H from element `at`, as they are; zeros past the end. PAST: they do not stay in the caches.
template <class T, int V, bool PAST>
__device__ __forceinline__ Raw<T, V> load_raw(const T* row, int at, int H) {
  Raw<T, V> r;
  if (at + V <= H) {
    if constexpr (PAST) {
      typedef typename Vec<T, V>::type VT;
      const VT q = __builtin_nontemporal_load(reinterpret_cast<const VT*>(row + at));
      __builtin_memcpy(r.v, &q, sizeof(r.v));
    } else {
      __builtin_memcpy(r.v, row + at, sizeof(r.v));
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) r.v[i] = at + i < H ? row[at + i] : T{};
  }
  return r;
}

// The same as fp32.
template <class D, int V, bool PAST>
__device__ __forceinline__ void load_vec(const typename D::T* row, int at, int H, float (&v)[V]) {
  const Raw<typename D::T, V> r = load_raw<typename D::T, V, PAST>(row, at, H);
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = D::get(r.v[i]);
}
template <class D, int V>
__device__ __forceinline__ void store_vec(typename D::T* row, int at, int H, const float (&v)[V]) {
  typename D::T raw[V];
#pragma unroll
  for (int i = 0; i < V; ++i) raw[i] = D::put(v[i]);
  if (at + V <= H) {
    __builtin_memcpy(row + at, raw, sizeof(raw));
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (at + i < H) row[at + i] = raw[i];
  }
}

// Sum over the wavefront, in every lane, in an order that does not depend on the lane.
__device__ __forceinline__ float wave_sum(float v) {
#define TMOE_STEP(CTRL, ROWS) \
  v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, ROWS, 0xF, false));
  TMOE_STEP(0x111, 0xF)
  TMOE_STEP(0x112, 0xF)
  TMOE_STEP(0x114, 0xF)
  TMOE_STEP(0x118, 0xF)
  TMOE_STEP(0x142, 0xA)
  TMOE_STEP(0x143, 0xC)
#undef TMOE_STEP
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

// Sum over the wavefronts of a row (WIDE: a whole workgroup). sh: 16 values, free for the next sum behind its barrier.
template <bool WIDE>
__device__ __forceinline__ float row_sum(float v, float* sh) {
  v = wave_sum(v);
  if constexpr (WIDE) {
    const int waves = blockDim.x >> 6;
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
    __syncthreads();
    v = sh[0];
    for (int p = 1; p < waves; ++p) v += sh[p];
  }
  return v;
}

template <class D, class W, int NV, bool WIDE, bool MX, bool PAST>
__global__ void k_rms_norm(NormArgs a) {
  constexpr int V = D::V;
  __shared__ float sh[16], sh_small[16];
  const int H = a.hidden, tid = threadIdx.x, threads = blockDim.x;
  const int t = blockIdx.x * blockDim.y + threadIdx.y;
  if (t >= a.tokens) return;                     // whole wavefronts; WIDE: the whole workgroup
  const typename D::T* x = static_cast<const typename D::T*>(a.x) + t * a.x_stride;
  const typename D::T* res = static_cast<const typename D::T*>(a.residual) + t * a.residual_stride;
  const long long row = static_cast<long long>(t) * H;
  float h[NV][V], sum = 0.0f;
#pragma unroll
  for (int j = 0; j < NV; ++j) load_vec<D, V, PAST>(x, (j * threads + tid) * V, H, h[j]);
  if (a.residual) {
    float r[NV][V];
#pragma unroll
    for (int j = 0; j < NV; ++j) load_vec<D, V, PAST>(res, (j * threads + tid) * V, H, r[j]);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
      for (int i = 0; i < V; ++i) h[j][i] = D::get(D::put(h[j][i] + r[j][i]));   // as it is stored
      store_vec<D, V>(static_cast<typename D::T*>(a.h) + row, (j * threads + tid) * V, H, h[j]);
    }
  }
  float g[NV][V];
#pragma unroll
  for (int j = 0; j < NV; ++j) load_vec<W, V, false>(static_cast<const typename W::T*>(a.weight), (j * threads + tid) * V, H, g[j]);
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < V; ++i) sum = fmaf(h[j][i], h[j][i], sum);
  sum = row_sum<WIDE>(sum, sh);
  const float square = sum / static_cast<float>(H) + a.eps;
  float rstd = 1.0f / sqrtf(square), up = 1.0f;
  if constexpr (D::SMALL) {
    // Squares below 2^-126 lose their bits and vanish below 2^-150. Beside 2^-100 that is nothing; a row with less, its eps
    // included, is taken 2^100 times as large (exactly): its values lie below 2^-43 (H <= 2^14), so their squares sum to at most
    // 2^114, and the smallest one's square is 2^-98.
    if (square < 0x1p-100f) {                    // the same for the whole row
      sum = 0.0f;
      up = 0x1p100f;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          h[j][i] *= up;
          sum = fmaf(h[j][i], h[j][i], sum);
        }
      sum = row_sum<WIDE>(sum, sh_small);
      rstd = 1.0f / sqrtf(sum / static_cast<float>(H) + a.eps * up * up);
    }
  }
  if (a.rstd && tid == 0) a.rstd[t] = rstd * up;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int at = (j * threads + tid) * V;
    float y[V];
#pragma unroll
    for (int i = 0; i < V; ++i) y[i] = h[j][i] * rstd * g[j][i];
    if constexpr (MX) {                          // H is a multiple of 32: whole blocks, 4 lanes (16-bit x) or 8 each
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const uint32_t b = __float_as_uint(y[i]) & 0x7fffffffu;
        m = b > m ? b : m;
      }
      const uint32_t byte = mxfp8_scale_byte(V == 8 ? mxfp4_quad_max(m) : mxfp8_oct_max(m));
      const float inv = mxfp4_inverse_scale(byte);
      if (at < H) {
        uint8_t* codes = static_cast<uint8_t*>(a.y) + row + at;
#pragma unroll
        for (int i = 0; i < V; i += 4) {
          const uint32_t c = mxfp8_codes4(y[i] * inv, y[i + 1] * inv, y[i + 2] * inv, y[i + 3] * inv);
          *reinterpret_cast<uint32_t*>(codes + i) = byte == 255u ? 0u : c;
        }
        if (at % 32 == 0) a.scales[(row + at) / 32] = static_cast<uint8_t>(byte);
      }
    } else {
      store_vec<D, V>(static_cast<typename D::T*>(a.y) + row, at, H, y);
    }
  }
}

// Wavefronts a SIMD. Rows of up to 8192 16-bit or 4096 fp32 values (one vector a lane) fit the registers of five, but for seven or
// eight of fp16 rows of up to 512 values that the caches hold, which spill. Longer rows have a workgroup of up to 16 wavefronts, four
// a SIMD, with 128 registers each: fp32 rows of up to 8192 values fit; beyond 8192 values 16-bit rows spill 5 - 133 registers (4096
// x 12288 bf16, past the caches: 76 us, 5.3 TB/s) and fp32 rows 173 - 189 (247 us, 3.3 TB/s).
constexpr int grad_waves(int nv) { return nv == 1 ? 5 : 4; }

// One pass over the rows, workgroup g of a.groups every groups-th batch of rows, the next row's loads ahead of this one's sum;
// dweight's sums over its rows stay in registers, are joined over the workgroup's rows and leave as one row of partial sums.
template <class D, class W, int NV, bool WIDE, bool PAST>
__global__ __launch_bounds__(WIDE ? 1024 : 512, grad_waves(NV)) void k_rms_norm_grad(NormGradArgs a) {
  constexpr int V = D::V;
  typedef typename D::T T;
  __shared__ float sh[2][16];
  const int H = a.hidden, tid = threadIdx.x, threads = blockDim.x, rows = blockDim.y;
  float g[NV][V], dg[NV][V] = {};
#pragma unroll
  for (int j = 0; j < NV; ++j) load_vec<W, V, false>(static_cast<const typename W::T*>(a.weight), (j * threads + tid) * V, H, g[j]);
  struct Row {
    Raw<T, V> h[NV], dy[NV], dh[NV];
    float r;
  };
  auto load = [&](long long t, Row& o) {
    const T* hp = static_cast<const T*>(a.h) + t * a.h_stride;
    const long long row = t * H;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int at = (j * threads + tid) * V;
      o.h[j] = load_raw<T, V, PAST>(hp, at, H);
      o.dy[j] = load_raw<T, V, PAST>(static_cast<const T*>(a.dy) + row, at, H);
      if (a.dh) o.dh[j] = load_raw<T, V, PAST>(static_cast<const T*>(a.dh) + row, at, H);
    }
    o.r = a.rstd[t];
  };
  const long long step = static_cast<long long>(a.groups) * rows;
  int turn = 0;
  Row now, next;
  long long t = static_cast<long long>(blockIdx.x) * rows + threadIdx.y;
  if (t < a.tokens) load(t, now);
  for (; t < a.tokens; t += step) {              // WIDE: the same rows for the whole workgroup
    if (t + step < a.tokens) load(t + step, next);
    float u[NV][V], d[NV][V], c = 0.0f;
    const float r = now.r;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        u[j][i] = D::get(now.h[j].v[i]) * r;     // the row's unit values
        const float dy = D::get(now.dy[j].v[i]);
        dg[j][i] = fmaf(dy, u[j][i], dg[j][i]);
        d[j][i] = dy * g[j][i];
        c = fmaf(d[j][i], u[j][i], c);
      }
    c = row_sum<WIDE>(c, sh[turn]) / static_cast<float>(H);
    turn ^= 1;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float o[V];
#pragma unroll
      for (int i = 0; i < V; ++i) o[i] = fmaf(r, fmaf(-u[j][i], c, d[j][i]), a.dh ? D::get(now.dh[j].v[i]) : 0.0f);
      store_vec<D, V>(static_cast<T*>(a.dx) + t * H, (j * threads + tid) * V, H, o);
    }
    now = next;
  }
  float* part = a.part + static_cast<long long>(blockIdx.x) * H;
  if constexpr (!WIDE) {                         // the rows' wavefronts add up in order
    __shared__ float sum[NV * V][64];
    for (int p = 0; p < rows; ++p) {
      if (threadIdx.y == p) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int i = 0; i < V; ++i) {
            if (p > 0) dg[j][i] += sum[j * V + i][tid];
            sum[j * V + i][tid] = dg[j][i];
          }
      }
      __syncthreads();
    }
    if (threadIdx.y != rows - 1) return;
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) store_vec<F32, V>(part, (j * threads + tid) * V, H, dg[j]);
}

// dweight: 16 columns a workgroup, 64 threads a column with every 64th partial row, joined in a fixed order.
template <class W>
__global__ __launch_bounds__(1024) void k_rms_norm_dweight(const float* part, int n, int H, void* dweight) {
  __shared__ float sh[64][17];
  const int c = blockIdx.x * 16 + threadIdx.x, at = min(c, H - 1);
  float s = 0.0f;
#pragma unroll 8
  for (int p = threadIdx.y; p < n; p += 64) s += part[static_cast<long long>(p) * H + at];
  sh[threadIdx.y][threadIdx.x] = s;
#pragma unroll
  for (int d = 32; d; d >>= 1) {
    __syncthreads();
    if (static_cast<int>(threadIdx.y) < d) sh[threadIdx.y][threadIdx.x] += sh[threadIdx.y + d][threadIdx.x];
  }
  if (threadIdx.y == 0 && c < H) static_cast<typename W::T*>(dweight)[c] = W::put(sh[0][threadIdx.x]);
}

// The gradient's: one vector a lane as far as a workgroup goes (it holds five of them at a time), eight rows of up to 64
// vectors a workgroup.
NormShape grad_shape(int hidden, int dtype) {
  const int v = dtype == TMOE_F32 ? 4 : 8, vecs = (hidden + v - 1) / v;
  NormShape n;
  n.nv = vecs <= 1024 ? 1 : vecs <= 2048 ? 2 : 4;
  n.threads = ((vecs + n.nv - 1) / n.nv + 63) / 64 * 64;
  n.rows = n.threads == 64 ? 8 : 1;
  return n;
}

template <class D, class W, bool MX, bool PAST>
void launch_norm(const NormArgs& a, int dtype, hipStream_t s) {
  const NormShape n = norm_shape(a.hidden, dtype);
  const dim3 g((a.tokens + n.rows - 1) / n.rows), b(n.threads, n.rows);
  if (n.threads == 64) {
    if (n.nv == 1) hipLaunchKernelGGL((k_rms_norm<D, W, 1, false, MX, PAST>), g, b, 0, s, a);
    else if (n.nv == 2) hipLaunchKernelGGL((k_rms_norm<D, W, 2, false, MX, PAST>), g, b, 0, s, a);
    else hipLaunchKernelGGL((k_rms_norm<D, W, 4, false, MX, PAST>), g, b, 0, s, a);
  } else {
    if (n.nv == 2) hipLaunchKernelGGL((k_rms_norm<D, W, 2, true, MX, PAST>), g, b, 0, s, a);
    else if constexpr (D::V == 4) hipLaunchKernelGGL((k_rms_norm<D, W, 4, true, MX, PAST>), g, b, 0, s, a);   // fp32 rows beyond 8192
  }
}

template <class D, class W, bool PAST>
void launch_grad(const NormGradArgs& a, int dtype, hipStream_t s) {
  const NormShape n = grad_shape(a.hidden, dtype);
  const dim3 g(a.groups), b(n.threads, n.rows);
  if (a.groups == 0) {
  } else if (n.threads == 64) {
    hipLaunchKernelGGL((k_rms_norm_grad<D, W, 1, false, PAST>), g, b, 0, s, a);
  } else if (n.nv == 1) {
    hipLaunchKernelGGL((k_rms_norm_grad<D, W, 1, true, PAST>), g, b, 0, s, a);
  } else if (n.nv == 2) {
    hipLaunchKernelGGL((k_rms_norm_grad<D, W, 2, true, PAST>), g, b, 0, s, a);
  } else {
    if constexpr (D::V == 4) hipLaunchKernelGGL((k_rms_norm_grad<D, W, 4, true, PAST>), g, b, 0, s, a);   // fp32 rows beyond 8192
  }
  hipLaunchKernelGGL((k_rms_norm_dweight<W>), dim3((a.hidden + 15) / 16), dim3(16, 64), 0, s, a.part, a.groups, a.hidden,
                     a.dweight);
}

}  // namespace

NormShape norm_shape(int hidden, int dtype) {
  const int v = dtype == TMOE_F32 ? 4 : 8, vecs = (hidden + v - 1) / v;
  NormShape n;
  if (vecs <= 256) {
    n.threads = 64;
    n.rows = 4;
    n.nv = vecs <= 64 ? 1 : vecs <= 128 ? 2 : 4;
  } else {
    n.rows = 1;
    n.nv = vecs <= 2048 ? 2 : 4;
    n.threads = ((vecs + n.nv - 1) / n.nv + 63) / 64 * 64;
  }
  return n;
}

// As many workgroups as the chip holds at once (more would come in a second round), but not so many that their partial sums
// count beside the rows (2047 rows of 2560 fp16: 1024 groups 27 us, 511 19).
int norm_grad_groups(int tokens, int hidden, int dtype) {
  const NormShape n = grad_shape(hidden, dtype);
  const int waves = n.threads * n.rows / 64, batches = (tokens + n.rows - 1) / n.rows;
  const int resident = 256 * std::clamp(4 * grad_waves(n.nv) / waves, 1, 8);
  return std::max(1, std::min({batches, resident, std::max(256, batches / 4)}));
}

void launch_rms_norm(const NormArgs& a, int dtype, bool weight_f32, bool mxfp8, hipStream_t s) {
  const int es = dtype == TMOE_F32 ? 4 : 2;
  const bool past = passes_caches(static_cast<long long>(a.tokens) * a.hidden * (es * (a.residual ? 3 : 1) + (mxfp8 ? 1 : es)));
  auto go = [&](auto d, auto w) {
    using D = decltype(d);
    using W = decltype(w);
    if (mxfp8) past ? launch_norm<D, W, true, true>(a, dtype, s) : launch_norm<D, W, true, false>(a, dtype, s);
    else past ? launch_norm<D, W, false, true>(a, dtype, s) : launch_norm<D, W, false, false>(a, dtype, s);
  };
  if (dtype == TMOE_F32) go(F32{}, F32{});
  else if (dtype == TMOE_BF16) weight_f32 ? go(BF16{}, F32{}) : go(BF16{}, BF16{});
  else weight_f32 ? go(F16{}, F32{}) : go(F16{}, F16{});
}

void launch_rms_norm_grad(const NormGradArgs& a, int dtype, bool weight_f32, hipStream_t s) {
  const bool past = passes_caches(static_cast<long long>(a.tokens) * a.hidden * (dtype == TMOE_F32 ? 4 : 2) * (a.dh ? 4 : 3));
  auto go = [&](auto d, auto w) {
    using D = decltype(d);
    using W = decltype(w);
    past ? launch_grad<D, W, true>(a, dtype, s) : launch_grad<D, W, false>(a, dtype, s);
  };
  if (dtype == TMOE_F32) go(F32{}, F32{});
  else if (dtype == TMOE_BF16) weight_f32 ? go(BF16{}, F32{}) : go(BF16{}, BF16{});
  else weight_f32 ? go(F16{}, F32{}) : go(F16{}, F16{});
}

}  // namespace tmoe
