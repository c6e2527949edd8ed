// k_router.hip -- the router: softmax top-k over expert logits, the balance loss with per-expert
// counts, and the gradient of the logits from both.
//
// One wavefront per token row of E <= 512 logits, expert e = 64 j + lane in register j. The row's
// maximum m and sum s = sum exp(l - m) are taken in fp32 whatever the logits' type; weights are
// exp(l - m) / s, never exp(l - lse), which would lose the digits that lse rounds away at large |l|.
#include "tmoe.h"
#include "tmoe_device.hpp"
#include "tmoe_router.hpp"

namespace tmoe {

namespace {

constexpr int kWavesPerGroup = 4;
constexpr float kNegInf = -__builtin_inff();

struct F32 {
  typedef float T;
  static __device__ __forceinline__ float get(float v) { return v; }
  static __device__ __forceinline__ float put(float v) { return v; }
};
struct BF16 {
  typedef uint16_t T;
  static __device__ __forceinline__ float get(uint16_t v) { return bf16_to_f32(v); }
  static __device__ __forceinline__ uint16_t put(float v) {   // round to nearest even, NaN kept
    const uint32_t u = __float_as_uint(v);
    if ((u & 0x7fffffffu) > 0x7f800000u) return static_cast<uint16_t>((u >> 16) | 0x40u);
    return static_cast<uint16_t>((u + 0x7fffu + ((u >> 16) & 1u)) >> 16);
  }
};
struct F16 {
  typedef uint16_t T;
  static __device__ __forceinline__ float get(uint16_t v) { return h2f(v); }
  static __device__ __forceinline__ uint16_t put(float v) {
    return __builtin_bit_cast(uint16_t, static_cast<_Float16>(v));
  }
};

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v = fmaxf(v, __shfl_xor(v, d, 64));
  return v;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d, 64);
  return v;
}

__device__ __forceinline__ long long read_id(const void* ids, int ids64, long long i) {
  return ids64 ? static_cast<const long long*>(ids)[i] : static_cast<long long>(static_cast<const int*>(ids)[i]);
}

// Order-preserving key of a float: larger floats, larger keys; the two zeros share one key.
__device__ __forceinline__ uint32_t order_key(float f) {
  const uint32_t u = __float_as_uint(f + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

template <class D, int V>
__device__ __forceinline__ void load_row(const void* logits, long long stride, int row, int E, int lane,
                                         float (&v)[V]) {
  const typename D::T* p = static_cast<const typename D::T*>(logits) + row * stride;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int e = 64 * j + lane;
    v[j] = e < E ? D::get(p[e]) : kNegInf;
  }
}

// exp(l - m) of the row in v (m: the row's largest value, 0 where that is -inf, so a row of -inf gives
// zeros and a NaN or +inf anywhere gives a NaN sum); returns the sum.
template <int V>
__device__ __forceinline__ float row_exp(float (&v)[V], float* m_out) {
  float m = kNegInf;
#pragma unroll
  for (int j = 0; j < V; ++j) m = fmaxf(m, v[j]);
  m = wave_max(m);
  if (m == kNegInf) m = 0.0f;
  float s = 0.0f;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    v[j] = expf(v[j] - m);
    s += v[j];
  }
  *m_out = m;
  return wave_sum(s);
}

// The k largest logits of a row, one round each: the largest (key, lowest expert) pair of the
// wavefront, then that entry's key is cleared. Key 0 marks an expert that is not available (-inf,
// NaN or past E).
template <class D, int V>
__global__ __launch_bounds__(64 * kWavesPerGroup) void k_router_topk(RouterTopkArgs a) {
  const int lane = threadIdx.x & 63;
  const int t = blockIdx.x * kWavesPerGroup + (threadIdx.x >> 6);
  if (t >= a.tokens) return;
  const int k = a.top_k;
  float v[V];
  uint32_t key[V];
  const bool in = a.mask == nullptr || a.mask[t] != 0;
  if (in) {
    load_row<D, V>(a.logits, a.stride, t, a.experts, lane, v);
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] = kNegInf;
  }
#pragma unroll
  for (int j = 0; j < V; ++j) key[j] = v[j] > kNegInf ? order_key(v[j]) : 0u;
  float m;
  const float s = row_exp<V>(v, &m);
  int my_id = -1;
  float my_e = 0.0f;                             // exp(l - m) of the lane's own choice (lane = rank)
  for (int r = 0; r < k; ++r) {
    uint32_t bk = 0;
    int bj = 0;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (key[j] > bk) {
        bk = key[j];
        bj = j;
      }
    unsigned long long best =
        (static_cast<unsigned long long>(bk) << 32) | (0xffffffffu - static_cast<uint32_t>(64 * bj + lane));
#pragma unroll
    for (int d = 32; d; d >>= 1) {
      const unsigned long long o = __shfl_xor(best, d, 64);
      best = o > best ? o : best;
    }
    if ((best >> 32) == 0) break;                // fewer than k experts available
    const int e = static_cast<int>(0xffffffffu - static_cast<uint32_t>(best));
    float x = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (j == (e >> 6)) {
        x = v[j];
        if (lane == (e & 63)) key[j] = 0;
      }
    x = __shfl(x, e & 63, 64);
    if (lane == r) {
      my_id = e;
      my_e = x;
    }
  }
  float total = a.renormalize ? wave_sum(my_e) : s;
  if (s != s) total = s;                         // a NaN or +inf in the row: every weight is NaN
  if (lane < k) {
    const long long at = static_cast<long long>(t) * k + lane;
    if (a.ids64) static_cast<long long*>(a.ids)[at] = my_id;
    else static_cast<int*>(a.ids)[at] = my_id;
    a.w[at] = s != s ? s : my_id >= 0 ? my_e / total : 0.0f;
  }
  if (lane == 0) a.lse[t] = m + logf(s);
}

// Balance loss, launch 1: a workgroup sums the probabilities and counts the routes of its rows.
template <class D, int V>
__global__ __launch_bounds__(64 * kWavesPerGroup) void k_balance_rows(BalanceArgs a) {
  __shared__ float ps[kWavesPerGroup][64 * V];
  __shared__ int cs[512];
  __shared__ int ns[kWavesPerGroup];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, E = a.experts;
  const int beg = blockIdx.x * a.rows_per_group, end = min(a.tokens, beg + a.rows_per_group);
  for (int e = threadIdx.x; e < E; e += blockDim.x) cs[e] = 0;
  __syncthreads();
  float acc[V];
#pragma unroll
  for (int j = 0; j < V; ++j) acc[j] = 0.0f;
  int n = 0;
  for (int t = beg + wv; t < end; t += kWavesPerGroup) {
    if (lane < a.top_k) {
      const long long e = read_id(a.ids, a.ids64, static_cast<long long>(t) * a.top_k + lane);
      if (e >= 0 && e < E) atomicAdd(&cs[e], 1);
    }
    if (a.lse[t] == kNegInf) continue;
    float v[V], m;
    load_row<D, V>(a.logits, a.stride, t, E, lane, v);
    const float s = row_exp<V>(v, &m);
#pragma unroll
    for (int j = 0; j < V; ++j) acc[j] += v[j] / s;
    ++n;
  }
#pragma unroll
  for (int j = 0; j < V; ++j) ps[wv][64 * j + lane] = acc[j];
  if (lane == 0) ns[wv] = n;
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    float p = 0.0f;
    for (int q = 0; q < kWavesPerGroup; ++q) p += ps[q][e];
    a.psum[static_cast<long long>(blockIdx.x) * E + e] = p;
    a.csum[static_cast<long long>(blockIdx.x) * E + e] = cs[e];
  }
  if (threadIdx.x == 0) {
    int c = 0;
    for (int q = 0; q < kWavesPerGroup; ++q) c += ns[q];
    a.nsum[blockIdx.x] = c;
  }
}

// Balance loss, launch 2 (one workgroup, an expert a thread): totals over the groups in a fixed
// order, then the loss and its slope for each expert. The sums of sums are held in 64 bits.
__global__ __launch_bounds__(512) void k_balance_finish(BalanceArgs a) {
  __shared__ double red[512];
  __shared__ int nred[512], cred[512];
  const int e = threadIdx.x, E = a.experts;
  double p = 0.0;
  int c = 0, n = 0;
  if (e < E)
    for (int g = 0; g < a.groups; ++g) {
      p += a.psum[static_cast<long long>(g) * E + e];
      c += a.csum[static_cast<long long>(g) * E + e];
    }
  for (int g = e; g < a.groups; g += 512) n += a.nsum[g];
  nred[e] = n;
  cred[e] = c;
  __syncthreads();
  for (int d = 256; d; d >>= 1) {
    if (e < d) {
      nred[e] += nred[e + d];
      cred[e] += cred[e + d];
    }
    __syncthreads();
  }
  const int nt = nred[0], ct = cred[0];
  const double f = ct > 0 ? static_cast<double>(c) / ct : 0.0;
  const double slope = nt > 0 ? static_cast<double>(a.coefficient) * E * f / nt : 0.0;
  red[e] = slope * p;
  __syncthreads();
  for (int d = 256; d; d >>= 1) {
    if (e < d) red[e] += red[e + d];
    __syncthreads();
  }
  if (e < E) {
    a.counts[e] = c;
    a.slope[e] = static_cast<float>(slope);
  }
  if (e == 0) *a.loss = static_cast<float>(red[0]);
}

// Gradient of one row. Top-k part: renormalised weights w_j over the selected logits give
// w_j (dw_j - sum_i w_i dw_i) at the selected ones; softmax weights give that sum's share of every
// expert. Balance part: dloss * p_e (slope_e - sum p slope).
template <class D, int V>
__global__ __launch_bounds__(64 * kWavesPerGroup) void k_router_grad(RouterGradArgs a) {
  __shared__ float at_expert[kWavesPerGroup][64 * V];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int t = blockIdx.x * kWavesPerGroup + wv;
  if (t >= a.tokens) return;                     // no workgroup barrier below: a wave keeps to its own LDS row
  const int E = a.experts, k = a.top_k;
  float* mine = at_expert[wv];
#pragma unroll
  for (int j = 0; j < V; ++j) mine[64 * j + lane] = 0.0f;
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  const bool in = a.lse[t] != kNegInf;
  float dot = 0.0f;
  if (a.dw) {
    long long e = -1;
    float w = 0.0f, g = 0.0f;
    if (in && lane < k) {
      const long long at = static_cast<long long>(t) * k + lane;
      e = read_id(a.ids, a.ids64, at);
      if (e >= 0 && e < E) {
        w = a.w[at];
        g = w * a.dw[at];
      } else {
        e = -1;
      }
    }
    dot = wave_sum(g);
    if (e >= 0) atomicAdd(&mine[e], a.renormalize ? g - w * dot : g);
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");   // the row's LDS entries are read across lanes below
  const bool soft = in && (a.slope != nullptr || (a.dw != nullptr && !a.renormalize));
  float v[V];
  float inv = 0.0f, mean = 0.0f, dl = 0.0f;
  float slope[V];
#pragma unroll
  for (int j = 0; j < V; ++j) v[j] = slope[j] = 0.0f;
  if (soft) {
    float m;
    load_row<D, V>(a.logits, a.stride, t, E, lane, v);
    inv = 1.0f / row_exp<V>(v, &m);
    if (a.slope) {
      dl = *a.dloss;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int e = 64 * j + lane;
        slope[j] = e < E ? a.slope[e] : 0.0f;
        mean += v[j] * inv * slope[j];
      }
      mean = wave_sum(mean);
    }
  }
  const float all = a.dw != nullptr && !a.renormalize ? dot : 0.0f;
  typename D::T* out = static_cast<typename D::T*>(a.dlogits) + static_cast<long long>(t) * E;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int e = 64 * j + lane;
    float d = mine[e];
    if (soft) {
      const float p = v[j] * inv;
      d += p * (dl * (slope[j] - mean) - all);
    }
    if (e < E) out[e] = D::put(d);
  }
}

// Calls f with the row registers (1, 2, 4 or 8 logits a lane) of E experts.
template <class F>
void with_width(int E, F&& f) {
  if (E <= 64) f(std::integral_constant<int, 1>{});
  else if (E <= 128) f(std::integral_constant<int, 2>{});
  else if (E <= 256) f(std::integral_constant<int, 4>{});
  else f(std::integral_constant<int, 8>{});
}

template <class F>
void with_dtype(int dtype, F&& f) {
  if (dtype == TMOE_F32) f(F32{});
  else if (dtype == TMOE_BF16) f(BF16{});
  else f(F16{});
}

unsigned row_groups(int tokens) { return static_cast<unsigned>((tokens + kWavesPerGroup - 1) / kWavesPerGroup); }

}  // namespace

void launch_router_topk(const RouterTopkArgs& a, int dtype, hipStream_t s) {
  with_dtype(dtype, [&](auto d) {
    with_width(a.experts, [&](auto v) {
      hipLaunchKernelGGL((k_router_topk<decltype(d), decltype(v)::value>), dim3(row_groups(a.tokens)),
                         dim3(64 * kWavesPerGroup), 0, s, a);
    });
  });
}

void launch_balance(const BalanceArgs& a, int dtype, hipStream_t s) {
  if (a.groups > 0)
    with_dtype(dtype, [&](auto d) {
      with_width(a.experts, [&](auto v) {
        hipLaunchKernelGGL((k_balance_rows<decltype(d), decltype(v)::value>), dim3(a.groups),
                           dim3(64 * kWavesPerGroup), 0, s, a);
      });
    });
  hipLaunchKernelGGL(k_balance_finish, dim3(1), dim3(512), 0, s, a);
}

void launch_router_grad(const RouterGradArgs& a, int dtype, hipStream_t s) {
  with_dtype(dtype, [&](auto d) {
    with_width(a.experts, [&](auto v) {
      hipLaunchKernelGGL((k_router_grad<decltype(d), decltype(v)::value>), dim3(row_groups(a.tokens)),
                         dim3(64 * kWavesPerGroup), 0, s, a);
    });
  });
}

}  // namespace tmoe
