// k_router.hip -- the router: softmax top-k over expert logits, the balance loss with per-expert
// counts, and the gradient of the logits from both.
//
// One wavefront per token row of E <= 512 logits, expert e = 64 j + lane in register j. Sums are fp32
// whatever the logits' type; weights and probabilities are divided by a sum of the same exponentials,
// never exp(l - lse) alone, which would lose the digits that lse rounds away at large |l|.
#include "tmoe.h"
#include "tmoe_device.hpp"
#include "tmoe_router.hpp"

namespace tmoe {

namespace {

constexpr int kWavesPerGroup = 4;
constexpr int kBalanceWaves = 16;
constexpr int kBatch = 4;
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
    return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
  }
};
struct F16 {
  typedef uint16_t T;
  static __device__ __forceinline__ float get(uint16_t v) { return h2f(v); }
  static __device__ __forceinline__ uint16_t put(float v) {
    return __builtin_bit_cast(uint16_t, static_cast<_Float16>(v));
  }
};

// Wavefront reductions by DPP: row_shr 1, 2, 4, 8 leave a 16-lane row's total in its last lane, the two
// row broadcasts carry it on to lane 63, and one readlane makes it uniform. Lanes without a source
// keep the identity (0 for the sum and for the unsigned maximum).
#define TMOE_WAVE_STEPS(OP)                                                         \
  OP(0x111, 0xF)                                                                    \
  OP(0x112, 0xF)                                                                    \
  OP(0x114, 0xF)                                                                    \
  OP(0x118, 0xF)                                                                    \
  OP(0x142, 0xA)                                                                    \
  OP(0x143, 0xC)
__device__ __forceinline__ float wave_sum(float v) {
#define TMOE_STEP(CTRL, ROWS) \
  v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, ROWS, 0xF, false));
  TMOE_WAVE_STEPS(TMOE_STEP)
#undef TMOE_STEP
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#define TMOE_STEP(CTRL, ROWS)                                                                       \
  {                                                                                                 \
    const uint32_t o = __builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, ROWS, 0xF, false); \
    v = o > v ? o : v;                                                                              \
  }
  TMOE_WAVE_STEPS(TMOE_STEP)
#undef TMOE_STEP
  return __builtin_amdgcn_readlane(v, 63);
}
#undef TMOE_WAVE_STEPS

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
  // lanes past E read the last value and drop it: loads without a branch stay in flight together
#pragma unroll
  for (int j = 0; j < V; ++j) v[j] = D::get(p[min(64 * j + lane, E - 1)]);
#pragma unroll
  for (int j = 0; j < V; ++j) v[j] = 64 * j + lane < E ? v[j] : kNegInf;
}

// exp(x) for x <= about 1, half the instructions of expf: 2^y with y = x log2(e) rounded, times 1 + r ln 2
// for the rest r of that product (from a two-word log2(e)); 2 units in the last place at most. 0 below
// -200 (and, with the hardware's 2^y, below 2^-126); NaN stays.
__device__ __forceinline__ float exp_neg(float x) {
  x = x < -200.0f ? -200.0f : x;
  constexpr float kHi = 0x1.715476p+0f, kLo = 0x1.4ae0cp-26f;    // log2(e) = kHi + kLo
  const float y = x * kHi;
  const float r = fmaf(x, kLo, fmaf(x, kHi, -y));
  const float p = __builtin_amdgcn_exp2f(y);
  return fmaf(p, r * 0.693147182f, p);
}

__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

// The k largest logits of a row, one round each: the largest key of the wavefront (uniform), the lowest
// expert that has it (one ballot per register; registers hold ascending experts), then that entry's key
// is cleared. Key 0 marks an expert that is not available (-inf, NaN or past E). A selected logit is its
// key read back, so the weights need no gather. The vector unit bounds it. Two rows a wavefront, side by
// side, measured the same (14 us at T = 16384, E = 256, k = 8).
template <class D, int V>
__global__ __launch_bounds__(64 * kWavesPerGroup) void k_router_topk(RouterTopkArgs a) {
  const int lane = threadIdx.x & 63;
  const int t = blockIdx.x * kWavesPerGroup + (threadIdx.x >> 6);
  if (t >= a.tokens) return;
  const int k = a.top_k;
  float v[V];
  uint32_t key[V];
  const uint32_t in = a.mask == nullptr ? 1u : a.mask[t];
  load_row<D, V>(a.logits, a.stride, t, a.experts, lane, v);
#pragma unroll
  for (int j = 0; j < V; ++j) {
    v[j] = in ? v[j] : kNegInf;
    key[j] = v[j] > kNegInf ? order_key(v[j]) : 0u;
  }
  int my_id = -1;                                // lane r holds the choice of rank r
  uint32_t my_key = 0, top = 0;
  for (int r = 0; r < k; ++r) {
    uint32_t lm = key[0];
#pragma unroll
    for (int j = 1; j < V; ++j) lm = key[j] > lm ? key[j] : lm;
    const uint32_t best = wave_max(lm);
    if (r == 0) top = best;
    if (best == 0) break;                        // fewer than k experts available
    unsigned long long has[V];
    int e = -1, n = 0;
#pragma unroll
    for (int j = V - 1; j >= 0; --j) {
      has[j] = __ballot(key[j] == best);
      n += __popcll(has[j]);
      if (has[j]) e = 64 * j + __ffsll(has[j]) - 1;
    }
    if (n == 1) {
#pragma unroll
      for (int j = 0; j < V; ++j) key[j] = key[j] == best ? 0u : key[j];
    } else {                                     // equal logits: only the lowest expert leaves
#pragma unroll
      for (int j = 0; j < V; ++j) key[j] = 64 * j + lane == e ? 0u : key[j];
    }
    if (lane == r) {
      my_id = e;
      my_key = best;
    }
  }
  // m: the row's largest logit, 0 where no expert is available: a row of -inf sums to 0, and a NaN or
  // +inf anywhere makes the sum NaN
  const float m = top ? key_value(top) : 0.0f;
  float s = 0.0f;
#pragma unroll
  for (int j = 0; j < V; ++j) s += exp_neg(v[j] - m);
  s = wave_sum(s);
  const float x = my_id >= 0 ? exp_neg(key_value(my_key) - m) : 0.0f;
  const float total = a.renormalize ? wave_sum(x) : s;
  if (lane < k) {
    const long long at = static_cast<long long>(t) * k + lane;
    if (a.ids64) static_cast<long long*>(a.ids)[at] = my_id;
    else static_cast<int*>(a.ids)[at] = my_id;
    a.w[at] = s != s ? s : my_id >= 0 ? x / total : 0.0f;   // a NaN or +inf in the row: every weight is NaN
  }
  if (lane == 0) a.lse[t] = m + logf(s);
}

// exp(l - lse) of the row in v and the reciprocal of its sum. lse only shifts the exponents near 0: its
// rounding (large at large |l|) cancels in the division by the sum.
template <int V>
__device__ __forceinline__ float row_softmax(float (&v)[V], float lse) {
  float s = 0.0f;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    v[j] = exp_neg(v[j] - lse);
    s += v[j];
  }
  return 1.0f / wave_sum(s);
}

// Balance loss, launch 1: a workgroup sums the probabilities and counts the routes of its rows.
template <class D, int V>
__global__ __launch_bounds__(64 * kBalanceWaves) void k_balance_rows(BalanceArgs a) {
  __shared__ float ps[kBalanceWaves][64 * V];
  __shared__ int cs[64 * V];
  __shared__ int ns[kBalanceWaves];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, E = a.experts;
  const int beg = blockIdx.x * a.rows_per_group, end = min(a.tokens, beg + a.rows_per_group);
  for (int e = threadIdx.x; e < 64 * V; e += blockDim.x) cs[e] = 0;
  __syncthreads();
  // the counts: the workgroup's ids are one run of memory
  const long long ids_end = static_cast<long long>(end) * a.top_k;
  for (long long i = static_cast<long long>(beg) * a.top_k + threadIdx.x; i < ids_end; i += blockDim.x) {
    const long long e = read_id(a.ids, a.ids64, i);
    if (e >= 0 && e < E) atomicAdd(&cs[e], 1);
  }
  float acc[V];
#pragma unroll
  for (int j = 0; j < V; ++j) acc[j] = 0.0f;
  int n = 0;
  // kBatch rows at a time, so that their loads are in flight together (one row at a time: 27.8 us at
  // T = 32768, E = 256 in bf16); a row that does not count adds zeros whatever it holds. Up to T = 4096 a wavefront has
  // one row, and the other three places repeat a row for nothing.
  for (int t0 = beg + wv; t0 < end; t0 += kBalanceWaves * kBatch) {
    float v[kBatch][V], lse[kBatch];
#pragma unroll
    for (int q = 0; q < kBatch; ++q) {
      const int t = t0 + q * kBalanceWaves, tc = min(t, end - 1);
      lse[q] = t < end ? a.lse[tc] : kNegInf;
      load_row<D, V>(a.logits, a.stride, tc, E, lane, v[q]);
    }
#pragma unroll
    for (int q = 0; q < kBatch; ++q) {
      const bool in = lse[q] > kNegInf;          // not so for a NaN: one bad row leaves the others' loss as it is
#pragma unroll
      for (int j = 0; j < V; ++j) v[q][j] = in ? v[q][j] : kNegInf;
      float inv = row_softmax<V>(v[q], in ? lse[q] : 0.0f);
      inv = in ? inv : 0.0f;
#pragma unroll
      for (int j = 0; j < V; ++j) acc[j] += v[q][j] * inv;
      n += in ? 1 : 0;
    }
  }
#pragma unroll
  for (int j = 0; j < V; ++j) ps[wv][64 * j + lane] = acc[j];
  if (lane == 0) ns[wv] = n;
  __syncthreads();
  for (int e = threadIdx.x; e < a.pitch; e += blockDim.x) {      // entries past E are zeros
    float p = 0.0f;
    for (int q = 0; q < kBalanceWaves; ++q) p += ps[q][e];
    a.psum[static_cast<long long>(blockIdx.x) * a.pitch + e] = p;
    a.csum[static_cast<long long>(blockIdx.x) * a.pitch + e] = cs[e];
  }
  if (threadIdx.x < 64) {                        // rows that count, and routes
    int c = 0;
    for (int e = lane; e < E; e += 64) c += cs[e];
#pragma unroll
    for (int d = 32; d; d >>= 1) c += __shfl_xor(c, d, 64);
    if (lane == 0) {
      int rows = 0;
      for (int q = 0; q < kBalanceWaves; ++q) rows += ns[q];
      a.nsum[2 * blockIdx.x] = rows;
      a.nsum[2 * blockIdx.x + 1] = c;
      if (blockIdx.x == 0) *a.done = 0;          // the second launch's counter
    }
  }
}

// Balance loss, launch 2: a workgroup adds up 32 experts over the groups, each thread four experts of every 32nd
// group, so that all its loads are in flight at once (one thread an expert walking 512 groups took 128 us,
// one workgroup for all experts 8.6 us at 256 groups, E = 256; 5.4 us here). The order of the sums is fixed and they are
// held in 64 bits; the workgroup that ends last adds the others' parts of the loss, in order.
__global__ __launch_bounds__(256) void k_balance_finish(BalanceArgs a) {
  __shared__ double pt[32][33];
  __shared__ int ct[32][33];
  __shared__ int nred[4], cred[4];
  const int tid = threadIdx.x, E = a.experts, quads = a.pitch / 4;
  const int row = tid / 8, col = blockIdx.x * 8 + tid % 8;
  double p[4] = {0, 0, 0, 0};
  int c[4] = {0, 0, 0, 0}, n = 0, all = 0;
  if (col < quads) {
#pragma unroll 8
    for (int g = row; g < a.groups; g += 32) {
      const float4 x = reinterpret_cast<const float4*>(a.psum)[static_cast<long long>(g) * quads + col];
      const int4 y = reinterpret_cast<const int4*>(a.csum)[static_cast<long long>(g) * quads + col];
      p[0] += x.x; p[1] += x.y; p[2] += x.z; p[3] += x.w;
      c[0] += y.x; c[1] += y.y; c[2] += y.z; c[3] += y.w;
    }
  }
  for (int g = tid; g < a.groups; g += 256) {
    n += a.nsum[2 * g];
    all += a.nsum[2 * g + 1];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    pt[row][4 * (tid % 8) + i] = p[i];
    ct[row][4 * (tid % 8) + i] = c[i];
  }
#pragma unroll
  for (int d = 32; d; d >>= 1) {
    n += __shfl_xor(n, d, 64);
    all += __shfl_xor(all, d, 64);
  }
  if ((tid & 63) == 0) {
    nred[tid >> 6] = n;
    cred[tid >> 6] = all;
  }
  __syncthreads();
  const int nt = nred[0] + nred[1] + nred[2] + nred[3], total = cred[0] + cred[1] + cred[2] + cred[3];
  if (tid < 64) {
    const int e = blockIdx.x * 32 + tid;
    double l = 0.0;
    if (tid < 32 && e < E) {
      double pe = 0.0;
      int ce = 0;
      for (int r = 0; r < 32; ++r) {
        pe += pt[r][tid];
        ce += ct[r][tid];
      }
      const double f = total > 0 ? static_cast<double>(ce) / total : 0.0;
      const double slope = nt > 0 ? static_cast<double>(a.coefficient) * E * f / nt : 0.0;
      a.counts[e] = ce;
      a.slope[e] = static_cast<float>(slope);
      l = slope * pe;
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) l += __shfl_xor(l, d, 64);
    if (tid == 0) {
      const int parts = gridDim.x;
      if (parts == 1 || a.groups == 0) {         // no groups: nothing cleared the counter, every part is 0
        *a.loss = static_cast<float>(l);
      } else {
        __hip_atomic_store(a.part + blockIdx.x, l, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        const bool last = __hip_atomic_fetch_add(a.done, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == parts - 1;
        if (last) {
          double s = 0.0;
          for (int i = 0; i < parts; ++i) s += __hip_atomic_load(a.part + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
          *a.loss = static_cast<float>(s);
        }
      }
    }
  }
}

// Gradient of one row. Top-k part: renormalised weights w_j over the selected logits give
// w_j (dw_j - sum_i w_i dw_i) at the selected ones (the logits are not read); softmax weights give that
// sum's share of every expert. Balance part: dloss * p_e (slope_e - sum p slope), for rows with lse > -inf. A row whose
// lse is NaN (a NaN or +inf logit) has no balance part; its weights are NaN, and the top-k part carries that on.
// Every load of the row is issued before the first wait; a row with lse = -inf is read and not used.
template <class D, int V>
__global__ __launch_bounds__(64 * kWavesPerGroup) void k_router_grad(RouterGradArgs a) {
  __shared__ float at_expert[kWavesPerGroup][64 * V];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int t = blockIdx.x * kWavesPerGroup + wv;
  if (t >= a.tokens) return;                     // no workgroup barrier below: a wave keeps to its own LDS row
  const int E = a.experts, k = a.top_k;
  const float lse = a.lse[t];
  const bool read = a.slope != nullptr || (a.dw != nullptr && !a.renormalize);   // the same for every row
  float v[V], slope[V], dl = 0.0f;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    v[j] = kNegInf;
    slope[j] = 0.0f;
  }
  if (read) load_row<D, V>(a.logits, a.stride, t, E, lane, v);
  if (a.slope) {
    dl = *a.dloss;
#pragma unroll
    for (int j = 0; j < V; ++j) slope[j] = 64 * j + lane < E ? a.slope[64 * j + lane] : 0.0f;
  }
  long long e = -1;
  float w = 0.0f, dw = 0.0f;
  if (a.dw && lane < k) {
    const long long at = static_cast<long long>(t) * k + lane;
    e = read_id(a.ids, a.ids64, at);
    w = a.w[at];
    dw = a.dw[at];
  }
  const bool in = lse != kNegInf;
  const bool soft = lse > kNegInf ? read : in && a.dw != nullptr && !a.renormalize;
  float* mine = at_expert[wv];
  float dot = 0.0f;
  if (a.dw) {
#pragma unroll
    for (int j = 0; j < V; ++j) mine[64 * j + lane] = 0.0f;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    const bool routed = in && e >= 0 && e < E;
    const float g = routed ? w * dw : 0.0f;
    dot = wave_sum(g);
    if (routed) atomicAdd(&mine[e], a.renormalize ? g - w * dot : g);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");   // the row's LDS entries are read across lanes below
  }
  float inv = 0.0f, mean = 0.0f;
  if (soft) {
    inv = row_softmax<V>(v, lse);
    if (a.slope) {
#pragma unroll
      for (int j = 0; j < V; ++j) mean += v[j] * inv * slope[j];
      mean = wave_sum(mean);
    }
  }
  const float all = a.dw != nullptr && !a.renormalize ? dot : 0.0f;
  typename D::T* out = static_cast<typename D::T*>(a.dlogits) + static_cast<long long>(t) * E;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int x = 64 * j + lane;
    float d = a.dw ? mine[x] : 0.0f;
    if (soft) {
      const float p = v[j] * inv;
      d += p * (dl * (slope[j] - mean) - all);
    }
    if (x < E) out[x] = D::put(d);
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
                           dim3(64 * kBalanceWaves), 0, s, a);
      });
    });
  hipLaunchKernelGGL(k_balance_finish, dim3((a.experts + 31) / 32), dim3(256), 0, s, a);
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
