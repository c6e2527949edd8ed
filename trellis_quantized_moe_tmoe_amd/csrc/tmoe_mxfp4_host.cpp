// tmoe_mxfp4_host.cpp -- C ABI of the MXFP4 calls: argument checks, the layer's plan, scratch layout and
// launch sequence. Every argument is checked before the first launch; nothing is allocated on the
// device and nothing synchronizes.
#include <algorithm>
#include <cstdint>
#include <cstring>
#include <new>

#include <hip/hip_runtime.h>

#include "tmoe.h"
#include "tmoe_internal.hpp"
#include "tmoe_mxfp4.hpp"

using namespace tmoe;

struct tmoe_mxfp4_plan_s {
  int H, I, E, K, max_tokens, ids64, y_dtype;
  int max_tiles, max_gtiles;                     // of the largest batch (exported and product tiles)
  size_t einfo, counts, offsets, sorted, slot_e, slot, tile_e, tile_r0, tile_rows, scalars, gtiles, wgc;
  size_t xq, xs, bq, bs, v, total;
};

namespace {

constexpr int kMaxExperts = 512;
constexpr int kMaxTopK = 32;
constexpr int kMaxDim = 8192;                    // of the layer
constexpr int kMaxLinearDim = 1 << 16;
constexpr int kMaxLinearTokens = 1 << 20;
constexpr long long kMaxRoutes = 1LL << 22;
constexpr long long kMaxValues = 1LL << 33;      // T * H: the weighted sum has a thread for four, a launch fewer than 2^32
constexpr int kBlockM = 64;                      // rows of the route map's own tile table (not read here)

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

template <class T>
T* at(void* base, size_t off) { return reinterpret_cast<T*>(static_cast<char*>(base) + off); }

tmoe_status launched() { return hipGetLastError() == hipSuccess ? TMOE_OK : TMOE_ERR_HIP; }

bool dtype_ok(int d) { return d == TMOE_F32 || d == TMOE_BF16 || d == TMOE_F16; }

tmoe_status check_blocks(const void* x, int32_t dtype, int64_t rows, int32_t cols, const void* codes,
                         const void* scales) {
  if (!dtype_ok(dtype) || rows < 0 || cols <= 0) return TMOE_ERR_INVALID_ARG;
  if (cols % 32 != 0 || rows > (int64_t{1} << 40) / cols) return TMOE_ERR_UNSUPPORTED;
  if (rows == 0) return TMOE_OK;
  if (!x || !codes || !scales) return TMOE_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(codes, 16)) return TMOE_ERR_ALIGNMENT;
  return TMOE_OK;
}

bool dim_ok(int n) { return n >= 32 && n <= kMaxDim && n % 32 == 0; }

}  // namespace

extern "C" {

tmoe_status tmoe_mxfp4_quantize(const void* x, int32_t dtype, int64_t rows, int32_t cols, uint8_t* codes,
                                uint8_t* scales, void* stream) {
  const tmoe_status st = check_blocks(x, dtype, rows, cols, codes, scales);
  if (st != TMOE_OK || rows == 0) return st;
  Mxfp4QuantArgs a;
  a.x = x;
  a.groups = rows * cols / 8;
  a.codes = codes;
  a.scales = scales;
  (void)hipGetLastError();
  launch_mxfp4_quantize(a, dtype, static_cast<hipStream_t>(stream));
  return launched();
}

tmoe_status tmoe_mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int32_t cols,
                                  int32_t dtype, void* x, void* stream) {
  const tmoe_status st = check_blocks(x, dtype, rows, cols, codes, scales);
  if (st != TMOE_OK || rows == 0) return st;
  Mxfp4DequantArgs a;
  a.codes = codes;
  a.scales = scales;
  a.groups = rows * cols / 8;
  a.x = x;
  (void)hipGetLastError();
  launch_mxfp4_dequantize(a, dtype, static_cast<hipStream_t>(stream));
  return launched();
}

tmoe_status tmoe_linear_mxfp4(const uint8_t* xq, const uint8_t* xs, int32_t T, const uint8_t* wq, const uint8_t* ws,
                              int32_t K, int32_t N, int32_t y_dtype, void* y, void* stream) {
  if (T < 0 || K <= 0 || N <= 0 || (y_dtype != TMOE_F32 && y_dtype != TMOE_BF16)) return TMOE_ERR_INVALID_ARG;
  if (K % 32 != 0 || K > kMaxLinearDim || N > kMaxLinearDim || T > kMaxLinearTokens) return TMOE_ERR_UNSUPPORTED;
  if (T == 0) return TMOE_OK;
  if (!xq || !xs || !wq || !ws || !y) return TMOE_ERR_INVALID_ARG;
  if (!aligned(xq, 16) || !aligned(wq, 16) || !aligned(y, 16)) return TMOE_ERR_ALIGNMENT;
  Mxfp4GemmArgs a;
  std::memset(&a, 0, sizeof(a));
  a.xq = xq;
  a.xs = xs;
  a.wq = wq;
  a.ws = ws;
  a.K = K;
  a.N = N;
  a.rows = T;
  a.y = y;
  (void)hipGetLastError();
  launch_mxfp4_dense(a, y_dtype, static_cast<hipStream_t>(stream));
  return launched();
}

tmoe_status tmoe_mxfp4_plan(const tmoe_mxfp4_config* c, tmoe_mxfp4_plan_t* out, size_t* scratch_bytes) {
  if (!c || !out) return TMOE_ERR_INVALID_ARG;
  *out = nullptr;
  if (c->hidden <= 0 || c->inter <= 0 || c->num_experts <= 0 || c->top_k <= 0 || c->max_tokens <= 0)
    return TMOE_ERR_INVALID_ARG;
  if (c->ids_dtype != TMOE_IDS_I32 && c->ids_dtype != TMOE_IDS_I64) return TMOE_ERR_INVALID_ARG;
  if (c->y_dtype != TMOE_F32 && c->y_dtype != TMOE_BF16) return TMOE_ERR_INVALID_ARG;
  if (!dim_ok(c->hidden) || !dim_ok(c->inter)) return TMOE_ERR_UNSUPPORTED;
  if (c->num_experts > kMaxExperts || c->top_k > kMaxTopK) return TMOE_ERR_UNSUPPORTED;
  const long long R = static_cast<long long>(c->max_tokens) * c->top_k;
  if (R > kMaxRoutes || static_cast<long long>(c->max_tokens) * c->hidden > kMaxValues) return TMOE_ERR_UNSUPPORTED;
  tmoe_mxfp4_plan_s* p = new (std::nothrow) tmoe_mxfp4_plan_s();
  if (!p) return TMOE_ERR_INVALID_ARG;
  p->H = c->hidden;
  p->I = c->inter;
  p->E = c->num_experts;
  p->K = c->top_k;
  p->max_tokens = c->max_tokens;
  p->ids64 = c->ids_dtype == TMOE_IDS_I64;
  p->y_dtype = c->y_dtype;
  p->max_tiles = static_cast<int>(R / kBlockM + p->E + 1);
  p->max_gtiles = static_cast<int>(R / 16 + p->E + 1);
  const size_t r = static_cast<size_t>(R), T = static_cast<size_t>(c->max_tokens);
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = (off + bytes + 255) / 256 * 256;
    return o;
  };
  p->einfo = take(sizeof(ExpertInfo) * p->E);
  p->counts = take(4ull * p->E);
  p->offsets = take(4ull * (p->E + 1));
  p->sorted = take(4 * r);
  p->slot_e = take(4 * r);
  p->slot = take(4 * r);
  p->tile_e = take(4ull * p->max_tiles);
  p->tile_r0 = take(4ull * p->max_tiles);
  p->tile_rows = take(4ull * p->max_tiles);
  p->scalars = take(32);                         // exported tiles, dropped routes, product tiles, splits[2]
  p->gtiles = take(16ull * p->max_gtiles);
  p->wgc = take(4ull * ((r + kRouteChunk - 1) / kRouteChunk) * (p->E + 1));
  p->xq = take(T * (p->H / 2));
  p->xs = take(T * (p->H / 32));
  p->bq = take(r * (p->I / 2));
  p->bs = take(r * (p->I / 32));
  p->v = take(4 * r * p->H);
  p->total = off;
  *out = p;
  if (scratch_bytes) *scratch_bytes = p->total;
  return TMOE_OK;
}

tmoe_status tmoe_mxfp4_plan_destroy(tmoe_mxfp4_plan_t plan) {
  if (!plan) return TMOE_ERR_INVALID_ARG;
  delete plan;
  return TMOE_OK;
}

tmoe_status tmoe_forward_mxfp4(tmoe_mxfp4_plan_t p, const void* x, const void* ids, const float* w, int32_t T,
                               const tmoe_mxfp4_weights* wt, void* y, void* scratch, size_t bytes, void* stream) {
  if (!p || T < 0) return TMOE_ERR_INVALID_ARG;
  if (T > p->max_tokens) return TMOE_ERR_CAPACITY;
  if (T == 0) return TMOE_OK;
  if (!scratch || !aligned(scratch, 16) || bytes < p->total) return TMOE_ERR_SCRATCH;
  if (!x || !ids || !w || !wt || !y || !wt->w1 || !wt->s1 || !wt->w2 || !wt->s2) return TMOE_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(y, 16) || !aligned(w, 4) || !aligned(ids, p->ids64 ? 8 : 4) ||
      !aligned(wt->w1, 16) || !aligned(wt->w2, 16))
    return TMOE_ERR_ALIGNMENT;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const long long R = static_cast<long long>(T) * p->K;
  const int rows = mxfp4_tile_rows(R, p->E);

  RouteMapArgs m;
  std::memset(&m, 0, sizeof(m));
  m.ids = ids;
  m.ids64 = p->ids64;
  m.routes = static_cast<int>(R);
  m.num_experts = p->E;
  m.block_m = kBlockM;
  m.gemm_rows = rows;
  m.counts = at<int32_t>(scratch, p->counts);
  m.offsets = at<int32_t>(scratch, p->offsets);
  m.sorted_routes = at<int32_t>(scratch, p->sorted);
  m.route_slot = at<int32_t>(scratch, p->slot);
  m.tile_expert = at<int32_t>(scratch, p->tile_e);
  m.tile_row0 = at<int32_t>(scratch, p->tile_r0);
  m.tile_rows = at<int32_t>(scratch, p->tile_rows);
  m.num_tiles = at<int32_t>(scratch, p->scalars);
  m.status = at<int32_t>(scratch, p->scalars) + 1;
  m.num_gtiles = at<int32_t>(scratch, p->scalars) + 2;
  m.splits = at<int32_t>(scratch, p->scalars) + 3;
  m.slot_expert = at<int32_t>(scratch, p->slot_e);
  m.wg_counts = at<int32_t>(scratch, p->wgc);
  m.gtiles = at<int4>(scratch, p->gtiles);
  m.einfo = at<ExpertInfo>(scratch, p->einfo);

  Mxfp4QuantArgs q;
  q.x = x;
  q.groups = static_cast<long long>(T) * p->H / 8;
  q.codes = at<uint8_t>(scratch, p->xq);
  q.scales = at<uint8_t>(scratch, p->xs);

  Mxfp4GemmArgs g;
  std::memset(&g, 0, sizeof(g));
  g.xq = q.codes;
  g.xs = q.scales;
  g.wq = wt->w1;
  g.ws = wt->s1;
  g.K = p->H;
  g.N = 2 * p->I;
  g.gtiles = m.gtiles;
  g.num_gtiles = m.num_gtiles;
  // every tile but an expert's last is full, and an expert without routes has none
  g.max_gtiles = rows == kFewRoutes ? 0 : static_cast<int>(std::min<long long>(R, p->E + R / rows));
  g.ids = ids;
  g.ids64 = p->ids64;
  g.routes = static_cast<int>(R);
  g.experts = p->E;
  g.sorted = m.sorted_routes;
  g.top_k = p->K;
  g.bq = at<uint8_t>(scratch, p->bq);
  g.bs = at<uint8_t>(scratch, p->bs);

  if (rows == kFewRoutes && p->H <= kQuantizeInPlaceMax) g.x = static_cast<const uint16_t*>(x);

  Mxfp4GemmArgs h = g;
  h.x = nullptr;
  h.xq = g.bq;
  h.xs = g.bs;
  h.wq = wt->w2;
  h.ws = wt->s2;
  h.K = p->I;
  h.N = p->H;
  h.y = at<float>(scratch, p->v);

  Mxfp4CombineArgs c;
  c.v = at<float>(scratch, p->v);
  c.route_slot = rows == kFewRoutes ? nullptr : m.route_slot;
  c.ids = ids;
  c.ids64 = p->ids64;
  c.experts = p->E;
  c.w = w;
  c.tokens = T;
  c.top_k = p->K;
  c.H = p->H;
  c.y = y;

  (void)hipGetLastError();
  if (rows != kFewRoutes) launch_route_map_mxfp4(m, q, s);
  else if (!g.x) launch_mxfp4_quantize(q, TMOE_BF16, s);
  launch_mxfp4_fc1(g, rows, s);
  launch_mxfp4_fc2(h, rows, s);
  launch_mxfp4_combine(c, p->y_dtype, s);
  return launched();
}

}  // extern "C"
