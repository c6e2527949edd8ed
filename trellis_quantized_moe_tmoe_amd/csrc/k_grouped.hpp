// k_grouped.hpp -- products grouped by expert over ragged rows: y_r = W_e x_r, dx_r = W_e^T dy_r and
// dW_e = sum_r dy_r x_r^T, for bf16 and fp16 operands, and the first one for MXFP8 operands.
//
// A workgroup of four wavefronts computes TR rows by TC columns of one group with 32x32 matrix instructions
// (v_mfma_f32_32x32x16 for 16-bit values, v_mfma_scale_f32_32x32x64 for MXFP8), sums in fp32. The columns are the
// instruction's first operand, so that a lane's results are neighbouring columns of one row.
//
// The depth passes through a ring of slots in LDS, 128 bytes of it a row and slot (64 or 128 values), copied from
// global memory straight to LDS. An operand comes in one of two layouts:
//  * KC, its depth contiguous (x, dy and W in the linear product): 128-byte rows; the 16-byte chunk c of row r lies at
//    place c ^ swizzle(r), so that the 16-byte reads of 8 or 16 neighbouring rows touch every bank once;
//  * KS, its depth along its rows (W in grad_x, both operands of grad_w): 64 rows of T values, read by
//    ds_read_b64_tr_b16, which hands each lane four values of one column; chunk c of row k lies at place
//    c ^ 4 (k % 4), so that the four rows that half a wavefront reads lie in different banks.
// The copies write LDS in lane order, so the swizzles are in the lanes' global addresses. They are range-checked
// buffer loads that give zeros past the end: rows past the group's, columns past the last and depth past K all become
// zeros in LDS and need no masks in the loop.
//
// Per slot there are four sub-steps; each multiplies fragments that were read from LDS during the one before. One barrier
// a slot, in front of its last sub-step: by then every wavefront has read all of the slot, and the copies of the slot
// that follows the ring go there.
#pragma once
#include <algorithm>
#include <type_traits>

#include "tmoe.h"
#include "tmoe_device.hpp"
#include "tmoe_grouped.hpp"

namespace tmoe {

namespace {

enum { kKindBf16 = 0, kKindF16 = 1, kKindMx8 = 2 };

typedef int i4v __attribute__((ext_vector_type(4)));
typedef float f16v __attribute__((ext_vector_type(16)));
typedef short s4v __attribute__((ext_vector_type(4)));
typedef __bf16 bf8v __attribute__((ext_vector_type(8)));
typedef __bf16 bf4v __attribute__((ext_vector_type(4)));
typedef _Float16 hf8v __attribute__((ext_vector_type(8)));
typedef _Float16 hf4v __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) uint8_t lds_u8;

__device__ __forceinline__ int swizzle(int r) { return ((r >> 1) & 7) ^ ((r & 1) << 2); }

constexpr int kRsrcFlags = 0x00027000;           // raw buffer, 32-bit data
constexpr int kPastEnd = static_cast<int>(0x80000000u);   // an offset outside every buffer

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const uint8_t* p, long long bytes) {
  const int n = static_cast<int>(bytes < 0 ? 0 : bytes > 0x7fffffff ? 0x7fffffff : bytes);
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p), 0, n, kRsrcFlags);
}

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

template <int KIND, int WT_, int WC_, int MT_, int NT_, int SLOTS_>
struct GTile {
  static constexpr int WT = WT_, WC = WC_, MT = MT_, NT = NT_, SLOTS = SLOTS_;
  static constexpr int ES = KIND == kKindMx8 ? 1 : 2;             // bytes a value
  static constexpr int DEPTH = 128 / ES;                          // depth of a slot
  static constexpr int TR = 32 * MT * WT, TC = 32 * NT * WC;
  static constexpr int kSlot = (TR + TC) * 128;
  static constexpr int kScaleRows = KIND == kKindMx8 ? TC + (TR + 63) / 64 * 64 : 0;
  static constexpr int kScaleSlot = 4 * kScaleRows;               // a dword a row
  static constexpr int kLds = SLOTS * (kSlot + kScaleSlot);
  static constexpr int SPW = (kScaleRows / 64 + 3) / 4;           // scale copies a wavefront and slot
  static constexpr int COPIES = (TR + TC) / 32 + SPW;             // copies a wavefront issues a slot
  static_assert(WT * WC == 4, "four wavefronts");
};

// A tile's place in the work: rows [row0, row0 + nrows) of the row operand (grad_w: output rows), columns from col0.
struct GroupedTile {
  long long expert;
  int row0, nrows, col0;
  int k0, depth;             // grad_w: the group's first row and row count; else 0 and the depth
  bool zero;                 // rows outside every group: zeros
};

__device__ __forceinline__ int read_offset(const GroupedArgs& a, int e) {
  const long long o = a.off64 ? static_cast<const long long*>(a.offsets)[e] : static_cast<const int*>(a.offsets)[e];
  return static_cast<int>(o < 0 ? 0 : o > a.rows ? a.rows : o);   // never outside the rows
}

template <int KIND>
__device__ __forceinline__ f16v mma(i4v c, i4v r, f16v acc) {
  if constexpr (KIND == kKindBf16)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf8v, c), __builtin_bit_cast(bf8v, r), acc, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(hf8v, c), __builtin_bit_cast(hf8v, r), acc, 0, 0, 0);
}

// Both kinds of operands give fp32 sums, but the 8-bit unit (with and without scales alike; measured on single products)
// aligns 16 neighbouring products to the largest of their powers of two and cuts each 13 bits below it before it adds them;
// sums of 16 are added in fp32. That is at most 16 * 2^-13 of the largest product for every 16 of the depth. Taken for
// twice the rate of bf16 products of decoded values (which would be exact): the operands themselves are rounded to 2^-4.
template <int STEP>                              // byte 2 STEP of the scale words
__device__ __forceinline__ f16v mma8(i8v c, int cs, i8v r, int rs, f16v acc) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(c, r, acc, 0, 0, 2 * STEP, cs, 2 * STEP, rs);
}

// Four depth values of this lane's column. The pointer is restrict (nothing else is written while this one read runs): without
// that the compiler puts a wait for every copy in flight in front of each of these reads (dW at 4096 x 4096 x 4096: 210 us);
// the loop has its own waits.
typedef __attribute__((address_space(3))) s4v lds_s4;
__device__ __forceinline__ s4v tr_read4(lds_s4* __restrict__ p) { return __builtin_amdgcn_ds_read_tr16_b64_v4i16(p); }

// Eight: from rows 4 apart.
__device__ __forceinline__ i4v tr_read(lds_u8* p, int next) {
  return __builtin_bit_cast(i4v, __builtin_shufflevector(tr_read4((lds_s4*)p), tr_read4((lds_s4*)(p + next)), 0, 1, 2, 3, 4, 5, 6, 7));
}

// One operand's copies: T rows (KC) or columns (KS) of a tile.
template <int T, bool KS, int ES>
struct Operand {
  const uint8_t* base;       // KC: first row; KS: first depth row
  long long pitch;           // bytes from row to row
  int rows;                  // KC: rows that exist; KS: depth rows that exist
  int depth_bytes;           // KC: bytes of a row
  int first;                 // offset of copy 0 of this lane
  int step;                  // from copy to copy
  int at;                    // KC: this lane's byte within the slot's 128

  static constexpr int N = T / 32;               // copies a wavefront and slot

  __device__ __forceinline__ void point(const uint8_t* p, int pitch_bytes, int n, int depth, int col0, int width, int wv, int lane) {
    pitch = pitch_bytes;
    rows = n;
    if constexpr (KS) {
      constexpr int CH = T / 8, RP = 64 / CH;    // chunks a depth row, depth rows a copy
      const int k = RP * wv + lane / CH, c = (lane % CH) ^ (4 * (k & 3));
      base = p;
      first = k * pitch_bytes + col0 * 2 + 16 * c;
      if (col0 + 8 * c >= width) first = kPastEnd;
      step = 4 * RP * pitch_bytes;
    } else {
      const int r = 8 * wv + (lane >> 3);
      at = 16 * ((lane & 7) ^ swizzle(8 * (wv & 1) + (lane >> 3)));
      base = p;
      depth_bytes = depth * ES;
      first = r * pitch_bytes + at;
      step = 32 * pitch_bytes;
    }
  }
  __device__ __forceinline__ __amdgpu_buffer_rsrc_t window(int slot) const {
    if constexpr (KS) {
      const long long from = 64LL * slot;
      const long long n = rows - from;
      return rsrc(base + from * pitch, (n < 64 ? n : 64) * pitch);
    } else {
      return rsrc(base + 128LL * slot, static_cast<long long>(rows) * pitch - 128LL * slot);
    }
  }
  // offset of copy i; behind the row's end: outside
  __device__ __forceinline__ int offset(int slot, int i) const {
    if constexpr (KS) return first < 0 ? first : first + i * step;
    else return 128 * slot + at < depth_bytes ? first + i * step : kPastEnd;
  }
};

template <int KIND, bool RKS, bool CKS, class S, int OUT, bool SCALES4>
__device__ __forceinline__ void grouped_body(const GroupedArgs& a, const GroupedTile& t, uint8_t* lds) {
  constexpr bool MX = KIND == kKindMx8;
  constexpr int MT = S::MT, NT = S::NT, SUBS = MX ? 2 : 4;
  const int tid = threadIdx.x, lane = tid & 63, wv = uniform(tid >> 6);
  const int r32 = lane & 31, h = lane >> 5, wt = wv / S::WC, wc = wv % S::WC;
  const int row_pitch = (RKS ? a.out_rows : a.depth) * S::ES;
  const int col_pitch = (CKS ? a.cols : a.depth) * S::ES;

  Operand<S::TR, RKS, S::ES> R;
  Operand<S::TC, CKS, S::ES> C;
  const uint8_t* rp = static_cast<const uint8_t*>(a.r);
  const uint8_t* cp = static_cast<const uint8_t*>(a.c);
  if constexpr (RKS) R.point(rp + static_cast<long long>(t.k0) * row_pitch, row_pitch, t.depth, 0, t.row0, a.out_rows, wv, lane);
  else R.point(rp + static_cast<long long>(t.row0) * row_pitch, row_pitch, t.nrows, a.depth, 0, 0, wv, lane);
  if constexpr (RKS)                             // grad_w: x, beside dy
    C.point(cp + static_cast<long long>(t.k0) * col_pitch, col_pitch, t.depth, 0, t.col0, a.cols, wv, lane);
  else if constexpr (CKS)
    C.point(cp + t.expert * a.depth * col_pitch, col_pitch, a.depth, 0, t.col0, a.cols, wv, lane);
  else
    C.point(cp + (t.expert * a.cols + t.col0) * col_pitch, col_pitch, min(S::TC, a.cols - t.col0), a.depth, 0, 0, wv, lane);
  const int slots = t.zero ? 0 : (t.depth + S::DEPTH - 1) / S::DEPTH;

  lds_u8* const ring = (lds_u8*)lds;
  auto issue = [&](int slot, int place, int i, __amdgpu_buffer_rsrc_t rr, __amdgpu_buffer_rsrc_t cr) {
    if (i < C.N)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(cr, (__attribute__((address_space(3))) void*)(ring + place * S::kSlot + S::TR * 128 + (wv + 4 * i) * 1024),
                                               16, C.offset(slot, i), 0, 0, 0);
    else
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rr, (__attribute__((address_space(3))) void*)(ring + place * S::kSlot + (wv + 4 * (i - C.N)) * 1024),
                                               16, R.offset(slot, i - C.N), 0, 0, 0);
  };
  // MXFP8 scales, four bytes a row and slot: columns first, then rows. SCALES4: rows of whole dwords, copied like the codes.
  const int nblk = MX ? a.depth / 32 : 0;
  auto issue_scales = [&](int slot, int place) {
    if constexpr (MX && SCALES4) {
      constexpr int CN = S::TC / 64, ALL = S::kScaleRows / 64;
#pragma unroll
      for (int i = 0; i < S::SPW; ++i) {
        const int j = min(wv + 4 * i, ALL - 1);
        const bool col = j < CN;
        const int row = 64 * (col ? j : j - CN) + lane, n = col ? min(S::TC, a.cols - t.col0) : t.nrows;
        const uint8_t* p = col ? a.cs + (t.expert * a.cols + t.col0) * nblk : a.rs + static_cast<long long>(t.row0) * nblk;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            rsrc(p + 4LL * slot, static_cast<long long>(n) * nblk - 4LL * slot),
            (__attribute__((address_space(3))) void*)(ring + S::SLOTS * S::kSlot + place * S::kScaleSlot + 256 * j), 4,
            4 * slot < nblk ? row * nblk : kPastEnd, 0, 0, 0);
      }
    }
  };

  struct Frags {
    i4v r[MT][MX ? 2 : 1], c[NT][MX ? 2 : 1];
    int rs[MT], cs[NT];
  };
  // An 8-bit operand of the 32x32x64 instruction: half h of the wavefront holds the bytes 16 h .. of both 32-blocks, and the
  // scale of block h.
  // KC: places of this lane's chunks; KS: byte offset of its first value, by fragment
  int chunk_at[4];                               // MXFP8: chunk 4 s + 2 j + h at [2 s + j]; else chunk 2 s + h at [s]
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c = MX ? 4 * (i >> 1) + 2 * (i & 1) + h : 2 * i + h;
    chunk_at[i] = 128 * r32 + 16 * (c ^ swizzle(r32));
  }
  int tr_r[MT], tr_c[NT];
  {
    const int i = lane & 15, g = (lane >> 4) & 1, m = i >> 2, k = 8 * h + m;
    const int in = 16 * (2 * g + ((i & 3) >> 1)) + 8 * (i & 1);
    if constexpr (RKS) {
#pragma unroll
      for (int f = 0; f < MT; ++f) tr_r[f] = k * 2 * S::TR + 64 * ((wt * MT + f) ^ m) + in;
    }
    if constexpr (CKS) {
#pragma unroll
      for (int f = 0; f < NT; ++f) tr_c[f] = k * 2 * S::TC + 64 * ((wc * NT + f) ^ m) + in;
    }
  }
  typedef __attribute__((address_space(3))) i4v lds_i4;
  typedef __attribute__((address_space(3))) int lds_i;
  // unaligned scales: straight from global memory, a byte a block
  auto scale_bytes = [&](const uint8_t* p, int n, int row, int slot) {
    const uint8_t* q = p + static_cast<long long>(min(row, n - 1)) * nblk;
    int w = 0;
#pragma unroll
    for (int b = 0; b < 4; ++b) w |= 4 * slot + b < nblk ? q[4 * slot + b] << (8 * b) : 0;
    return w;
  };
  auto read_piece = [&](int slot, int place, int s, int p, Frags& f) {
    lds_u8* const base = ring + place * S::kSlot;
    if (p < NT) {
      lds_u8* const at = base + S::TR * 128;
      if constexpr (CKS) {
        f.c[p][0] = tr_read(at + tr_c[p] + s * 16 * 2 * S::TC, 4 * 2 * S::TC);
      } else {
        const int fr = 4096 * (wc * NT + p);
        if constexpr (MX) {
          f.c[p][0] = *(lds_i4*)(at + fr + chunk_at[2 * s]);
          f.c[p][1] = *(lds_i4*)(at + fr + chunk_at[2 * s + 1]);
          if (s == 0) {
            const int row = 32 * (wc * NT + p) + r32;
            int w;
            if constexpr (SCALES4) w = *(lds_i*)(ring + S::SLOTS * S::kSlot + place * S::kScaleSlot + 4 * row);
            else w = scale_bytes(a.cs + (t.expert * a.cols + t.col0) * nblk, a.cols - t.col0, row, slot);
            f.cs[p] = static_cast<int>(static_cast<uint32_t>(w) >> (8 * h));
          }
        } else {
          f.c[p][0] = *(lds_i4*)(at + fr + chunk_at[s]);
        }
      }
    } else {
      const int m = p - NT;
      if constexpr (RKS) {
        f.r[m][0] = tr_read(base + tr_r[m] + s * 16 * 2 * S::TR, 4 * 2 * S::TR);
      } else {
        const int fr = 4096 * (wt * MT + m);
        if constexpr (MX) {
          f.r[m][0] = *(lds_i4*)(base + fr + chunk_at[2 * s]);
          f.r[m][1] = *(lds_i4*)(base + fr + chunk_at[2 * s + 1]);
          if (s == 0) {
            const int row = 32 * (wt * MT + m) + r32;
            int w;
            if constexpr (SCALES4) w = *(lds_i*)(ring + S::SLOTS * S::kSlot + place * S::kScaleSlot + 4 * (S::TC + row));
            else w = scale_bytes(a.rs + static_cast<long long>(t.row0) * nblk, t.nrows, row, slot);
            f.rs[m] = static_cast<int>(static_cast<uint32_t>(w) >> (8 * h));
          }
        } else {
          f.r[m][0] = *(lds_i4*)(base + fr + chunk_at[s]);
        }
      }
    }
  };

  f16v acc[MT][NT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[m][n] = f16v{};

  if (slots > 0) {
#pragma unroll
    for (int d = 0; d < S::SLOTS; ++d) {
      issue_scales(d, d);
      const auto rr = R.window(d), cr = C.window(d);
#pragma unroll
      for (int i = 0; i < R.N + C.N; ++i) issue(d, d, i, rr, cr);
    }
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"((S::SLOTS - 1) * S::COPIES) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    Frags f[2];
#pragma unroll
    for (int p = 0; p < MT + NT; ++p) read_piece(0, 0, 0, p, f[0]);
    constexpr int MM = MT * NT, RD = MT + NT, CP = R.N + C.N;
    int place = 0;
    for (int slot = 0; slot < slots; ++slot) {
      const int next = place + 1 == S::SLOTS ? 0 : place + 1;
      int rs[MT], cs[NT];
      if constexpr (MX) {
#pragma unroll
        for (int m = 0; m < MT; ++m) rs[m] = f[0].rs[m];
#pragma unroll
        for (int n = 0; n < NT; ++n) cs[n] = f[0].cs[n];
      }
      const auto rr = R.window(slot + S::SLOTS), cr = C.window(slot + S::SLOTS);
#pragma unroll
      for (int s = 0; s < SUBS; ++s) {
        Frags &cur = f[s & 1], &nxt = f[(s + 1) & 1];
        const bool last = s == SUBS - 1;
        if (last) {
          asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"((S::SLOTS - 2) * S::COPIES) : "memory");
          __builtin_amdgcn_s_barrier();
          asm volatile("" ::: "memory");
          issue_scales(slot + S::SLOTS, place);
        }
#pragma unroll
        for (int j = 0; j < MM; ++j) {
          constexpr int per = (RD + MM - 1) / MM;
#pragma unroll
          for (int p = j * per; p < (j + 1) * per && p < RD; ++p)
            read_piece(last ? slot + 1 : slot, last ? next : place, last ? 0 : s + 1, p, nxt);
          if (last) {
#pragma unroll
            for (int i = j * CP / MM; i < (j + 1) * CP / MM; ++i) issue(slot + S::SLOTS, place, i, rr, cr);
          }
          __builtin_amdgcn_sched_barrier(0);
          const int m = j / NT, n = j % NT;
          if constexpr (MX) {
            const i8v c8 = __builtin_shufflevector(cur.c[n][0], cur.c[n][1], 0, 1, 2, 3, 4, 5, 6, 7);
            const i8v r8 = __builtin_shufflevector(cur.r[m][0], cur.r[m][1], 0, 1, 2, 3, 4, 5, 6, 7);
            acc[m][n] = s == 0 ? mma8<0>(c8, cs[n], r8, rs[m], acc[m][n]) : mma8<1>(c8, cs[n], r8, rs[m], acc[m][n]);
          } else {
            acc[m][n] = mma<KIND>(cur.c[n][0], cur.r[m][0], acc[m][n]);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      place = next;
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // copies past the end land before LDS is used again
  }

  // Results leave through the wavefront's own part of LDS, 32 rows at a time, so that a store covers whole rows.
  constexpr int OS = OUT == TMOE_F32 ? 4 : 2, EPL = 16 / OS, PITCH = 32 * NT * OS + 16;
  static_assert(4 * 32 * PITCH <= S::kLds, "four wavefronts' rows fit the ring");
  const int wcol = t.col0 + 32 * NT * wc;
  uint8_t* y = static_cast<uint8_t*>(a.y);
  if constexpr (RKS) y += t.expert * a.out_rows * a.cols * OS;
  __syncthreads();
  uint8_t* mine = lds + wv * 32 * PITCH;
#pragma unroll
  for (int m = 0; m < MT; ++m) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const f4 v = {acc[m][n][4 * q], acc[m][n][4 * q + 1], acc[m][n][4 * q + 2], acc[m][n][4 * q + 3]};
        uint8_t* to = mine + r32 * PITCH + (32 * n + 8 * q + 4 * h) * OS;
        if constexpr (OUT == TMOE_BF16) *reinterpret_cast<bf4v*>(to) = __builtin_convertvector(v, bf4v);
        else if constexpr (OUT == TMOE_F16) *reinterpret_cast<hf4v*>(to) = __builtin_convertvector(v, hf4v);
        else *reinterpret_cast<f4*>(to) = v;
      }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    constexpr int LPR = 32 * NT / EPL, RPI = 64 / LPR;
    const int c = wcol + (lane % LPR) * EPL;
#pragma unroll
    for (int i = 0; i < 32 / RPI; ++i) {
      const int r = RPI * i + lane / LPR, row = 32 * (wt * MT + m) + r;
      const i4v v = *reinterpret_cast<const i4v*>(mine + r * PITCH + (lane % LPR) * 16);
      if (row < t.nrows && c < a.cols)
        *reinterpret_cast<i4v*>(y + (static_cast<long long>(t.row0 + row) * a.cols + c) * OS) = v;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
}

// The tile list is implied by the offsets: expert e has ceil(rows / TR) row tiles; the rows in front of the first group
// and behind the last come after all experts. Each workgroup finds its own tile by one scan (two experts a thread).
// The tiles are dealt to the eight XCDs in contiguous runs (workgroups go to the XCDs in turn), within an expert in
// groups of four row tiles, so that an XCD's L2 holds what its tiles share.
template <class S>
__device__ __forceinline__ bool find_tile(const GroupedArgs& a, int col_tiles, int* sh, GroupedTile& t) {
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6, E = a.experts;
  int lo[2], n[2], cnt[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int e = 2 * tid + i;
    lo[i] = read_offset(a, min(e, E));
    const int hi = read_offset(a, min(e + 1, E));
    n[i] = max(0, hi - lo[i]);
    cnt[i] = (n[i] + S::TR - 1) / S::TR;
  }
  int sum = cnt[0] + cnt[1];
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(sum, d, 64);
    if (lane >= d) sum += o;
  }
  if (lane == 63) sh[wv] = sum;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    if (p < wv) before += sh[p];
    all += sh[p];
  }
  const int front = uniform(read_offset(a, 0)), back = uniform(read_offset(a, E));
  const int ft = (front + S::TR - 1) / S::TR, bt = (a.rows - back + S::TR - 1) / S::TR;
  all = uniform(all);
  const long long total = static_cast<long long>(all + ft + bt) * col_tiles;
  const long long per = (total + 7) / 8, j = blockIdx.x / 8;
  const long long w = (blockIdx.x % 8) * per + j;
  if (j >= per || w >= total) return false;                  // the same for the whole workgroup
  const int rt = static_cast<int>(w / col_tiles);
  int ex = before + sum - cnt[0] - cnt[1];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (rt >= ex && rt < ex + cnt[i]) {
      sh[4] = 2 * tid + i;
      sh[5] = lo[i];
      sh[6] = n[i];
      sh[7] = ex;
    }
    ex += cnt[i];
  }
  __syncthreads();
  t.zero = rt >= all;
  t.k0 = 0;
  t.depth = a.depth;
  if (t.zero) {
    const int z = rt - all;
    t.expert = 0;
    t.row0 = z < ft ? z * S::TR : back + (z - ft) * S::TR;
    t.nrows = min(S::TR, (z < ft ? front : a.rows) - t.row0);
    t.col0 = static_cast<int>(w % col_tiles) * S::TC;
    return true;
  }
  const int rows = uniform(sh[6]), first = uniform(sh[7]), tiles = (rows + S::TR - 1) / S::TR;
  constexpr int G = 4;
  const int in = static_cast<int>(w - static_cast<long long>(first) * col_tiles);   // within the expert
  const int g = in / (G * col_tiles), at = in % (G * col_tiles), rg = min(G, tiles - g * G);
  const int r = g * G + at % rg;
  t.expert = uniform(sh[4]);
  t.row0 = uniform(sh[5]) + r * S::TR;
  t.nrows = min(S::TR, rows - r * S::TR);
  t.col0 = at / rg * S::TC;
  return true;
}

template <int KIND, bool CKS, class S, int OUT, bool SCALES4>
__global__ __launch_bounds__(256, S::kLds > 81920 ? 1 : 2) void k_grouped_rows(GroupedArgs a, int col_tiles) {
  __shared__ __align__(16) uint8_t lds[S::kLds];
  GroupedTile t;
  if (!find_tile<S>(a, col_tiles, reinterpret_cast<int*>(lds), t)) return;
  __syncthreads();
  grouped_body<KIND, false, CKS, S, OUT, SCALES4>(a, t, lds);
}

template <int KIND, class S, int OUT>
__global__ __launch_bounds__(256, S::kLds > 81920 ? 1 : 2) void k_grouped_grad_w(GroupedArgs a, int row_tiles, int col_tiles) {
  __shared__ __align__(16) uint8_t lds[S::kLds];
  const long long per_expert = static_cast<long long>(row_tiles) * col_tiles, total = per_expert * a.experts;
  const long long per = gridDim.x / 8;
  const long long w = (blockIdx.x % 8) * per + blockIdx.x / 8;
  if (w >= total) return;
  GroupedTile t;
  t.expert = w / per_expert;
  const int in = static_cast<int>(w - t.expert * per_expert);
  const int e = static_cast<int>(t.expert);
  t.k0 = uniform(read_offset(a, e));
  t.depth = max(0, uniform(read_offset(a, e + 1)) - t.k0);
  t.zero = false;
  constexpr int G = 4;
  const int g = in / (G * col_tiles), at = in % (G * col_tiles), rg = min(G, row_tiles - g * G);
  t.row0 = (g * G + at % rg) * S::TR;
  t.nrows = min(S::TR, a.out_rows - t.row0);
  t.col0 = at / rg * S::TC;
  grouped_body<KIND, true, true, S, OUT, false>(a, t, lds);
}

constexpr long long kMaxGroups = (1LL << 24) - 8;   // workgroups of 256 threads: a launch has fewer than 2^32 threads

template <int KIND, bool CKS, class S, int OUT, bool SCALES4>
bool launch_rows(const GroupedArgs& a, hipStream_t s) {
  const int ct = (a.cols + S::TC - 1) / S::TC;
  // every row tile but a group's last is full, the rows in front and behind are two groups more
  const long long tiles = std::min<long long>(a.rows, a.experts + 2 + a.rows / S::TR);
  const long long g = (tiles * ct + 7) / 8 * 8;
  if (g > kMaxGroups) return false;
  hipLaunchKernelGGL((k_grouped_rows<KIND, CKS, S, OUT, SCALES4>), dim3(static_cast<unsigned>(g)), dim3(256), 0, s, a, ct);
  return true;
}

template <int KIND, class S, int OUT>
bool launch_grad_w(const GroupedArgs& a, hipStream_t s) {
  const int rt = (a.out_rows + S::TR - 1) / S::TR, ct = (a.cols + S::TC - 1) / S::TC;
  const long long g = (static_cast<long long>(rt) * ct * a.experts + 7) / 8 * 8;
  if (g > kMaxGroups) return false;
  hipLaunchKernelGGL((k_grouped_grad_w<KIND, S, OUT>), dim3(static_cast<unsigned>(g)), dim3(256), 0, s, a, rt, ct);
  return true;
}

template <int KIND> using Few = GTile<KIND, 1, 4, 1, 1, 2>;    // 32 x 128
template <int KIND> using Mid = GTile<KIND, 2, 2, 2, 2, 2>;    // 128 x 128
template <int KIND> using Big = GTile<KIND, 2, 2, 4, 4, 2>;    // 256 x 256

template <int KIND, bool CKS, int OUT, bool SCALES4>
bool launch_rows_by_size(const GroupedArgs& a, hipStream_t s) {
  if (a.rows <= 16LL * a.experts) return launch_rows<KIND, CKS, Few<KIND>, OUT, SCALES4>(a, s);
  if constexpr (KIND != kKindMx8 || SCALES4) {   // byte loads of scales leave no registers for 256 x 256
    if (a.rows >= 1024LL * a.experts) return launch_rows<KIND, CKS, Big<KIND>, OUT, SCALES4>(a, s);
  }
  return launch_rows<KIND, CKS, Mid<KIND>, OUT, SCALES4>(a, s);
}

template <int KIND, int OUT>
bool launch_16bit(const GroupedArgs& a, int op, hipStream_t s) {
  if (op == kGroupedLinear) return launch_rows_by_size<KIND, false, OUT, false>(a, s);
  if (op == kGroupedGradX) return launch_rows_by_size<KIND, true, OUT, false>(a, s);
  if (a.rows < 1024LL * a.experts) return launch_grad_w<KIND, Mid<KIND>, OUT>(a, s);
  return launch_grad_w<KIND, Big<KIND>, OUT>(a, s);
}

}  // namespace

}  // namespace tmoe
