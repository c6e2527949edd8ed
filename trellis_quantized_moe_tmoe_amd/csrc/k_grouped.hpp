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
// Per slot there are two or four sub-steps; each multiplies fragments that were read from LDS during the one before. One barrier
// a slot (256 x 256 tiles: two), in front of its last sub-step: by then every wavefront has read all of the slot, and the
// copies of the slot that follows the ring go there.
#pragma once
#include <algorithm>
#include <type_traits>

#include "tmoe.h"
#include "tmoe_device.hpp"
#include "tmoe_grouped.hpp"
#include "tmoe_grouped_scales.hpp"

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

constexpr int kRingSlots = 2;                    // the waits of the loop count on two; three and four gained nothing
constexpr int kRsrcFlags = 0x00027000;           // raw buffer, 32-bit data
constexpr int kNontemporal = 2;                  // a load's nt bit
constexpr int kPastEnd = static_cast<int>(0x80000000u);   // an offset outside every buffer

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const uint8_t* p, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p), 0, max(bytes, 0), kRsrcFlags);
}

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// SCALES (MXFP8): scales are copied to LDS, those of four slots at a time; else they are loaded byte by byte.
// DEPTH: depth of a slot; 128 bytes, or less where both operands are KS.
// PAST: what does not stay in L2 (kResults, kWeights).
enum { kResults = 1, kWeights = 2 };
template <int KIND, int WT_, int WC_, int MT_, int NT_, bool SCALES_ = false, int DEPTH_ = KIND == kKindMx8 ? 128 : 64,
          int PAST_ = kResults>
struct GTile {
  template <int P> using With = GTile<KIND, WT_, WC_, MT_, NT_, SCALES_, DEPTH_, P>;
  static constexpr int PAST = PAST_;
  static constexpr bool SCALES = SCALES_;
  static constexpr int WT = WT_, WC = WC_, MT = MT_, NT = NT_;
  static constexpr int ES = KIND == kKindMx8 ? 1 : 2;             // bytes a value
  static constexpr int DEPTH = DEPTH_;
  static constexpr int TR = 32 * MT * WT, TC = 32 * NT * WC;
  static constexpr int kSlot = (TR + TC) * DEPTH * ES;
  static constexpr int kScaleRows = SCALES ? TC + (TR + 63) / 64 * 64 : 0;
  static constexpr int kScaleBuffer = 16 * kScaleRows;            // one of two
  static constexpr int kRing = kRingSlots * kSlot;
  static constexpr int kLds = kRing + 2 * kScaleBuffer;
  static constexpr int SPW = (kScaleRows / 64 + 3) / 4;           // scale copies of a wavefront
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
template <int T, bool KS, int ES, int DEPTH>
struct Operand {
  static_assert(KS || DEPTH * ES == 128, "whole lines");
  const uint8_t* base;       // KC: first row; KS: first depth row
  int pitch;                 // bytes from row to row, at most 2^17
  int rows;                  // KC: rows that exist; KS: depth rows that exist
  int depth_bytes;           // KC: bytes of a row
  int first;                 // offset of copy 0 of this lane
  int step;                  // from copy to copy
  int at;                    // KC: this lane's byte within the slot's 128

  static constexpr int N = T * DEPTH * ES / 4096;   // copies a wavefront and slot

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
      const int n = rows - DEPTH * slot;
      return rsrc(base + static_cast<long long>(DEPTH) * slot * pitch, min(n, DEPTH) * pitch);
    } else {
      return rsrc(base + 128LL * slot, rows * pitch - 128 * slot);
    }
  }
  // offset of copy i; behind the row's end: outside
  __device__ __forceinline__ int offset(int slot, int i) const {
    if constexpr (KS) return first < 0 ? first : first + i * step;
    else return 128 * slot + at < depth_bytes ? first + i * step : kPastEnd;
  }
};

template <int KIND, bool RKS, bool CKS, class S, int OUT>
__device__ __forceinline__ void grouped_body(const GroupedArgs& a, const GroupedTile& t, uint8_t* lds) {
  constexpr bool MX = KIND == kKindMx8;
  constexpr int MT = S::MT, NT = S::NT, SUBS = MX ? 2 : S::DEPTH / 16;
  const int tid = threadIdx.x, lane = tid & 63, wv = uniform(tid >> 6);
  const int r32 = lane & 31, h = lane >> 5, wt = wv / S::WC, wc = wv % S::WC;
  const int row_pitch = (RKS ? a.out_rows : a.depth) * S::ES;
  const int col_pitch = (CKS ? a.cols : a.depth) * S::ES;

  Operand<S::TR, RKS, S::ES, S::DEPTH> R;
  Operand<S::TC, CKS, S::ES, S::DEPTH> C;
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
  int islot = 0;                                 // the slot that is copied
  auto issue = [&](int place, int i, __amdgpu_buffer_rsrc_t rr, __amdgpu_buffer_rsrc_t cr) __attribute__((always_inline)) {
    if (i < C.N)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(cr, (__attribute__((address_space(3))) void*)(ring + place * S::kSlot + S::TR * S::DEPTH * S::ES + (wv + 4 * i) * 1024),
                                               16, C.offset(islot, i), 0, 0, S::PAST & kWeights ? kNontemporal : 0);
    else
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rr, (__attribute__((address_space(3))) void*)(ring + place * S::kSlot + (wv + 4 * (i - C.N)) * 1024),
                                               16, R.offset(islot, i - C.N), 0, 0, 0);
  };
  // MXFP8 scales, columns first, then rows, in two buffers: with the first slot of every four 16 bytes a row, the last ones of
  // a row starting where they end with it (one slot at a time, 4 bytes a row, asks L2 for as many lines as
  // the codes: 535 us instead of 519 at 8192 x 8192 x 8192).
  const int nblk = MX ? a.depth / 32 : 0;
  auto issue_scales = [&]() __attribute__((always_inline)) {
    if constexpr (S::SCALES) {
      if (islot % kScaleSlots != 0) return;
      constexpr int CN = S::TC / 64, ALL = S::kScaleRows / 64;
      const int from = scales_from(islot, nblk);
#pragma unroll
      for (int i = 0; i < S::SPW; ++i) {
        const int j = min(wv + 4 * i, ALL - 1);
        const bool col = j < CN;
        const int row = 64 * (col ? j : j - CN) + lane, n = col ? min(S::TC, a.cols - t.col0) : t.nrows;
        const uint8_t* p = col ? a.cs + (t.expert * a.cols + t.col0) * nblk : a.rs + static_cast<long long>(t.row0) * nblk;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            rsrc(p + from, n * nblk - from),
            (__attribute__((address_space(3))) void*)(ring + S::kRing + islot / kScaleSlots % 2 * S::kScaleBuffer + 1024 * j),
            16, row * nblk, 0, 0, 0);
      }
    }
  };
  auto scales_at = [&](int slot, int row) __attribute__((always_inline)) {
    typedef __attribute__((address_space(3))) int lds_i;
    return *(lds_i*)(ring + S::kRing + slot / kScaleSlots % 2 * S::kScaleBuffer + 16 * row + scale_place(slot, nblk));
  };

  struct Frags {
    i4v r[MT][MX ? 2 : 1], c[NT][MX ? 2 : 1];
    int rs[MT], cs[NT];
  };
  // Row fragment m of a wavefront is the tile's (m WT + wt)-th, so that short tiles need few of every wavefront's.
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
      for (int f = 0; f < MT; ++f) tr_r[f] = k * 2 * S::TR + 64 * ((f * S::WT + wt) ^ m) + in;
    }
    if constexpr (CKS) {
#pragma unroll
      for (int f = 0; f < NT; ++f) tr_c[f] = k * 2 * S::TC + 64 * ((wc * NT + f) ^ m) + in;
    }
  }
  typedef __attribute__((address_space(3))) i4v lds_i4;
  // unaligned scales: straight from global memory, a byte a block
  auto scale_bytes = [&](const uint8_t* p, int n, int row, int slot) __attribute__((always_inline)) {
    const uint8_t* q = p + static_cast<long long>(min(row, n - 1)) * nblk;
    int w = 0;
#pragma unroll
    for (int b = 0; b < 4; ++b) w |= 4 * slot + b < nblk ? q[4 * slot + b] << (8 * b) : 0;
    return w;
  };
  auto read_piece = [&](int slot, int place, int s, int p, Frags& f) __attribute__((always_inline)) {
    lds_u8* const base = ring + place * S::kSlot;
    if (p < NT) {
      lds_u8* const at = base + S::TR * S::DEPTH * S::ES;
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
            if constexpr (S::SCALES) w = scales_at(slot, row);
            else w = scale_bytes(a.cs + (t.expert * a.cols + t.col0) * nblk, a.cols - t.col0, row, slot);
            f.cs[p] = w;
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
        const int fr = 4096 * (m * S::WT + wt);
        if constexpr (MX) {
          f.r[m][0] = *(lds_i4*)(base + fr + chunk_at[2 * s]);
          f.r[m][1] = *(lds_i4*)(base + fr + chunk_at[2 * s + 1]);
          if (s == 0) {
            const int row = 32 * (m * S::WT + wt) + r32;
            int w;
            if constexpr (S::SCALES) w = scales_at(slot, S::TC + row);
            else w = scale_bytes(a.rs + static_cast<long long>(t.row0) * nblk, t.nrows, row, slot);
            f.rs[m] = w;
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
  constexpr int MM = MT * NT, RD = MT + NT, CP = Operand<S::TR, RKS, S::ES, S::DEPTH>::N + Operand<S::TC, CKS, S::ES, S::DEPTH>::N;
  // A slot's P = SUBS * MM matrix instructions are positions 0 .. P - 1. In front of position kFree every wavefront has read all of
  // the slot: the copies that take its place start there; in front of kLanded the next slot's copies have landed and it may be
  // read. In 256 x 256 tiles (one wavefront a SIMD: nothing else hides what it waits for) the two are barriers of their own, as
  // far apart as the fragments' registers allow, and a copy goes out every kEvery positions (all at once they stand in each
  // other's way and hold up the matrix instructions behind them); those past P belong to the next round of the loop.
  constexpr int P = SUBS * MM;
  constexpr bool APART = MM == 16;
  constexpr int kFree = APART ? P - MM - (MX ? 2 : 6) : P - MM, kLanded = APART ? P - MM / 2 : kFree, kEvery = MX ? 1 : 3;
  auto position = [](int i) { return APART ? kFree + i * kEvery : kFree + i * MM / CP; };
  auto copies_below = [position](int q) {
    int n = 0;
    for (int i = 0; i < CP; ++i) n += position(i) < q;
    return n;
  };
  constexpr int kFirst = copies_below(P), kNewer = copies_below(kLanded);
  static_assert(position(CP - 1) < P + kFree, "a slot's copies have gone out when the next one's start");
  // fragments in the order in which the matrix instructions want them
  auto piece = [](int p) { return p == 0 ? 0 : p == 1 ? NT : p <= NT ? p - 1 : p; };
  if (slots > 0) {
    int place = 0, into = kRingSlots - 1;        // the place that is read, the one that is written
    __amdgpu_buffer_rsrc_t rr, cr;
    Frags f[2];
#pragma unroll
    for (int d = 0; d < kRingSlots; ++d) {
      islot = d;
      issue_scales();
      rr = R.window(d), cr = C.window(d);
#pragma unroll
      for (int i = 0; i < (d == kRingSlots - 1 ? kFirst : CP); ++i) issue(d, i, rr, cr);
    }
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(kFirst) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
#pragma unroll
    for (int p = 0; p < MT + NT; ++p) read_piece(0, 0, 0, p, f[0]);
    const int fragments = (t.nrows + 32 * S::WT - 1) / (32 * S::WT);
    for (int slot = 0; slot < slots; ++slot) {
      const int next = place + 1 == kRingSlots ? 0 : place + 1;
      int rs[MT], cs[NT];
      if constexpr (MX) {
#pragma unroll
        for (int m = 0; m < MT; ++m) rs[m] = static_cast<int>(static_cast<uint32_t>(f[0].rs[m]) >> (8 * h));   // bytes 0 and 2: this half's
#pragma unroll
        for (int n = 0; n < NT; ++n) cs[n] = static_cast<int>(static_cast<uint32_t>(f[0].cs[n]) >> (8 * h));
      }
#pragma unroll
      for (int s = 0; s < SUBS; ++s) {
        Frags &now = f[s & 1], &nxt = f[(s + 1) & 1];
        const bool last = s == SUBS - 1;
#pragma unroll
        for (int j = 0; j < MM; ++j) {
          const int q = s * MM + j;
          if (q == kFree) {
            if constexpr (APART) asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            else asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(kNewer) : "memory");
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
            islot = slot + kRingSlots;           // past the last one: zeros, which nobody reads
            into = place;
            rr = R.window(islot), cr = C.window(islot);
          }
          if (q == kLanded) {
            if constexpr (APART) {
              asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kNewer) : "memory");
              __builtin_amdgcn_s_barrier();
              asm volatile("" ::: "memory");
            }
            issue_scales();
          }
          const int from = last && APART ? MM / 2 : 0;
          const int per = (RD + MM - from - 1) / (MM - from);
#pragma unroll
          for (int p = (j - from) * per; j >= from && p < (j - from + 1) * per && p < RD; ++p)
            read_piece(last ? slot + 1 : slot, last ? next : place, last ? 0 : s + 1, piece(p), nxt);
#pragma unroll
          for (int i = 0; i < CP; ++i)
            if (position(i) % P == q) issue(into, i, rr, cr);
          __builtin_amdgcn_sched_barrier(0);
          const int m = j / NT, n = j % NT;
          if constexpr (MX) {
            // rows that a short tile does not have are left out (16-bit values: the branches cost full tiles a tenth)
            if (m >= fragments) continue;
            const i8v c8 = __builtin_shufflevector(now.c[n][0], now.c[n][1], 0, 1, 2, 3, 4, 5, 6, 7);
            const i8v r8 = __builtin_shufflevector(now.r[m][0], now.r[m][1], 0, 1, 2, 3, 4, 5, 6, 7);
            acc[m][n] = s == 0 ? mma8<0>(c8, cs[n], r8, rs[m], acc[m][n]) : mma8<1>(c8, cs[n], r8, rs[m], acc[m][n]);
          } else {
            acc[m][n] = mma<KIND>(now.c[n][0], now.r[m][0], acc[m][n]);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      place = next;
    }
  }

  // Results leave through the wavefront's own part of LDS, MB by NC fragments at a time, so that a store covers whole lines of
  // a row.
  constexpr int OS = OUT == TMOE_F32 ? 4 : 2, EPL = 16 / OS;
  constexpr int NC = 4 * 32 * (32 * NT * OS + 16) > S::kLds ? NT / 2 : NT, PITCH = 32 * NC * OS + 16;
  constexpr int MB = MT == 1 || 4 * 2 * 32 * PITCH > S::kLds ? 1 : 2;
  static_assert(4 * MB * 32 * PITCH <= S::kLds && MT % MB == 0 && NT % NC == 0, "four wavefronts' rows fit the ring");
  const int wcol = t.col0 + 32 * NT * wc;
  uint8_t* y = static_cast<uint8_t*>(a.y);
  if constexpr (RKS) y += t.expert * a.out_rows * a.cols * OS;
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // copies past the end land before the ring is used again
  __syncthreads();
  uint8_t* mine = lds + wv * MB * 32 * PITCH;
#pragma unroll
  for (int m0 = 0; m0 < MT; m0 += MB)
#pragma unroll
    for (int n0 = 0; n0 < NT; n0 += NC) {
#pragma unroll
      for (int b = 0; b < MB; ++b)
#pragma unroll
        for (int n = 0; n < NC; ++n) {
          f16v& c = acc[m0 + b][n0 + n];
          if constexpr (MM == 16) asm volatile("" : "+a"(c));   // 256 sums a lane stay where they are until their turn, or spill
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const f4 v = {c[4 * q], c[4 * q + 1], c[4 * q + 2], c[4 * q + 3]};
            uint8_t* to = mine + (32 * b + r32) * PITCH + (32 * n + 8 * q + 4 * h) * OS;
            if constexpr (OUT == TMOE_BF16) *reinterpret_cast<bf4v*>(to) = __builtin_convertvector(v, bf4v);
            else if constexpr (OUT == TMOE_F16) *reinterpret_cast<hf4v*>(to) = __builtin_convertvector(v, hf4v);
            else *reinterpret_cast<f4*>(to) = v;
          }
        }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      constexpr int LPR = 32 * NC / EPL, RPI = 64 / LPR;   // lanes a row, rows a store
      const int c = wcol + 32 * n0 + (lane % LPR) * EPL;
#pragma unroll
      for (int i = 0; i < MB * 32 / RPI; ++i) {
        const int r = RPI * i + lane / LPR, row = 32 * ((m0 + r / 32) * S::WT + wt) + r % 32;
        const i4v v = *reinterpret_cast<const i4v*>(mine + r * PITCH + (lane % LPR) * 16);
        if (row < t.nrows && c < a.cols) {
          i4v* const to = reinterpret_cast<i4v*>(y + (static_cast<long long>(t.row0 + row) * a.cols + c) * OS);
          if constexpr (S::PAST & kResults) __builtin_nontemporal_store(v, to);
          else *to = v;
        }
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
}

constexpr int kMaxTiles = (1 << 24) - 8;         // workgroups of 256 threads: a launch has fewer than 2^32 threads

// The workgroup's tile of linear or grad_x; false: none. The row tiles are implied by the offsets: expert e has ceil(rows / TR)
// of them; the rows in front of the first group and behind the last come after all experts. Every wavefront looks the tile up
// by itself: lane l holds the tiles in front of experts 8 l .. 8 l + 7. The work is dealt to the eight XCDs in contiguous runs
// (workgroups go to the XCDs in turn), within an expert in groups of four row tiles, so that an XCD's L2 holds what its tiles
// share.
template <class S>
__device__ __forceinline__ bool find_rows_tile(const GroupedArgs& a, int col_tiles, GroupedTile& t) {
  const int lane = threadIdx.x & 63, E = a.experts;
  int o[9], first[8], sum = 0;
#pragma unroll
  for (int i = 0; i < 9; ++i) o[i] = read_offset(a, min(8 * lane + i, E));
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    first[i] = sum;
    sum += (max(0, o[i + 1] - o[i]) + S::TR - 1) / S::TR;
  }
  // the lanes' prefix sums by DPP: within 16 lanes, then across them
  int up = sum;
  up += __builtin_amdgcn_update_dpp(0, up, 0x111, 0xF, 0xF, false);   // row_shr 1, 2, 4, 8
  up += __builtin_amdgcn_update_dpp(0, up, 0x112, 0xF, 0xF, false);
  up += __builtin_amdgcn_update_dpp(0, up, 0x114, 0xF, 0xF, false);
  up += __builtin_amdgcn_update_dpp(0, up, 0x118, 0xF, 0xF, false);
  up += __builtin_amdgcn_update_dpp(0, up, 0x142, 0xA, 0xF, false);   // row_bcast 15 to rows 1 and 3, 31 to rows 2 and 3
  up += __builtin_amdgcn_update_dpp(0, up, 0x143, 0xC, 0xF, false);
  const int all = __builtin_amdgcn_readlane(up, 63), front = uniform(o[0]), back = __builtin_amdgcn_readlane(o[8], 63);
  const int ft = (front + S::TR - 1) / S::TR;
  // offsets that descend may count rows twice: tiles past the launch's own are left out
  const int total = min(all + ft + (a.rows - back + S::TR - 1) / S::TR, kMaxTiles / col_tiles) * col_tiles;
  const int per = (total + 7) / 8, j = static_cast<int>(blockIdx.x / 8), w = static_cast<int>(blockIdx.x % 8) * per + j;
  if (j >= per || w >= total) return false;      // the same for the whole workgroup
  const int rt = w / col_tiles;
  t.zero = rt >= all;
  t.k0 = 0;
  t.depth = a.depth;
  if (t.zero) {
    const int behind = max(0, rt - all - ft), before = min(rt - all, ft);
    t.expert = 0;
    t.row0 = rt < all + ft ? before * S::TR : back + behind * S::TR;
    t.nrows = min(S::TR, rt < all + ft ? front - before * S::TR : a.rows - back - behind * S::TR);
    t.col0 = w % col_tiles * S::TC;
    return true;
  }
  // experts that start at or in front of this row tile; of this lane's, the last one's first tile, first row and end
  int n = 0, mine = 0, mlo = 0, mhi = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int f = first[i] + up - sum;
    n += __popcll(__ballot(f <= rt));
    mine = f <= rt ? f : mine;
    mlo = f <= rt ? o[i] : mlo;
    mhi = f <= rt ? o[i + 1] : mhi;
  }
  const int e = n - 1;                           // the last of all; the ones without rows in front of it start there too
  const int before = __builtin_amdgcn_readlane(mine, e >> 3), lo = __builtin_amdgcn_readlane(mlo, e >> 3);
  const int rows = __builtin_amdgcn_readlane(mhi, e >> 3) - lo;
  const int tiles = (rows + S::TR - 1) / S::TR;
  constexpr int G = 4;
  const int in = w - before * col_tiles;         // within the expert
  const int g = in / (G * col_tiles), at = in % (G * col_tiles), rg = min(G, tiles - g * G);
  const int r = g * G + at % rg;
  t.expert = e;
  t.row0 = lo + r * S::TR;
  t.nrows = min(S::TR, rows - r * S::TR);
  t.col0 = at / rg * S::TC;
  return true;
}

// The workgroup's tile of grad_w. Every expert has as many, but their depth is its rows: the experts with more than kPopular
// times the average come first (`popular` of them at most: that many cannot be more than E / kPopular), their tiles dealt to
// the XCDs in turn; then the others in contiguous runs, so that an XCD's L2 holds what they share. In the order of the
// experts, popular ones that come late keep their XCD busy alone (E = 96, K = N = 1024, popularity falling as 1 / rank^1.1,
// 16384 and 65536 rows: 68 and 222 us, popular ones first 64.5 and 180; 4096 rows 41 and 45).
constexpr int kPopular = 3;

template <class S>
__device__ __forceinline__ bool find_weight_tile(const GroupedArgs& a, int row_tiles, int col_tiles, int popular, GroupedTile& t) {
  const int each = row_tiles * col_tiles, total = each * a.experts, per = (total + 7) / 8;
  const int ahead = (popular * each + 7) / 8 * 8, b = static_cast<int>(blockIdx.x) - ahead;
  auto is_popular = [&](int n) { return static_cast<long long>(n) * a.experts > static_cast<long long>(kPopular) * a.rows; };
  int e, in;
  if (b < 0) {                                   // the same for the whole workgroup
    const int lane = threadIdx.x & 63, w = static_cast<int>(blockIdx.x);
    int place = w / each, left = -1, base = 0;   // the popular expert at this place: count down over 64 experts at a time
    in = w - place * each;
    unsigned long long set = 0;
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      const int x = min(64 * r + lane, a.experts);   // past the last one: no rows
      const unsigned long long has = __ballot(is_popular(read_offset(a, min(x + 1, a.experts)) - read_offset(a, x)));
      const int n = __popcll(has);
      const bool here = place >= 0 && place < n;
      set = here ? has : set;
      base = here ? 64 * r : base;
      left = here ? place : left;
      place -= n;                                // negative behind the one that holds it
    }
    if (left < 0) return false;
    const int rank = __builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(set >> 32),
                                               __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(set), 0));
    e = uniform(base + __ffsll(__ballot((set >> lane & 1) && rank == left)) - 1);
  } else {
    const int w = b % 8 * per + b / 8;
    if (w >= total) return false;
    e = w / each;
    in = w - e * each;
  }
  t.expert = e;
  t.k0 = uniform(read_offset(a, e));
  t.depth = max(0, uniform(read_offset(a, e + 1)) - t.k0);
  if (b >= 0 && popular > 0 && is_popular(t.depth)) return false;
  t.zero = false;
  constexpr int G = 4;
  const int g = in / (G * col_tiles), at = in % (G * col_tiles), rg = min(G, row_tiles - g * G);
  t.row0 = (g * G + at % rg) * S::TR;
  t.nrows = min(S::TR, a.out_rows - t.row0);
  t.col0 = at / rg * S::TC;
  return true;
}

template <class S>
constexpr int kWavesPerSimd = S::kLds > 81920 ? 1 : S::kLds > 40960 ? 2 : 4;

template <int KIND, bool CKS, class S, int OUT>
__global__ __launch_bounds__(256, kWavesPerSimd<S>) void k_grouped_rows(GroupedArgs a, int col_tiles) {
  __shared__ __align__(16) uint8_t lds[S::kLds];
  GroupedTile t;
  if (!find_rows_tile<S>(a, col_tiles, t)) return;
  if constexpr (S::MT == 4 && KIND != kKindMx8) {
    // A group's last tile, of at most half the rows, with half the fragments (E = 96, K = N = 1024, 16384 rows with uneven
    // popularity: linear 68 -> 65 us, grad_x 64.5 -> 63; MXFP8 leaves single fragments out).
    using Half = GTile<KIND, S::WT, S::WC, 2, S::NT, false, S::DEPTH, S::PAST>;
    if (t.nrows <= Half::TR) {
      grouped_body<KIND, false, CKS, Half, OUT>(a, t, lds);
      return;
    }
  }
  grouped_body<KIND, false, CKS, S, OUT>(a, t, lds);
}

template <int KIND, class S, int OUT>
__global__ __launch_bounds__(256, kWavesPerSimd<S>) void k_grouped_grad_w(GroupedArgs a, int row_tiles, int col_tiles, int popular) {
  __shared__ __align__(16) uint8_t lds[S::kLds];
  GroupedTile t;
  if (find_weight_tile<S>(a, row_tiles, col_tiles, popular, t)) grouped_body<KIND, true, true, S, OUT>(a, t, lds);
}

// Fewer tiles than this leave CUs idle that smaller tiles would use.
constexpr long long kFillsChip = 192;

// Results go past L2, where they would push out the operands (us, past it and not, E = 96, K = N = 1024, 16384 rows of uneven
// popularity: dW 66 - 79 and 95, grad_x 60 - 65 and 66 - 70, MXFP8 37 - 46 and 43 - 46, the first where operands are in the
// memory-side cache; 8192 rows: dW 50 and 75; E = 8, K = 2048, N = 4096, 16384 rows: grad_x 275 and 287, MXFP8 157 - 177 and
// 180; linear with the quantisation of its result behind it 282 and 291, E = 96, 65536 rows 197 and 193), but for dW of few rows
// an expert that fits the memory-side cache: that is little else than stores (E = 96, K = N = 1024, 1 row 36.4 and 31.4, 21
// rows 37.5 and 36.5, 43 rows 44 and 55; E = 128, K = 2560, N = 640, 419 MB, 9 rows 77 and 91).
//
// 16-bit weights that about one row tile reads go past L2, where enough workgroups have work to hide that these loads take longer
// (us, past it and not, E = 96, K = N = 1024: 16 tokens of 8 experts 32.4 and 34.8, grad_x 30.2 and 34.0; 64: 30.9 and 34.7; 2048
// 67.7 and 71.0; one token, 64 workgroups, 14.2 and 11.2; E = 1, 16 rows, K = N = 4096, 32 workgroups, 50.6 and 33.6). MXFP8 weights
// are half as large: from HBM the gain is 2 to 5 %, but where one layer's are still in the memory-side cache they lose a fifth
// (256 tokens 28.5 and 29.6, and 27.6 and 24.0).
constexpr long long kHidesLatency = 256;

template <int KIND, bool CKS, class S, int OUT>
bool launch_rows(const GroupedArgs& a, hipStream_t s) {
  const int ct = (a.cols + S::TC - 1) / S::TC;
  // every row tile but a group's last is full, the rows in front and behind are two groups more
  const long long tiles = std::min<long long>(a.rows, a.experts + 2 + a.rows / S::TR);
  const long long g = (tiles * ct + 7) / 8 * 8;
  if (g > kMaxTiles) return false;
  const dim3 grid(static_cast<unsigned>(g)), block(256);
  if constexpr (KIND != kKindMx8) {
    if (a.rows <= static_cast<long long>(S::TR) * a.experts && static_cast<long long>(std::min(a.rows, a.experts)) * ct >= kHidesLatency) {
      hipLaunchKernelGGL((k_grouped_rows<KIND, CKS, typename S::template With<kResults | kWeights>, OUT>), grid, block, 0, s, a, ct);
      return true;
    }
  }
  hipLaunchKernelGGL((k_grouped_rows<KIND, CKS, S, OUT>), grid, block, 0, s, a, ct);
  return true;
}

template <int KIND, class S, int OUT>
bool launch_grad_w(const GroupedArgs& a, hipStream_t s) {
  const int rt = (a.out_rows + S::TR - 1) / S::TR, ct = (a.cols + S::TC - 1) / S::TC;
  const int popular = a.rows >= 64LL * a.experts ? (a.experts - 1) / kPopular : 0;
  const long long each = static_cast<long long>(rt) * ct;
  const long long g = (each * popular + 7) / 8 * 8 + (each * a.experts + 7) / 8 * 8;
  if (g > kMaxTiles) return false;
  hipLaunchKernelGGL((k_grouped_grad_w<KIND, S, OUT>), dim3(static_cast<unsigned>(g)), dim3(256), 0, s, a, rt, ct, popular);
  return true;
}

// Row tiles by columns: 32 x 128 (four workgroups a CU; three where MXFP8 scales are copied to LDS too) while the weights' bytes
// count, 128 x 128 (two), 256 x 256 (one; with MXFP8 operands it spills 80 registers for fp32 results and 112 for bf16 ones).
template <int KIND, bool SCALES = false> using Few = GTile<KIND, 1, 4, 1, 1, SCALES>;
template <int KIND, bool SCALES = false> using Mid = GTile<KIND, 2, 2, 2, 2, SCALES>;
template <int KIND, bool SCALES = false> using Big = GTile<KIND, 2, 2, 4, 4, SCALES>;
template <int KIND> using Flat = GTile<KIND, 2, 2, 2, 2, false, 32>;   // 128 x 128, slots of 32 (four)

// The tile of linear and grad_x (us; bf16, E = 96, K = N = 1024 unless said; rows an expert on average):
//   up to 24 rows   32 x 128 (1: 28, 128 x 128 40; 5: 30 and 41.5; 21: 41 and 47.5; 32: 51.5 and 47; 43: 52.5 and 49)
//   up to 128       128 x 128 (85: 53, 256 x 256 56.5; 170: 72.5 and 63.5; 683: 203 and 165)
//   more            256 x 256, where there are enough of them (E = 8, K = 2048, N = 4096, 256 rows: linear, 192 tiles, 53 and
//                   128 x 128 73; grad_x, 96 tiles, 81.5 and 75.5; E = 1, 1024 rows, K = N = 4096, 72 tiles: 70 and 42.5)
// MXFP8: 32 x 128 up to 32 rows (32: 24 and 25; 43: 26 and 25). It has half the slots for the same depth, so what a tile costs
// before and behind them counts more: 256 x 256 from a depth of 4096 on (E = 1, 4096 rows, K = N = 4096: 65.5 and 76; depth 2048,
// E = 8, N = 4096, 2048 rows: 177 and 155; 1024, E = 96, 683 rows: 144 and 127).
template <int KIND, bool CKS, int OUT, bool SCALES = false>
bool launch_rows_by_size(const GroupedArgs& a, hipStream_t s) {
  const long long E = a.experts, R = a.rows;
  if (R <= (KIND == kKindMx8 ? 32 : 24) * E) return launch_rows<KIND, CKS, Few<KIND, SCALES>, OUT>(a, s);
  if constexpr (KIND != kKindMx8 || SCALES) {   // byte loads of scales leave no registers for 256 x 256
    const long long tiles = (R / 256 + (E + 1) / 2) * ((a.cols + 255) / 256);
    if (R >= 128 * E && tiles >= kFillsChip && (KIND != kKindMx8 || a.depth >= 4096)) return launch_rows<KIND, CKS, Big<KIND, SCALES>, OUT>(a, s);
  }
  return launch_rows<KIND, CKS, Mid<KIND, SCALES>, OUT>(a, s);
}

// The tile of grad_w: 128 x 128 with short slots up to 512 rows an expert (E = 96, K = N = 1024: 1 row 31, 256 x 256 44; 21: 36
// and 48; 170: 66 and 76; E = 8, 256 rows, K = 2048, N = 4096: 49 and 58), 256 x 256 beyond (683: 204 and 188; E = 8, 2048 rows,
// K = 2048, N = 4096: 280 and 221), where there are enough of them.
template <int KIND, int OUT>
bool launch_16bit(const GroupedArgs& a, int op, hipStream_t s) {
  if (op == kGroupedLinear) return launch_rows_by_size<KIND, false, OUT>(a, s);
  if (op == kGroupedGradX) return launch_rows_by_size<KIND, true, OUT>(a, s);
  const long long tiles = static_cast<long long>((a.out_rows + 255) / 256) * ((a.cols + 255) / 256) * a.experts;
  if (a.rows >= 512LL * a.experts && tiles >= kFillsChip) return launch_grad_w<KIND, Big<KIND>, OUT>(a, s);
  const long long bytes = static_cast<long long>(a.experts) * a.out_rows * a.cols * (OUT == TMOE_F32 ? 4 : 2);
  if (a.rows > 32LL * a.experts || passes_caches(bytes)) return launch_grad_w<KIND, Flat<KIND>, OUT>(a, s);
  return launch_grad_w<KIND, typename Flat<KIND>::template With<0>, OUT>(a, s);
}

}  // namespace

}  // namespace tmoe
