// tmoe_grouped_scales.hpp -- where the MXFP8 scales of a slot lie in LDS. Plain arithmetic, without HIP, so that a host program
// can go through every depth.
//
// A slot is 128 values deep, four blocks of 32, and so four scale bytes a row. The scales of kScaleSlots slots are copied at a time, 16
// bytes a row: from block 4 * slot on, or, where the row ends before, its last 16 blocks. Depths are multiples of 128, at least 512.
#pragma once

namespace tmoe {

constexpr int kScaleSlots = 4;

// The first block that is copied with slot `slot`, a multiple of kScaleSlots, of rows of nblk blocks.
constexpr int scales_from(int slot, int nblk) { return 4 * slot < nblk - 16 ? 4 * slot : nblk - 16; }

// Byte, within a row's 16, of the scales of slot `slot`. The loop reads one slot past the last, whose value nobody uses: it gets the
// row's last four bytes (the next ones belong to another row, and behind the last row LDS ends).
constexpr int scale_place(int slot, int nblk) {
  const int place = 4 * slot - scales_from(slot / kScaleSlots * kScaleSlots, nblk);
  return place < 12 ? place : 12;
}

}  // namespace tmoe
