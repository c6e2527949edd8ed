// Every depth that copies MXFP8 scales to LDS and every slot whose scales the kernel's loop reads: the four bytes lie within the row's 16,
// and up to the last slot they are that slot's blocks.
#include <cstdio>

#include "tmoe_grouped_scales.hpp"

int main() {
  using namespace tmoe;
  for (int depth = 512; depth <= 65536; depth += 128) {
    const int nblk = depth / 32, slots = depth / 128;
    for (int slot = 0; slot <= slots; ++slot) {  // in the last slot the loop reads one ahead
      const int from = scales_from(slot / kScaleSlots * kScaleSlots, nblk), place = scale_place(slot, nblk);
      if (place < 0 || place + 4 > 16) {
        std::printf("depth %d slot %d of %d: bytes %d .. %d of a row's 16\n", depth, slot, slots, place, place + 3);
        return 1;
      }
      if (slot < slots && (from < 0 || from + 16 > nblk || from + place != 4 * slot)) {
        std::printf("depth %d slot %d: block %d, expected %d\n", depth, slot, from + place, 4 * slot);
        return 1;
      }
    }
  }
  std::puts("PASSED");
  return 0;
}
