// k_grouped_mxfp8.hip -- the product grouped by expert for MXFP8 operands.
#include "k_grouped.hpp"

namespace tmoe {

bool launch_grouped_mxfp8(const GroupedArgs& a, bool out_f32, hipStream_t s) {
  // scales are copied in rows of 16 bytes from 4-byte aligned places
  const bool copies = a.depth % 128 == 0 && a.depth >= 512 &&
                      ((reinterpret_cast<uintptr_t>(a.rs) | reinterpret_cast<uintptr_t>(a.cs)) & 3) == 0;
  if (copies)
    return out_f32 ? launch_rows_by_size<kKindMx8, false, TMOE_F32, true>(a, s)
                   : launch_rows_by_size<kKindMx8, false, TMOE_BF16, true>(a, s);
  return out_f32 ? launch_rows_by_size<kKindMx8, false, TMOE_F32>(a, s)
                 : launch_rows_by_size<kKindMx8, false, TMOE_BF16>(a, s);
}

}  // namespace tmoe
