// k_grouped_mxfp8.hip -- the product grouped by expert for MXFP8 operands.
#include "k_grouped.hpp"

namespace tmoe {

bool launch_grouped_mxfp8(const GroupedArgs& a, bool out_f32, hipStream_t s) {
  const bool dwords = a.depth % 128 == 0 &&
                      ((reinterpret_cast<uintptr_t>(a.rs) | reinterpret_cast<uintptr_t>(a.cs)) & 3) == 0;
  if (dwords)
    return out_f32 ? launch_rows_by_size<kKindMx8, false, TMOE_F32, true>(a, s)
                   : launch_rows_by_size<kKindMx8, false, TMOE_BF16, true>(a, s);
  return out_f32 ? launch_rows_by_size<kKindMx8, false, TMOE_F32, false>(a, s)
                 : launch_rows_by_size<kKindMx8, false, TMOE_BF16, false>(a, s);
}

}  // namespace tmoe
