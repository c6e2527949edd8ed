// k_grouped_f16.hip -- the products grouped by expert for fp16 operands.
#include "k_grouped.hpp"

namespace tmoe {

bool launch_grouped_f16(const GroupedArgs& a, int op, bool out_f32, hipStream_t s) {
  return out_f32 ? launch_16bit<kKindF16, TMOE_F32>(a, op, s) : launch_16bit<kKindF16, TMOE_F16>(a, op, s);
}

}  // namespace tmoe
