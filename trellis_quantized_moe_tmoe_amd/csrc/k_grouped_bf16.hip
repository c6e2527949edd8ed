// k_grouped_bf16.hip -- the products grouped by expert for bf16 operands.
#include "k_grouped.hpp"

namespace tmoe {

bool launch_grouped_bf16(const GroupedArgs& a, int op, bool out_f32, hipStream_t s) {
  return out_f32 ? launch_16bit<kKindBf16, TMOE_F32>(a, op, s) : launch_16bit<kKindBf16, TMOE_BF16>(a, op, s);
}

}  // namespace tmoe
