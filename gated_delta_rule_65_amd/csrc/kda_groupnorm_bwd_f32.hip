// Backward pass of the group norm with an activation for fp32 x (kda_groupnorm.h).
#include "kda_groupnorm.h"

namespace kda {

template <>
void groupnorm_bwd_of<true, false>(const GroupNormArgs& a, hipStream_t st) { groupnorm_launch<true, false, true>(a, st); }
template <>
void groupnorm_bwd_of<true, true>(const GroupNormArgs& a, hipStream_t st) { groupnorm_launch<true, true, true>(a, st); }

}  // namespace kda
