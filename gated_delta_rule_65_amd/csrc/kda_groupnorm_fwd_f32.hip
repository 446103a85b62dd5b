// Forward pass of the group norm with an activation for fp32 x (kda_groupnorm.h).
#include "kda_groupnorm.h"

namespace kda {

template <>
void groupnorm_fwd_of<true, false>(const GroupNormArgs& a, hipStream_t st) { groupnorm_launch<true, false, false>(a, st); }
template <>
void groupnorm_fwd_of<true, true>(const GroupNormArgs& a, hipStream_t st) { groupnorm_launch<true, true, false>(a, st); }

}  // namespace kda
