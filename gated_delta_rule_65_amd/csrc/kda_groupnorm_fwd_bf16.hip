// Forward pass of the group norm with an activation for bf16 x (kda_groupnorm.h).
#include "kda_groupnorm.h"

namespace kda {

template <>
void groupnorm_fwd_of<false, false>(const GroupNormArgs& a, hipStream_t st) { groupnorm_launch<false, false, false>(a, st); }
template <>
void groupnorm_fwd_of<false, true>(const GroupNormArgs& a, hipStream_t st) { groupnorm_launch<false, true, false>(a, st); }

}  // namespace kda
