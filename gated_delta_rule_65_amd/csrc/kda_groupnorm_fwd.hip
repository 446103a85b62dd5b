// Forward pass of the group norm with an activation (kda_groupnorm.h).
#include "kda_groupnorm.h"

namespace kda {

template <bool XF, bool YF>
void groupnorm_fwd_of(const GroupNormArgs& a, hipStream_t st) {
    gn_shape(groupnorm_wide(a), a.width, [&](auto cpl, auto p, auto iter) {
        constexpr int CPL = decltype(cpl)::value, P = decltype(p)::value, ITER = decltype(iter)::value;
        int64_t columns;
        const GnPlan plan = gn_plan(a, P, 4096, 1, columns);
        hipLaunchKernelGGL((groupnorm_kernel<XF, YF, CPL, P, ITER, false>), dim3((unsigned)columns, (unsigned)plan.blocks),
                           dim3(kGnThreads), 0, st, a, plan);
    });
}

template void groupnorm_fwd_of<true, true>(const GroupNormArgs&, hipStream_t);
template void groupnorm_fwd_of<true, false>(const GroupNormArgs&, hipStream_t);
template void groupnorm_fwd_of<false, true>(const GroupNormArgs&, hipStream_t);
template void groupnorm_fwd_of<false, false>(const GroupNormArgs&, hipStream_t);

}  // namespace kda
