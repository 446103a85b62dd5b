// Backward pass of the group norm with an activation (kda_groupnorm.h).
#include "kda_groupnorm.h"

namespace kda {

namespace {

// The sums over the blocks of tokens, 64 columns (of both weights' gradients) a workgroup: 16 rows of threads take every 16th
// block each, and are added up in their order.
__global__ __launch_bounds__(1024) void groupnorm_sums_kernel(const float* part, int64_t blocks, int64_t C, float* dweight,
                                                              float* dbias) {
    __shared__ float rows[16][64];
    const int64_t c = (int64_t)blockIdx.x * 64 + threadIdx.x % 64;
    const int r = threadIdx.x / 64;
    float sum = 0.f;
    if (c < 2 * C)
        for (int64_t i = r; i < blocks; i += 16) sum += part[i * 2 * C + c];
    rows[r][threadIdx.x % 64] = sum;
    __syncthreads();
    if (r || c >= 2 * C) return;
#pragma unroll
    for (int i = 1; i < 16; ++i) sum += rows[i][threadIdx.x];
    (c < C ? dweight : dbias - C)[c] = sum;
}

}  // namespace

void groupnorm_sums(const GroupNormArgs& a, int64_t blocks, hipStream_t st) {
    const int64_t C = a.groups * a.width;
    hipLaunchKernelGGL(groupnorm_sums_kernel, dim3((unsigned)((2 * C + 63) / 64)), dim3(1024), 0, st,
                       static_cast<const float*>(a.ws), blocks, C, a.dweight, a.dbias);
}

template <bool XF, bool YF>
void groupnorm_bwd_of(const GroupNormArgs& a, hipStream_t st) {
    gn_shape(groupnorm_wide(a), a.width, [&](auto cpl, auto p, auto iter) {
        constexpr int CPL = decltype(cpl)::value, P = decltype(p)::value, ITER = decltype(iter)::value;
        int64_t columns;
        const GnPlan plan = gn_plan(a, P, kGnBlocks, kGnBlockTokens, columns);
        hipLaunchKernelGGL((groupnorm_kernel<XF, YF, CPL, P, ITER, true>), dim3((unsigned)columns, (unsigned)plan.blocks),
                           dim3(kGnThreads), 0, st, a, plan);
        if (a.dweight) groupnorm_sums(a, plan.blocks, st);
    });
}

template void groupnorm_bwd_of<true, true>(const GroupNormArgs&, hipStream_t);
template void groupnorm_bwd_of<true, false>(const GroupNormArgs&, hipStream_t);
template void groupnorm_bwd_of<false, true>(const GroupNormArgs&, hipStream_t);
template void groupnorm_bwd_of<false, false>(const GroupNormArgs&, hipStream_t);

}  // namespace kda
