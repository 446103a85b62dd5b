// Group norm with an activation over channels-last rows (mathematics and layouts: include/kda_layer.h): rows that are too wide
// for registers, and which kernel a call takes.
#include "kda_groupnorm.h"

namespace kda {

namespace {

// The sums over the blocks of tokens, 32 columns (of both weights' gradients) a workgroup, so that a row of threads reads a line:
// 32 rows take every 32nd block each, and are added up in their order.
__global__ __launch_bounds__(1024) void groupnorm_sums_kernel(const float* part, int64_t blocks, int64_t C, float* dweight,
                                                              float* dbias) {
    __shared__ float rows[32][33];
    const int64_t c = (int64_t)blockIdx.x * 32 + threadIdx.x % 32;
    const int r = threadIdx.x / 32;
    float sum = 0.f;
    if (c < 2 * C) {
        constexpr int AHEAD = 8;
        for (int64_t i = r; i < blocks; i += 32 * AHEAD) {
            float v[AHEAD];
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) v[k] = i + 32 * k < blocks ? part[(i + 32 * k) * 2 * C + c] : 0.f;
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) sum += v[k];
        }
    }
    rows[r][threadIdx.x % 32] = sum;
    __syncthreads();
    if (r || c >= 2 * C) return;
#pragma unroll
    for (int i = 1; i < 32; ++i) sum += rows[i][threadIdx.x];
    (c < C ? dweight : dbias - C)[c] = sum;
}

__device__ __forceinline__ float block_sum(float x, float* lds) {
    x = lanes_sum<64>(x);
    __syncthreads();
    if (threadIdx.x % 64 == 0) lds[threadIdx.x / 64] = x;
    __syncthreads();
    return lds[0] + lds[1] + lds[2] + lds[3];
}

template <bool XF>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
    float x[1];
    gn_values<1, XF>(gn_load<1, XF>(p, i), x);
    return x[0];
}

__device__ __forceinline__ void act_of(float v, int act, float& f, float& slope) {
    f = v;
    slope = 1.f;
    if (act) gn_act<true, true>(v, act == 2, f, slope);
}

// A workgroup for a group of a token, an element a thread at a time; the passes after the first find the row in the caches.  4096 tokens
// of one group of 4096 in bf16, gated: 44 us forward and 93, 38 and 5 backward; its bytes take 16 and 27.
// stats: mean and 1/deviation of every row, for the weights' sums.
template <bool XF, bool YF>
__global__ __launch_bounds__(kGnThreads) void groupnorm_rows_kernel(GroupNormArgs a, float* stats) {
    __shared__ float lds[4];
    const int64_t row = blockIdx.x, t = row / a.groups, c0 = row % a.groups * a.width, C = a.groups * a.width;
    const int64_t x0 = t * a.x_stride + c0, g0 = t * a.gate_stride + c0, y0 = t * C + c0;
    const float mean_of = 1.f / a.width;
    float sum = 0.f, squares = 0.f;
    for (int64_t c = threadIdx.x; c < a.width; c += kGnThreads) sum += load1<XF>(a.x, x0 + c);
    const float mean = block_sum(sum, lds) * mean_of;
    for (int64_t c = threadIdx.x; c < a.width; c += kGnThreads) {
        const float d = load1<XF>(a.x, x0 + c) - mean;
        squares = fmaf(d, d, squares);
    }
    const float rstd = 1.f / sqrtf(fmaf(block_sum(squares, lds), mean_of, a.eps));
    if (stats && threadIdx.x == 0) {
        stats[2 * row] = mean;
        stats[2 * row + 1] = rstd;
    }
    auto terms = [&](int64_t c, float& n, float& z, float& w, float& f, float& slope) {
        n = (load1<XF>(a.x, x0 + c) - mean) * rstd;
        w = a.weight ? a.weight[c0 + c] : 1.f;
        z = fmaf(n, w, a.bias ? a.bias[c0 + c] : 0.f);
        const float v = a.gate ? load1<YF>(a.gate, g0 + c) : z;
        act_of(v, a.act, f, slope);
    };
    float n, z, w, f, slope;
    if (!a.dy) {
        for (int64_t c = threadIdx.x; c < a.width; c += kGnThreads) {
            terms(c, n, z, w, f, slope);
            const float y = a.gate ? z * f : f;
            gn_store<1, YF>(a.y, y0 + c, &y);
        }
        return;
    }
    float s1 = 0.f, s2 = 0.f;
    for (int64_t c = threadIdx.x; c < a.width; c += kGnThreads) {
        terms(c, n, z, w, f, slope);
        const float dn = load1<YF>(a.dy, y0 + c) * (a.gate ? f : slope) * w;
        s1 += dn;
        s2 = fmaf(dn, n, s2);
    }
    s1 = block_sum(s1, lds) * mean_of;
    s2 = block_sum(s2, lds) * mean_of;
    for (int64_t c = threadIdx.x; c < a.width; c += kGnThreads) {
        terms(c, n, z, w, f, slope);
        const float dy = load1<YF>(a.dy, y0 + c), dx = rstd * (dy * (a.gate ? f : slope) * w - fmaf(n, s2, s1));
        const float dgate = dy * z * slope;
        if (a.gate) gn_store<1, YF>(a.dgate, y0 + c, &dgate);
        gn_store<1, XF>(a.dx, y0 + c, &dx);
    }
}

// The weights' sums over blocks of tokens, a thread a channel.
template <bool XF, bool YF>
__global__ __launch_bounds__(kGnThreads) void groupnorm_columns_kernel(GroupNormArgs a, const float* stats, int64_t block) {
    const int64_t c = (int64_t)blockIdx.x * kGnThreads + threadIdx.x, C = a.groups * a.width;
    if (c >= C) return;
    const float w = a.weight ? a.weight[c] : 1.f, b = a.bias ? a.bias[c] : 0.f;
    const int64_t first = blockIdx.y * block, end = first + block < a.tokens ? first + block : a.tokens;
    float dw = 0.f, db = 0.f;
    for (int64_t t = first; t < end; ++t) {
        const float* s = stats + 2 * (t * a.groups + c / a.width);
        const float n = (load1<XF>(a.x, t * a.x_stride + c) - s[0]) * s[1], z = fmaf(n, w, b);
        float f, slope;
        act_of(a.gate ? load1<YF>(a.gate, t * a.gate_stride + c) : z, a.act, f, slope);
        const float dz = load1<YF>(a.dy, t * C + c) * (a.gate ? f : slope);
        dw = fmaf(dz, n, dw);
        db += dz;
    }
    float* out = static_cast<float*>(a.ws) + blockIdx.y * 2 * C;
    out[c] = dw;
    out[C + c] = db;
}

int64_t token_blocks(int64_t tokens) {
    const int64_t most = (tokens + kGnBlockTokens - 1) / kGnBlockTokens;
    return most < kGnBlocks ? most : kGnBlocks;
}

template <bool XF, bool YF>
void wide_rows(const GroupNormArgs& a, hipStream_t st) {
    const int64_t C = a.groups * a.width, blocks = token_blocks(a.tokens);
    float* stats = a.dweight ? static_cast<float*>(a.ws) + blocks * 2 * C : nullptr;
    hipLaunchKernelGGL((groupnorm_rows_kernel<XF, YF>), dim3((unsigned)(a.tokens * a.groups)), dim3(kGnThreads), 0, st, a, stats);
    if (!a.dweight) return;
    hipLaunchKernelGGL((groupnorm_columns_kernel<XF, YF>), dim3((unsigned)((C + kGnThreads - 1) / kGnThreads), (unsigned)blocks),
                       dim3(kGnThreads), 0, st, a, stats, (a.tokens + blocks - 1) / blocks);
    groupnorm_sums(a, blocks, st);
}

template <typename F>
void by_type(const GroupNormArgs& a, F&& f) {
    if (a.x_f32) a.y_f32 ? f(std::true_type(), std::true_type()) : f(std::true_type(), std::false_type());
    else a.y_f32 ? f(std::false_type(), std::true_type()) : f(std::false_type(), std::false_type());
}

}  // namespace

void groupnorm_sums(const GroupNormArgs& a, int64_t blocks, hipStream_t st) {
    const int64_t C = a.groups * a.width;
    hipLaunchKernelGGL(groupnorm_sums_kernel, dim3((unsigned)((2 * C + 31) / 32)), dim3(1024), 0, st,
                       static_cast<const float*>(a.ws), blocks, C, a.dweight, a.dbias);
}

bool groupnorm_wide(const GroupNormArgs& a) {
    uintptr_t starts = 0;
    for (const void* p : {a.x, a.gate, a.dy, static_cast<const void*>(a.weight), static_cast<const void*>(a.bias),
                          static_cast<const void*>(a.y), static_cast<const void*>(a.dx), static_cast<const void*>(a.dgate)})
        starts |= reinterpret_cast<uintptr_t>(p);
    return a.width % 8 == 0 && a.x_stride % 8 == 0 && a.gate_stride % 8 == 0 && starts % 16 == 0;
}

int64_t groupnorm_groups(const GroupNormArgs& a) {
    if (!gn_in_registers(a)) return a.tokens * a.groups;
    return 8192 + a.groups;
}

int64_t groupnorm_bwd_workspace_bytes(int64_t tokens, int64_t groups, int64_t width) {
    const int64_t stats = width > 1024 ? 2 * tokens * groups : 0;
    return 4 * (token_blocks(tokens) * 2 * groups * width + stats);
}

hipError_t launch_groupnorm_fwd(const GroupNormArgs& a, hipStream_t st) {
    by_type(a, [&](auto xf, auto yf) {
        constexpr bool XF = decltype(xf)::value, YF = decltype(yf)::value;
        gn_in_registers(a) ? groupnorm_fwd_of<XF, YF>(a, st) : wide_rows<XF, YF>(a, st);
    });
    return hipGetLastError();
}

hipError_t launch_groupnorm_bwd(const GroupNormArgs& a, hipStream_t st) {
    if (a.tokens == 0) {  // sums of nothing
        groupnorm_sums(a, 0, st);
        return hipGetLastError();
    }
    by_type(a, [&](auto xf, auto yf) {
        constexpr bool XF = decltype(xf)::value, YF = decltype(yf)::value;
        gn_in_registers(a) ? groupnorm_bwd_of<XF, YF>(a, st) : wide_rows<XF, YF>(a, st);
    });
    return hipGetLastError();
}

}  // namespace kda
