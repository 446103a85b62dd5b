// Group norm with an activation over channels-last rows (mathematics and layouts: include/kda_layer.h): a plain form, a
// wave for each group of a token, for every size and type.
#include "kda_device.h"
#include "kda_layer_launch.h"

namespace kda {

namespace {

template <bool F32>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
    if constexpr (F32) return static_cast<const float*>(p)[i];
    else return bf16_bits_to_float(static_cast<const uint16_t*>(p)[i]);
}
template <bool F32>
__device__ __forceinline__ void store1(void* p, int64_t i, float x) {
    if constexpr (F32) static_cast<float*>(p)[i] = x;
    else static_cast<__bf16*>(p)[i] = (__bf16)x;
}
__device__ __forceinline__ float wave_sum(float x) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) x += __shfl_xor(x, off);
    return x;
}

// act(u) and its slope.
struct Act {
    float f, slope;
};
__device__ __forceinline__ Act act_of(float u, int act) {
    if (act == 0) return {u, 1.f};
    const float s = 1.f / (1.f + expf(-u));
    return act == 2 ? Act{s, s * (1.f - s)} : Act{u * s, s * (1.f + u * (1.f - s))};
}

struct Row {
    float mean, rstd;
};
template <bool XF>
__device__ __forceinline__ Row row_of(const GroupNormArgs& a, int64_t x0, int lane) {
    float sum = 0.f, sq = 0.f;
    for (int64_t c = lane; c < a.width; c += 64) sum += load1<XF>(a.x, x0 + c);
    const float mean = wave_sum(sum) / a.width;
    for (int64_t c = lane; c < a.width; c += 64) {
        const float d = load1<XF>(a.x, x0 + c) - mean;
        sq = fmaf(d, d, sq);
    }
    return {mean, 1.f / sqrtf(wave_sum(sq) / a.width + a.eps)};
}

template <bool XF, bool YF>
__global__ __launch_bounds__(256) void groupnorm_plain_kernel(GroupNormArgs a) {
    const int64_t row = (int64_t)blockIdx.x * 4 + threadIdx.x / 64, t = row / a.groups, c0 = row % a.groups * a.width;
    const int lane = threadIdx.x % 64;
    if (t >= a.tokens) return;
    const int64_t x0 = t * a.x_stride + c0, g0 = t * a.gate_stride + c0, y0 = t * a.groups * a.width + c0;
    const Row r = row_of<XF>(a, x0, lane);
    if (!a.dy) {
        for (int64_t c = lane; c < a.width; c += 64) {
            const float n = (load1<XF>(a.x, x0 + c) - r.mean) * r.rstd;
            const float z = fmaf(n, a.weight ? a.weight[c0 + c] : 1.f, a.bias ? a.bias[c0 + c] : 0.f);
            store1<YF>(a.y, y0 + c, a.gate ? z * act_of(load1<YF>(a.gate, g0 + c), a.act).f : act_of(z, a.act).f);
        }
        return;
    }
    float s1 = 0.f, s2 = 0.f;
    auto grads = [&](int64_t c, float& n, float& dgate) {
        n = (load1<XF>(a.x, x0 + c) - r.mean) * r.rstd;
        const float w = a.weight ? a.weight[c0 + c] : 1.f, z = fmaf(n, w, a.bias ? a.bias[c0 + c] : 0.f);
        const float dy = load1<YF>(a.dy, y0 + c);
        const Act f = act_of(a.gate ? load1<YF>(a.gate, g0 + c) : z, a.act);
        dgate = dy * z * f.slope;
        return dy * (a.gate ? f.f : f.slope) * w;
    };
    float n, dgate;
    for (int64_t c = lane; c < a.width; c += 64) {
        const float dn = grads(c, n, dgate);
        s1 += dn;
        s2 = fmaf(dn, n, s2);
    }
    s1 = wave_sum(s1) / a.width;
    s2 = wave_sum(s2) / a.width;
    for (int64_t c = lane; c < a.width; c += 64) {
        const float dn = grads(c, n, dgate);
        if (a.gate) store1<YF>(a.dgate, y0 + c, dgate);
        store1<XF>(a.dx, y0 + c, r.rstd * (dn - s1 - n * s2));
    }
}

// The weights' sums: a wave for each channel's group of a column of tokens, one workgroup for the group.
template <bool XF, bool YF>
__global__ __launch_bounds__(64) void groupnorm_plain_sums_kernel(GroupNormArgs a) {
    const int64_t c0 = blockIdx.x * a.width;
    const int lane = threadIdx.x;
    for (int64_t first = 0; first < a.width; first += 64) {
        const int64_t c = first + lane;
        float dw = 0.f, db = 0.f;
        for (int64_t t = 0; t < a.tokens; ++t) {
            const Row r = row_of<XF>(a, t * a.x_stride + c0, lane);
            if (c >= a.width) continue;
            const float n = (load1<XF>(a.x, t * a.x_stride + c0 + c) - r.mean) * r.rstd;
            const float z = fmaf(n, a.weight ? a.weight[c0 + c] : 1.f, a.bias ? a.bias[c0 + c] : 0.f);
            const Act f = act_of(a.gate ? load1<YF>(a.gate, t * a.gate_stride + c0 + c) : z, a.act);
            const float dz = load1<YF>(a.dy, t * a.groups * a.width + c0 + c) * (a.gate ? f.f : f.slope);
            dw = fmaf(dz, n, dw);
            db += dz;
        }
        if (c < a.width) {
            a.dweight[c0 + c] = dw;
            a.dbias[c0 + c] = db;
        }
    }
}

template <bool XF, bool YF>
void launch(const GroupNormArgs& a, hipStream_t st) {
    if (a.tokens)
        hipLaunchKernelGGL((groupnorm_plain_kernel<XF, YF>), dim3((unsigned)groupnorm_groups(a)), dim3(256), 0, st, a);
    if (a.dweight) hipLaunchKernelGGL((groupnorm_plain_sums_kernel<XF, YF>), dim3((unsigned)a.groups), dim3(64), 0, st, a);
}

void by_type(const GroupNormArgs& a, hipStream_t st) {
    if (a.x_f32) a.y_f32 ? launch<true, true>(a, st) : launch<true, false>(a, st);
    else a.y_f32 ? launch<false, true>(a, st) : launch<false, false>(a, st);
}

}  // namespace

bool groupnorm_wide(const GroupNormArgs&) { return false; }
int64_t groupnorm_groups(const GroupNormArgs& a) { return (a.tokens * a.groups + 3) / 4; }
int64_t groupnorm_bwd_workspace_bytes(int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_groupnorm_fwd(const GroupNormArgs& a, hipStream_t st) {
    by_type(a, st);
    return hipGetLastError();
}

hipError_t launch_groupnorm_bwd(const GroupNormArgs& a, hipStream_t st) {
    by_type(a, st);
    return hipGetLastError();
}

}  // namespace kda
