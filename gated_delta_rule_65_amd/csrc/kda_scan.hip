// Gated scan over channels: h_t = a_t h_{t-1} + w_t x_t, its gradients and its single-token step
// (mathematics and layouts: include/kda_layer.h).
#include "kda_ckpt8.h"
#include "kda_layer_launch.h"

namespace kda {

namespace {

template <bool F32>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
    if constexpr (F32) return static_cast<const float*>(p)[i];
    else return __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
}
template <bool F32>
__device__ __forceinline__ void store1(void* p, int64_t i, float v) {
    if constexpr (F32) static_cast<float*>(p)[i] = v;
    else static_cast<__bf16*>(p)[i] = (__bf16)v;
}

constexpr float kLog2e = 1.4426950408889634f;

// 1 - e^l for l in [-5, 0]: by its series where the difference would cancel.
__device__ __forceinline__ float one_minus_exp(float l, float a) {
    // l (1 + l/2 (1 + l/3 (1 + ...))) to l^8 / 8!: below 2^-24 of the result for |l| <= 0.4
    float p = fmaf(l, 1.f / 8.f, 1.f);
    p = fmaf(l * (1.f / 7.f), p, 1.f);
    p = fmaf(l * (1.f / 6.f), p, 1.f);
    p = fmaf(l * (1.f / 5.f), p, 1.f);
    p = fmaf(l * (1.f / 4.f), p, 1.f);
    p = fmaf(l * (1.f / 3.f), p, 1.f);
    p = fmaf(l * (1.f / 2.f), p, 1.f);
    return l > -0.4f ? -l * p : 1.f - a;
}

// What a gate input g gives: the decay a = e^l of the clamped log gate l, and 1 - a.
//   log gates: l = clamp(g, -5, 0).
//   logits: e^(-softplus(g)) = 1 / (1 + e^g), so a = 1 / (1 + t) and 1 - a = t a with t = e^g, without a logarithm
//     and without cancellation; l >= -5 is g <= ln(e^5 - 1).
// NaN stays NaN.
constexpr float kLogitEdge = 4.993239165f;  // ln(e^5 - 1)
struct Gate {
    float a, rest;
};
__device__ __forceinline__ Gate gate_of(float g, bool logit, bool need_rest) {
    if (logit) {
        const float t = __builtin_amdgcn_exp2f(__builtin_elementwise_minimum(g, kLogitEdge) * kLog2e);
        const float a = __builtin_amdgcn_rcpf(1.f + t);
        return {a, t * a};
    }
    const float l = __builtin_elementwise_minimum(__builtin_elementwise_maximum(g, -5.f), 0.f);
    const float a = __builtin_amdgcn_exp2f(l * kLog2e);
    return {a, need_rest ? one_minus_exp(l, a) : 0.f};
}
// The derivative of l by g: 1 inside the clamp (ends included) and 0 outside; with logits -sigmoid(g) = -(1 - a).
__device__ __forceinline__ float gate_slope(float g, float rest, bool logit) {
    if (logit) return g > kLogitEdge ? 0.f : -rest;
    return (g < -5.f || g > 0.f) ? 0.f : 1.f;
}

struct Span {
    int64_t first, end, slot;  // rows of sequence n, and the segment index of its first row (equal lengths)
};
__device__ __forceinline__ Span span_of(const ScanArgs& a, int64_t n) {
    if (!a.cu) return {n * a.T_fixed, (n + 1) * a.T_fixed, n * ((a.T_fixed + kScanSeg - 1) / kScanSeg)};
    // offsets outside [0, total] are cut there: no access leaves the buffers whatever they hold
    const int64_t lo = a.cu[n], hi = a.cu[n + 1];
    const int64_t f = lo < 0 ? 0 : lo > a.total ? a.total : lo, e = hi < f ? f : hi > a.total ? a.total : hi;
    return {f, e, 0};
}
// Index of the segment that begins at row r of a sequence, or -1 where none does.
__device__ __forceinline__ int64_t segment_at(const ScanArgs& a, const Span& s, int64_t r) {
    if (a.cu) return r % kScanSeg ? -1 : r / kScanSeg;
    return (r - s.first) % kScanSeg ? -1 : s.slot + (r - s.first) / kScanSeg;
}

// A channel of a sequence to a lane, one token after the other.
template <bool XF, bool GF>
__global__ __launch_bounds__(64) void scan_fwd_kernel(ScanArgs a) {
    const int64_t cols = (a.D + 63) / 64, n = blockIdx.x / cols;
    const int64_t c = (blockIdx.x - n * cols) * 64 + threadIdx.x;
    const bool in = c < a.D;
    const int64_t cc = in ? c : a.D - 1;
    const Span s = span_of(a, n);
    float h = a.h0 ? a.h0[n * a.D + cc] : 0.f;
    const int64_t blocks = (a.D + kCkptBlock - 1) / kCkptBlock;
    for (int64_t r = s.first; r < s.end; ++r) {
        const int64_t i = r * a.D + cc;
        if (a.carry_out) {
            const int64_t seg = segment_at(a, s, r);
            if (seg >= 0 && in) a.carry_out[seg * a.D + c] = h;
        }
        const Gate q = gate_of(load1<GF>(a.g, i), a.logit, a.complement);
        const float x = load1<XF>(a.x, i);
        if (a.u_out) {
            const float u = a.complement ? h - x : h;
            uint32_t top = in ? finite_abs_bits(u) : 0u;
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) {
                const uint32_t o = (uint32_t)__shfl_xor((int)top, off);
                top = top > o ? top : o;
            }
            const int sc = ckpt_scale(top);
            if (in) {
                a.u_out[i] = (uint8_t)ckpt_code2(u, 0.f, ckpt_inverse(sc));
                if ((c & 31) == 0) a.us_out[r * blocks + c / kCkptBlock] = (uint8_t)sc;
            }
        }
        h = fmaf(q.a, h, a.complement ? q.rest * x : x);
        if (in) store1<XF>(a.y, i, h);
    }
    if (in && a.h_final) a.h_final[n * a.D + c] = h;
}

template <bool XF, bool GF>
__global__ __launch_bounds__(64) void scan_bwd_kernel(ScanArgs a) {
    const int64_t cols = (a.D + 63) / 64, n = blockIdx.x / cols;
    const int64_t c = (blockIdx.x - n * cols) * 64 + threadIdx.x;
    if (c >= a.D) return;
    const Span s = span_of(a, n);
    float e = a.dh_final ? a.dh_final[n * a.D + c] : 0.f;
    const int64_t blocks = (a.D + kCkptBlock - 1) / kCkptBlock;
    int64_t end = s.end;
    while (end > s.first) {
        // the segment's rows, and the states before them from the carry
        int64_t from = a.cu ? (end - 1) / kScanSeg * kScanSeg
                            : s.first + (end - 1 - s.first) / kScanSeg * kScanSeg;
        const bool head = from <= s.first;
        if (head) from = s.first;
        float before[kScanSeg];
        if (!a.u) {
            float h = head ? (a.h0 ? a.h0[n * a.D + c] : 0.f) : a.carry[segment_at(a, s, from) * a.D + c];
            for (int64_t r = from; r < end; ++r) {
                before[r - from] = h;
                const Gate q = gate_of(load1<GF>(a.g, r * a.D + c), a.logit, a.complement);
                const float x = load1<XF>(a.x, r * a.D + c);
                h = fmaf(q.a, h, a.complement ? q.rest * x : x);
            }
        }
        for (int64_t r = end - 1; r >= from; --r) {
            const int64_t i = r * a.D + c;
            const float g = load1<GF>(a.g, i);
            const Gate q = gate_of(g, a.logit, true);
            float u;
            if (a.u) u = ckpt_value<0>(a.u[i], a.us[r * blocks + c / kCkptBlock]);
            else u = before[r - from] - (a.complement ? load1<XF>(a.x, i) : 0.f);
            const float dh = load1<XF>(a.dy, i) + e;
            e = q.a * dh;
            store1<XF>(a.dx, i, a.complement ? q.rest * dh : dh);
            store1<GF>(a.dg, i, u * e * gate_slope(g, q.rest, a.logit));
        }
        end = from;
    }
    if (a.dh0) a.dh0[n * a.D + c] = e;
}

template <bool XF, bool GF>
__global__ __launch_bounds__(256) void scan_step_kernel(ScanArgs a, const float* h_in, float* h_out, int64_t count) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= count) return;
    const Gate q = gate_of(load1<GF>(a.g, i), a.logit, a.complement);
    const float x = load1<XF>(a.x, i);
    const float h = fmaf(q.a, h_in[i], a.complement ? q.rest * x : x);
    store1<XF>(a.y, i, h);
    h_out[i] = h;
}

}  // namespace

int64_t scan_workspace_bytes(int64_t, int64_t, int64_t) { return 0; }

#define KDA_SCAN_TYPES(KERNEL, GRID, BLOCK, ...)                                                            \
    do {                                                                                                    \
        if (a.x_f32 && a.g_f32) hipLaunchKernelGGL((KERNEL<true, true>), GRID, BLOCK, 0, st, __VA_ARGS__);  \
        else if (a.x_f32) hipLaunchKernelGGL((KERNEL<true, false>), GRID, BLOCK, 0, st, __VA_ARGS__);       \
        else if (a.g_f32) hipLaunchKernelGGL((KERNEL<false, true>), GRID, BLOCK, 0, st, __VA_ARGS__);       \
        else hipLaunchKernelGGL((KERNEL<false, false>), GRID, BLOCK, 0, st, __VA_ARGS__);                   \
    } while (0)

hipError_t launch_scan_fwd(const ScanArgs& a, hipStream_t st) {
    const dim3 grid((unsigned)((a.D + 63) / 64 * a.N));
    KDA_SCAN_TYPES(scan_fwd_kernel, grid, dim3(64), a);
    return hipGetLastError();
}

hipError_t launch_scan_bwd(const ScanArgs& a, hipStream_t st) {
    const dim3 grid((unsigned)((a.D + 63) / 64 * a.N));
    KDA_SCAN_TYPES(scan_bwd_kernel, grid, dim3(64), a);
    return hipGetLastError();
}

hipError_t launch_scan_step(const ScanArgs& a, const float* h_in, float* h_out, hipStream_t st) {
    const int64_t count = a.N * a.D;
    const dim3 grid((unsigned)((count + 255) / 256));
    KDA_SCAN_TYPES(scan_step_kernel, grid, dim3(256), a, h_in, h_out, count);
    return hipGetLastError();
}

}  // namespace kda
