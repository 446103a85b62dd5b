// Gated scan over channels: the single-token step, and what a call of the scan launches beside its kernel.
#include "kda_scan.h"

namespace kda {

namespace {

// Empties the published words and the counter; sequences without tokens pass their state through.  A kernel of its own, 4 to 8
// us for the 9.6 MB of a call of 128 segments by 4 sequences by 2048 channels: the words have to be empty before the
// first workgroup looks, whatever ran before in this memory.
__global__ __launch_bounds__(256) void scan_begin_kernel(u64* words, int64_t count, uint32_t* counter, const int32_t* cu,
                                                         int64_t N, int64_t T_fixed, int64_t total, int64_t D,
                                                         const float* from, float* to) {
    const int64_t i0 = (int64_t)blockIdx.x * 256 + threadIdx.x, step = (int64_t)gridDim.x * 256;
    for (int64_t i = i0; i < count; i += step) words[i] = kEmpty;
    if (counter && i0 == 0) *counter = 0;
    if (!to) return;
    for (int64_t n = blockIdx.x; n < N; n += gridDim.x) {
        int64_t rows = T_fixed;
        if (cu) rows = cu[n] < total ? (int64_t)cu[n + 1] - cu[n] : 0;
        if (rows > 0) continue;
        for (int64_t c = threadIdx.x; c < D; c += 256) to[n * D + c] = from ? from[n * D + c] : 0.f;
    }
}

// Zeros for the rows behind the last sequence; where that is only the device knows.  Whole 16-byte words, and what lies before
// the first and behind the last of them 2 bytes at a time (rows are of 2- or 4-byte elements, buffers aligned).
struct Behind {
    void* p;
    int64_t row;  // bytes
};
__global__ __launch_bounds__(256) void scan_zero_behind_kernel(Behind a, Behind b, const int32_t* cu, int64_t N, int64_t total) {
    const int64_t used = cu[N] < 0 ? 0 : cu[N];
    if (used >= total) return;
    const Behind to = blockIdx.y ? b : a;
    char* base = static_cast<char*>(to.p);
    const int64_t from = used * to.row, end = total * to.row, up = (from + 15) / 16 * 16;
    const int64_t first = up < end ? up : end, last = first > end / 16 * 16 ? first : end / 16 * 16;
    const int64_t i0 = (int64_t)blockIdx.x * 256 + threadIdx.x, step = (int64_t)gridDim.x * 256;
    for (int64_t i = first / 16 + i0; i < last / 16; i += step) reinterpret_cast<uint4*>(base)[i] = make_uint4(0, 0, 0, 0);
    if (i0 < 8 && from + 2 * i0 < first) *reinterpret_cast<uint16_t*>(base + from + 2 * i0) = 0;
    if (i0 < 8 && last + 2 * i0 < end) *reinterpret_cast<uint16_t*>(base + last + 2 * i0) = 0;
}

// One token: an element a value, 4 to a lane.  Bound by the launch: 64 x 2048 channels take 3 us of 0.3 us of traffic, and
// the call 8 us from the host.
template <bool XF, bool GF, int CPL>
__global__ __launch_bounds__(256) void scan_step_kernel(ScanArgs a, const float* h_in, float* h_out, int64_t count) {
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * CPL;
    if (i >= count) return;
    const Raw<GF, CPL> g = load_raw<GF, CPL>(a.g, i);
    const Raw<XF, CPL> x = load_raw<XF, CPL>(a.x, i);
    const Raw<true, CPL> h = load_raw<true, CPL>(h_in, i);
    float v[CPL];
#pragma unroll
    for (int k = 0; k < CPL; ++k) {
        const float u = raw_get(x, k);
        by_form(a, [&](auto logit, auto mix) {
            const Gate q = gate_of<decltype(logit)::value, decltype(mix)::value>(raw_get(g, k), Run());
            v[k] = fmaf(q.a, raw_get(h, k), decltype(mix)::value ? q.rest * u : u);
        });
    }
    store_row<XF, CPL>(a.y, i, v);
    store_row<true, CPL>(h_out, i, v);
}

template <bool XF, bool GF, int CPL>
void step(const ScanArgs& a, const float* h_in, float* h_out, hipStream_t st) {
    const int64_t count = a.N * a.D;
    const dim3 grid((unsigned)((count + 256 * CPL - 1) / (256 * CPL)));
    hipLaunchKernelGGL((scan_step_kernel<XF, GF, CPL>), grid, dim3(256), 0, st, a, h_in, h_out, count);
}

int64_t words_of(int64_t chains, int64_t per_chain, int64_t D) {
    return chains * D * (per_chain + (per_chain + kGroup - 1) / kGroup + (per_chain + kBlock - 1) / kBlock);
}

}  // namespace

ScanPlan scan_plan(const ScanArgs& a, int cpl, const float* from, float* to, hipStream_t st) {
    ScanPlan p{};
    p.cols = (uint32_t)((a.D + 64 * cpl - 1) / (64 * cpl));
    p.chains = scan_flat(a) ? 1 : (uint32_t)a.N;
    p.per_chain = (uint32_t)(scan_segments(a) / p.chains);
    int64_t words = 0;
    if (p.per_chain > 1) {
        p.counter = static_cast<uint32_t*>(a.ws);
        p.pairs = static_cast<u64*>(a.ws) + 32;
        p.groups = p.pairs + (int64_t)p.chains * p.per_chain * a.D;
        p.states = p.groups + (int64_t)p.chains * ((p.per_chain + kGroup - 1) / kGroup) * a.D;
        words = words_of(p.chains, p.per_chain, a.D);
    }
    const bool pass = to && (a.cu || a.T_fixed == 0);
    if (words > 0 || pass) {
        int64_t groups = (words + 1023) / 1024;
        if (pass && groups < a.N) groups = a.N;
        if (groups > 2048) groups = 2048;
        hipLaunchKernelGGL(scan_begin_kernel, dim3((unsigned)groups), dim3(256), 0, st, p.pairs, words, p.counter, a.cu,
                           a.N, a.T_fixed, a.total, a.D, from, pass ? to : nullptr);
    }
    return p;
}

int64_t scan_places(const ScanArgs& a) {
    const int64_t wide = a.D % 4 == 0 ? 256 : 64;
    return (a.D + wide - 1) / wide * scan_segments(a);
}

// The most segments that N sequences of total tokens in all make, packed or of equal lengths.  Only equally long sequences of
// half a segment or more have segments of their own, so there are at most total / 32 of these and each rounds up once;
// packed rows are one chain.
static int64_t own_chains(int64_t N, int64_t total) {
    const int64_t most = total / (kScanSeg / 2) + 1;
    return N < most ? N : most;
}
int64_t scan_most_segments(int64_t N, int64_t total) { return total / kScanSeg + own_chains(N, total); }

// Groups and blocks are started anew for each chain.
int64_t scan_workspace_bytes(int64_t N, int64_t total, int64_t D) {
    if (total <= kScanSeg) return 0;
    const int64_t s = scan_most_segments(N, total), m = own_chains(N, total);
    return 256 + 8 * D * (s + s / kGroup + m + s / kBlock + m);
}

hipError_t launch_scan_fwd(const ScanArgs& a, hipStream_t st) {
    a.x_f32 ? scan_fwd_of<true>(a, st) : scan_fwd_of<false>(a, st);
    return hipGetLastError();
}

hipError_t launch_scan_bwd(const ScanArgs& a, hipStream_t st) {
    a.x_f32 ? scan_bwd_of<true>(a, st) : scan_bwd_of<false>(a, st);
    return hipGetLastError();
}

hipError_t launch_scan_zero_behind(const int32_t* cu, int64_t N, int64_t total, void* a, int64_t a_row, void* b,
                                   int64_t b_row, hipStream_t st) {
    const int64_t words = total * (a_row > b_row ? a_row : b_row) / 16, groups = words / 1024 + 1;
    hipLaunchKernelGGL(scan_zero_behind_kernel, dim3((unsigned)(groups < 512 ? groups : 512), b ? 2 : 1), dim3(256), 0, st,
                       Behind{a, a_row}, Behind{b, b_row}, cu, N, total);
    return hipGetLastError();
}

hipError_t launch_scan_step(const ScanArgs& a, const float* h_in, float* h_out, hipStream_t st) {
    by_type(a, [&](auto xf, auto gf) {
        if (a.N * a.D % 4 == 0) step<decltype(xf)::value, decltype(gf)::value, 4>(a, h_in, h_out, st);
        else step<decltype(xf)::value, decltype(gf)::value, 1>(a, h_in, h_out, st);
    });
    return hipGetLastError();
}

}  // namespace kda
