// Gated scan: the forward kernel (kda_scan.h for the scheme).
//
// Measured, this kernel alone: B = 4, T = 8192, D = 2048 in bf16 with logits, 403 MB, 92 us (4.4 TB/s); one sequence of
// 131072 tokens of 1024 channels, bf16 with fp32 gates, 1074 MB, 225 us (4.8 TB/s); 32 packed sequences, 20011 tokens of
// 1000 fp32 channels, 240 MB, 63 us (3.8 TB/s); 16 packed sequences, 24001 tokens of 2048 bf16 channels with the 8-bit
// factor written, 346 MB, 89 us (3.9 TB/s).
#pragma once
#include "kda_scan.h"

namespace kda {

namespace {

// The rows of a wave with what a row gives: its decay and its input's share.  The gates are made again in the second run
// rather than kept: as they come, in 16 bits, the rows of a wave take half the registers of decays and inputs in 32,
// and twice the workgroups are on a CU while they wait for memory and for one another.  (A form for
// bf16 that keeps them at two workgroups a CU took 95 us for the first call above against 98, too little for a second
// form of the kernel.)
template <bool XF, bool GF, int CPL>
struct Rows {
    Raw<XF, CPL> x[kRows];
    Raw<GF, CPL> g[kRows];
};
template <bool LOGIT, bool MIX, bool XF, bool GF, int CPL>
__device__ __forceinline__ void step_of(const Rows<XF, GF, CPL>& rows, int i, int k, const Run& run, float& a, float& b) {
    const Gate q = gate_of<LOGIT, MIX>(raw_get(rows.g[i], k, run.shift, run.mask), run);
    const float v = raw_get(rows.x[i], k, run.shift, run.mask);
    a = q.a;
    b = MIX ? q.rest * v : v;
}

template <bool LOGIT, bool MIX, bool XF, bool GF, int CPL, bool FLAT, bool PACK, bool STREAM>
__device__ __forceinline__ void fwd_body(const ScanArgs& a, const ScanPlan& p, const Tile& t, const Marks& m,
                                         const Rows<XF, GF, CPL>& raw, int rows, int64_t r0, int64_t c, bool in,
                                         int64_t reach, Exchange<CPL>& x) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    float A[CPL], h[CPL];
    Run run = again();
#pragma unroll
    for (int k = 0; k < CPL; ++k) A[k] = 1.f, h[k] = 0.f;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        if (i >= rows) break;
        if (FLAT && (m.begins >> i & 1)) {
            state_of<CPL>(a.h0, m.seq(i) * a.D + c, in, h);
#pragma unroll
            for (int k = 0; k < CPL; ++k) A[k] = __uint_as_float(kBegins);
        }
#pragma unroll
        for (int k = 0; k < CPL; ++k) {
            float al, b;
            step_of<LOGIT, MIX>(raw, i, k, run, al, b);
            A[k] *= al;  // -0 stays -0
            h[k] = fmaf(al, h[k], b);
        }
    }
    put<CPL>(&x.A[wave][lane * CPL], A);
    put<CPL>(&x.b[wave][lane * CPL], h);
    __syncthreads();
    join_waves<false, CPL>(a, p, t, x, a.h0 && !FLAT ? a.h0 + t.chain * a.D : nullptr, reach, a.carry_out);
    __syncthreads();
    take<CPL>(&x.b[wave][lane * CPL], h);

    run = again();
    const int64_t blocks = (a.D + kCkptBlock - 1) / kCkptBlock;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        if (i >= rows) break;
        const int64_t r = r0 + i;
        if (FLAT && (m.begins >> i & 1)) state_of<CPL>(a.h0, m.seq(i) * a.D + c, in, h);
        if constexpr (PACK) {
            float u[CPL];
#pragma unroll
            for (int k = 0; k < CPL; ++k) u[k] = MIX ? h[k] - raw_get(raw.x[i], k, run.shift, run.mask) : h[k];
            bool any;
            const int s = ckpt_block<kCkptBlock / CPL, CPL>(u, in, any);
            const float inv = ckpt_inverse(s);
            if (in) {
                uint8_t* codes = a.u_out + r * a.D + c;
                if constexpr (CPL == 1) {
                    *codes = (uint8_t)ckpt_code_any(u[0], inv);
                } else {
                    static_assert(CPL == 1 || CPL == 4, "a word of codes");
                    *reinterpret_cast<uint32_t*>(codes) = ckpt_code4(u, inv, any);
                }
                if (c % kCkptBlock == 0) a.us_out[r * blocks + c / kCkptBlock] = (uint8_t)s;
            }
        }
#pragma unroll
        for (int k = 0; k < CPL; ++k) {
            float al, b;
            step_of<LOGIT, MIX>(raw, i, k, run, al, b);
            h[k] = fmaf(al, h[k], b);
        }
        if (in) store_row<XF, CPL, STREAM>(a.y, r * a.D + c, h);
        if (a.h_final && in) {
            bool ends;
            int64_t n;
            if constexpr (FLAT) ends = m.ends >> i & 1, n = m.seq(i);
            else ends = r + 1 == (t.chain + 1) * a.T_fixed, n = t.chain;
            if (ends) store_row<true, CPL>(a.h_final, n * a.D + c, h);
        }
    }
}

// Waves of a SIMD that the registers are cut to: two to a workgroup.
constexpr int fwd_waves(bool xf, bool gf) { return xf && gf ? 4 : xf || gf ? 5 : 7; }

template <bool XF, bool GF, int CPL, bool FLAT, bool PACK, bool STREAM>
__global__ __launch_bounds__(kThreads, fwd_waves(XF, GF)) void scan_fwd_kernel(ScanArgs a, ScanPlan p) {
    __shared__ Exchange<CPL> x;
    __shared__ uint32_t place;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t pl = take_place(p.counter, &place);
    const Tile t = tile_of<FLAT, false>(a, p, pl, rows_used<FLAT>(a));
    const int64_t c = t.col * 64 * CPL + lane * CPL;
    const bool in = c < a.D;
    const int64_t r0 = t.row0 + wave * kRows, last = t.rows > 0 ? t.row0 + t.rows - 1 : 0;
    const int rows = rows_of_wave(t, wave);

    Rows<XF, GF, CPL> raw;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int64_t at = (r0 + i < last ? r0 + i : last) * a.D + (in ? c : 0);
        raw.g[i] = load_raw<GF, CPL, STREAM>(a.g, at);
        raw.x[i] = load_raw<XF, CPL, STREAM>(a.x, at);
    }
    Marks m{0, 0, 0};
    int64_t reach = t.at > 0 ? t.at : -1;
    if constexpr (FLAT) {
        m = marks_of(a, r0, rows);
        // segments back to the one where the sequence of the first row begins
        reach = 0;
        if (t.rows > 0) {
            const int64_t begin = offset_of(a, seq_of(a, t.row0));
            reach = begin < t.row0 ? t.at - (begin < 0 ? 0 : begin) / kScanSeg : 0;
        }
    }
    by_form(a, [&](auto logit, auto mix) {
        fwd_body<decltype(logit)::value, decltype(mix)::value, XF, GF, CPL, FLAT, PACK, STREAM>(a, p, t, m, raw, rows, r0, c, in,
                                                                                       reach, x);
    });
}

template <bool XF, bool GF, int CPL>
void fwd(const ScanArgs& a, hipStream_t st) {
    const ScanPlan p = scan_plan(a, CPL, a.h0, a.h_final, st);
    if (a.total == 0) return;
    const dim3 grid(p.cols * p.chains * p.per_chain), block(kThreads);
    const bool stream = a.total * a.D * ((XF ? 8 : 4) + (GF ? 4 : 2)) > kStreamBytes;
    by_kind<CPL>(scan_flat(a), a.u_out, stream, [&](auto flat, auto packed, auto s) {
        hipLaunchKernelGGL((scan_fwd_kernel<XF, GF, CPL, decltype(flat)::value, decltype(packed)::value, decltype(s)::value>),
                           grid, block, 0, st, a, p);
    });
}

}  // namespace

template <bool XF>
void scan_fwd_of(const ScanArgs& a, hipStream_t st) {
    const bool wide = a.D % 4 == 0;
    if (a.g_f32) wide ? fwd<XF, true, 4>(a, st) : fwd<XF, true, 1>(a, st);
    else wide ? fwd<XF, false, 4>(a, st) : fwd<XF, false, 1>(a, st);
}

}  // namespace kda
