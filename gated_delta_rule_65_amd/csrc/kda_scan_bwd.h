// Gated scan: the backward kernel, the same scan with time reversed (kda_scan.h for the scheme).
//
// With e_t = a_t (dy_t + e_{t+1}), the gradient of the state behind token t being dh_t = dy_t + e_{t+1}: dx_t = w_t dh_t,
// dl_t = e_t u_t with u_t = h_{t-1} (less x_t with complement, where 1 - a_t carries part of the gradient), dh0 = e_1.
//
// What bounds it: from the carry the vector units, busy 78% of the time (the gates are made four times: for the states' pairs,
// the states, the reversed pairs and the results); from the 8-bit factor, which needs two, they are busy 49% (log gates) and
// memory and the waits weigh more.  Then the registers of two workgroups a CU (half of the factors u lie in LDS for that;
// forms with fp32 rows from the carry still spill 20 to 88 bytes a lane).  Measured: B = 4, T = 8192, D = 2048 in
// bf16 from the carry, 671 MB, 158 us (4.3 TB/s); 24001 packed tokens of 2048 bf16 channels from the 8-bit factor,
// 444 MB, 100 us (4.4 TB/s).  Both passes and what goes before them: 256 us and 199 us.
#pragma once
#include "kda_scan.h"

namespace kda {

namespace {

// PACKED: the factor u of the gate's gradient comes from its 8-bit codes; else the states of the segment are made again
// from the carry and x.
template <bool XF, bool GF, int CPL, bool PACKED>
struct BackRows {
    Raw<GF, CPL> g[kRows];
    Raw<XF, CPL> dy[kRows], x[PACKED ? 1 : kRows];
    uint32_t code[PACKED ? kRows : 1][(CPL + 3) / 4];
    uint32_t scale[PACKED ? kRows / 4 : 1];  // a byte a row
    __device__ __forceinline__ int scale_of(int i) const { return scale[i / 4] >> (i % 4 * 8) & 0xff; }
};

template <bool LOGIT, bool MIX, bool XF, bool GF, int CPL, bool FLAT, bool PACKED, bool STREAM>
__device__ __forceinline__ void bwd_body(const ScanArgs& a, const ScanPlan& p, const Tile& t, const Marks& m,
                                         const BackRows<XF, GF, CPL, PACKED>& raw, int rows, int64_t r0, int64_t c,
                                         bool in, int64_t reach, Exchange<CPL>& x, Kept<CPL, !PACKED>& kept) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    float A[CPL], s[CPL];
    float u[PACKED ? 1 : kRows - kKept][CPL];
    if constexpr (!PACKED) {
        // the states again: the waves' pairs from x, joined from the carry
        Run run = again();
#pragma unroll
        for (int k = 0; k < CPL; ++k) A[k] = 1.f, s[k] = 0.f;
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            if (i >= rows) break;
            if (FLAT && (m.begins >> i & 1)) {
                state_of<CPL>(a.h0, m.seq(i) * a.D + c, in, s);
#pragma unroll
                for (int k = 0; k < CPL; ++k) A[k] = __uint_as_float(kBegins);
            }
#pragma unroll
            for (int k = 0; k < CPL; ++k) {
                const Gate q = gate_of<LOGIT, MIX>(raw_get(raw.g[i], k, run.shift, run.mask), run);
                const float v = raw_get(raw.x[i], k, run.shift, run.mask);
                A[k] *= q.a;
                s[k] = fmaf(q.a, s[k], MIX ? q.rest * v : v);
            }
        }
        put<CPL>(&x.A[wave][lane * CPL], A);
        put<CPL>(&x.b[wave][lane * CPL], s);
        __syncthreads();
        for (int ch = threadIdx.x; ch < 64 * CPL; ch += kThreads) {
            const int64_t cf = t.col * 64 * CPL + ch;
            if (cf >= a.D) continue;
            float h;
            if (!FLAT && t.id == t.chain * p.per_chain) h = a.h0 ? a.h0[t.chain * a.D + cf] : 0.f;
            else h = a.carry[t.id * a.D + cf];  // not used where the segment's first row begins a sequence
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                const Pair q = {x.A[w][ch], x.b[w][ch]};
                x.b[w][ch] = h;
                h = apply(q, h);
            }
        }
        __syncthreads();
        take<CPL>(&x.b[wave][lane * CPL], s);
        __syncthreads();
        run = again();
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            if (FLAT && (m.begins >> i & 1)) state_of<CPL>(a.h0, m.seq(i) * a.D + c, in, s);
            float f[CPL];
#pragma unroll
            for (int k = 0; k < CPL; ++k) {
                const Gate q = gate_of<LOGIT, MIX>(raw_get(raw.g[i], k, run.shift, run.mask), run);
                const float v = raw_get(raw.x[i], k, run.shift, run.mask);
                f[k] = MIX ? s[k] - v : s[k];
                s[k] = fmaf(q.a, s[k], MIX ? q.rest * v : v);
            }
            if (i < kKept) {
                put<CPL>(&kept.rows[i < kKept ? i : 0][wave][lane * CPL], f);
            } else {
#pragma unroll
                for (int k = 0; k < CPL; ++k) u[i < kKept ? 0 : i - kKept][k] = f[k];
            }
        }
    }
    // the reversed scan
    const Run back = again();
#pragma unroll
    for (int k = 0; k < CPL; ++k) A[k] = 1.f, s[k] = 0.f;
#pragma unroll
    for (int i = kRows - 1; i >= 0; --i) {
        if (i >= rows) continue;
        if (FLAT && (m.ends >> i & 1)) {
            state_of<CPL>(a.dh_final, m.seq(i) * a.D + c, in, s);
#pragma unroll
            for (int k = 0; k < CPL; ++k) A[k] = __uint_as_float(kBegins);
        }
#pragma unroll
        for (int k = 0; k < CPL; ++k) {
            const float al = gate_of<LOGIT, false>(raw_get(raw.g[i], k, back.shift, back.mask), back).a;
            A[k] *= al;
            s[k] = al * (raw_get(raw.dy[i], k, back.shift, back.mask) + s[k]);
        }
    }
    put<CPL>(&x.A[wave][lane * CPL], A);
    put<CPL>(&x.b[wave][lane * CPL], s);
    __syncthreads();
    join_waves<true, CPL>(a, p, t, x, a.dh_final && !FLAT ? a.dh_final + t.chain * a.D : nullptr, reach, nullptr);
    __syncthreads();
    take<CPL>(&x.b[wave][lane * CPL], s);
    const Run run = again();
#pragma unroll
    for (int i = kRows - 1; i >= 0; --i) {
        if (i >= rows) continue;
        const int64_t r = r0 + i;
        if (FLAT && (m.ends >> i & 1)) state_of<CPL>(a.dh_final, m.seq(i) * a.D + c, in, s);
        float dx[CPL], dg[CPL], f[(CPL + 3) / 4 * 4];
        if constexpr (PACKED) {
            const float unit = ckpt_unit(raw.scale_of(i));
#pragma unroll
            for (int k = 0; k < CPL; k += 4) ckpt_value4(raw.code[i][k / 4], unit, f + k);
        } else if (i < kKept) {
            take<CPL>(&kept.rows[i < kKept ? i : 0][wave][lane * CPL], f);
        } else {
#pragma unroll
            for (int k = 0; k < CPL; ++k) f[k] = u[i < kKept ? 0 : i - kKept][k];
        }
#pragma unroll
        for (int k = 0; k < CPL; ++k) {
            const float g = raw_get(raw.g[i], k, run.shift, run.mask);
            const Gate q = gate_of<LOGIT, MIX>(g, run);
            const float dh = raw_get(raw.dy[i], k, run.shift, run.mask) + s[k];
            s[k] = q.a * dh;
            dx[k] = MIX ? q.rest * dh : dh;
            dg[k] = f[k] * s[k] * gate_slope<LOGIT>(g, q.rest);
        }
        if (in) {
            store_row<XF, CPL, STREAM>(a.dx, r * a.D + c, dx);
            store_row<GF, CPL, STREAM>(a.dg, r * a.D + c, dg);
            if (a.dh0) {
                bool begins;
                int64_t n;
                if constexpr (FLAT) begins = m.begins >> i & 1, n = m.seq(i);
                else begins = r == t.chain * a.T_fixed, n = t.chain;
                if (begins) store_row<true, CPL>(a.dh0, n * a.D + c, s);
            }
        }
    }
}

// Waves of a SIMD that the registers are cut to: two to a workgroup.
constexpr int bwd_waves(bool xf, bool gf, bool packed) { return packed && !xf && !gf ? 5 : 4; }

template <bool XF, bool GF, int CPL, bool FLAT, bool PACKED, bool STREAM>
__global__ __launch_bounds__(kThreads, bwd_waves(XF, GF, PACKED)) void scan_bwd_kernel(ScanArgs a, ScanPlan p) {
    __shared__ Exchange<CPL> x;
    __shared__ Kept<CPL, !PACKED> kept;
    __shared__ uint32_t place;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t pl = take_place(p.counter, &place);
    const int64_t total = rows_used<FLAT>(a);
    const Tile t = tile_of<FLAT, true>(a, p, pl, total);
    const int64_t c = t.col * 64 * CPL + lane * CPL;
    const bool in = c < a.D;
    const int64_t r0 = t.row0 + wave * kRows, last = t.rows > 0 ? t.row0 + t.rows - 1 : 0;
    const int rows = rows_of_wave(t, wave);
    const int64_t blocks = (a.D + kCkptBlock - 1) / kCkptBlock;

    BackRows<XF, GF, CPL, PACKED> raw;
    uint32_t scales[PACKED ? kRows : 1];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int64_t r = r0 + i < last ? r0 + i : last, cc = in ? c : 0, at = r * a.D + cc;
        raw.g[i] = load_raw<GF, CPL, STREAM>(a.g, at);
        raw.dy[i] = load_raw<XF, CPL, STREAM>(a.dy, at);
        if constexpr (PACKED) {
            if constexpr (CPL == 1) raw.code[i][0] = a.u[at];
            else load_words<CPL / 4, STREAM>(a.u + at, raw.code[i]);
            scales[i] = a.us[r * blocks + cc / kCkptBlock];
        } else {
            raw.x[i] = load_raw<XF, CPL, STREAM>(a.x, at);
        }
    }
    if constexpr (PACKED) {
#pragma unroll
        for (int i = 0; i < kRows; i += 4)
            raw.scale[i / 4] = scales[i] | scales[i + 1] << 8 | scales[i + 2] << 16 | scales[i + 3] << 24;
    }
    Marks m{0, 0, 0};
    int64_t reach = t.at > 0 ? t.at : -1;
    if constexpr (FLAT) {
        m = marks_of(a, r0, rows);
        reach = 0;
        if (t.rows == kScanSeg) {  // segments on to the one where the sequence of the last row ends
            const int64_t next = offset_of(a, seq_of(a, last) + 1), end = next < total ? next : total;
            reach = end > last ? (end - 1) / kScanSeg - t.id : 0;
        }
    }
    by_form(a, [&](auto logit, auto mix) {
        bwd_body<decltype(logit)::value, decltype(mix)::value, XF, GF, CPL, FLAT, PACKED, STREAM>(a, p, t, m, raw, rows, r0, c, in,
                                                                                         reach, x, kept);
    });
}

template <bool XF, bool GF, int CPL>
void bwd(const ScanArgs& a, hipStream_t st) {
    const ScanPlan p = scan_plan(a, CPL, a.dh_final, a.dh0, st);
    if (a.total == 0) return;
    const dim3 grid(p.cols * p.chains * p.per_chain), block(kThreads);
    const bool stream = a.total * a.D * ((XF ? 8 : 4) + (GF ? 8 : 4)) > kStreamBytes;
    by_kind<CPL>(scan_flat(a), a.u, stream, [&](auto flat, auto packed, auto s) {
        hipLaunchKernelGGL((scan_bwd_kernel<XF, GF, CPL, decltype(flat)::value, decltype(packed)::value, decltype(s)::value>),
                           grid, block, 0, st, a, p);
    });
}

}  // namespace

template <bool XF>
void scan_bwd_of(const ScanArgs& a, hipStream_t st) {
    const bool wide = a.D % 4 == 0;
    if (a.g_f32) wide ? bwd<XF, true, 4>(a, st) : bwd<XF, true, 1>(a, st);
    else wide ? bwd<XF, false, 4>(a, st) : bwd<XF, false, 1>(a, st);
}

}  // namespace kda
