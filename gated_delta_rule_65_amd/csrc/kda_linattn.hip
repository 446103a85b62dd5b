// Linear attention with a decay for each head, forward and backward (mathematics and layouts: include/kda_layer.h).
//
// Over a chunk of C tokens that begins with state S (rows r, i of the chunk from 0; a the decay):
//     o_r = scale (a^(r+1) S^T q_r + sum over i <= r of a^(r-i) (q_r . k_i) v_i)
//     S'  = a^n S + sum over i of a^(n-1-i) k_i v_i^T                                   (n tokens in the chunk)
// The backward pass is three recurrences of the same shape: dq_t = scale S_t d_o_t is the forward one of S^T with d_o, v, k in
// the places of q, k, v.  dk_t = dS_t v_t and dv_t = dS_t^T k_t run from the last token back, on dS^T with v, d_o, q and on dS
// with k, q, d_o; their state is carried as dL/dS of the token before (decayed already), so that a decay of zero divides
// nothing: row r (from the end) takes a^r of it, and a token leaves a^(n-i) of its product.  One kernel does all four.
#include <type_traits>

#include "kda_device.h"
#include "kda_layer_launch.h"

namespace kda {

namespace {

constexpr int kThreads = 256;

// The log of a head's decay: e^-10000 is zero in 32 bits, and has powers where minus infinity has none; a NaN stays one.
__device__ __forceinline__ float log_decay(float g) { return g > 0.f ? 0.f : g < -1e4f ? -1e4f : g; }

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

// ------------------------------------------------------------------------------------------------ segments
//
// A sequence is cut into segments of L tokens, each a workgroup's way through its chunks; the states between them come from a
// pass over k and v before (segments' own states, then a fold over them).
struct Segs {
    const int32_t* cu;
    int64_t T_fixed, N, total, L;
    int64_t per_seq;  // equally long sequences: segments of each (at least one)
    int H;
};

struct Where {
    int64_t n, begin, end;  // sequence, and the segment's tokens
    int64_t slot;           // its place among the states
    int64_t j, count;       // segment j of count; count 0: a sequence without tokens
};

__device__ __forceinline__ int64_t seq_begin(const Segs& s, int64_t n) {
    const int64_t x = s.cu[n];
    return x < 0 ? 0 : x > s.total ? s.total : x;
}

// The segment of a slot; count < 0: there is none.  Packed sequence n takes the slots from floor(begin / L) + n on: no two
// the same, and one at least for each sequence.  64 sequences are looked at together.
__device__ __forceinline__ Where where_of(const Segs& s, int64_t slot) {
    Where w;
    w.slot = slot;
    if (!s.cu) {
        w.n = slot / s.per_seq;
        w.j = slot - w.n * s.per_seq;
        w.count = (s.T_fixed + s.L - 1) / s.L;
        w.begin = w.n * s.T_fixed;
        w.end = w.begin + s.T_fixed;
    } else {
        int64_t lo = 0, hi = s.N;
        while (hi - lo > 1) {
            const int64_t step = (hi - lo + 63) / 64, at = lo + (int64_t)(threadIdx.x & 63) * step;
            const uint64_t below = __ballot(at < hi && seq_begin(s, at < hi ? at : lo) / s.L + at <= slot);
            if (!below) break;
            lo += (63 - __builtin_clzll(below)) * step;
            hi = lo + step < hi ? lo + step : hi;
        }
        w.n = lo;
        w.begin = seq_begin(s, lo);
        const int64_t e = seq_begin(s, lo + 1);
        w.end = e < w.begin ? w.begin : e;
        w.j = slot - (w.begin / s.L + lo);
        w.count = (w.end - w.begin + s.L - 1) / s.L;
    }
    if (w.n >= s.N || w.j < 0 || w.j >= (w.count ? w.count : 1)) {
        w.count = -1;
        return w;
    }
    w.begin += w.j * s.L;
    if (w.end > w.begin + s.L) w.end = w.begin + s.L;
    return w;
}

// ------------------------------------------------------------------------------------------------ the chunk kernel

// One of the four recurrences, or one of the two passes for the segments' states.
struct LinOp {
    const void *a, *b, *c;  // in the places of q, k, v
    void* out;              // rows, c's shape; without rows, the segments' states
    const float* x0;        // what there is before the first token (behind the last one), or nullptr
    const float* states;    // folded states of the segments, natural [Dk][Dv]
    float* fin;             // what there is at the end, or nullptr
    bool turned;            // states and x0 are taken transposed
    bool back;
    float su, so;           // scales of the state's products, and of the outputs
};

template <bool F32>
struct LFrag;
template <>
struct LFrag<false> {
    bf16x8_t v;
};
template <>
struct LFrag<true> {
    float v[8];
};
__device__ __forceinline__ f32x4_t mma(const LFrag<false>& a, const LFrag<false>& b, f32x4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v, b.v, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4_t mma(const LFrag<true>& a, const LFrag<true>& b, f32x4_t c) {
#pragma unroll
    for (int j = 0; j < 8; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[j], b.v[j], c, 0, 0, 0);
    return c;
}

// x as a sum of PLANES bf16 values, each the nearest to what the ones before leave; in fp32 x itself.
template <int PLANES, bool F32>
__device__ __forceinline__ void split(const float x[8], LFrag<F32> f[PLANES]) {
    if constexpr (F32) {
#pragma unroll
        for (int j = 0; j < 8; ++j) f[0].v[j] = x[j];
    } else {
        float r[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) r[j] = x[j];
#pragma unroll
        for (int p = 0; p < PLANES; ++p)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const __bf16 h = (__bf16)r[j];
                f[p].v[j] = h;
                r[j] -= (float)h;
            }
    }
}

// Rows of UNITS 16-byte units in LDS.  A unit's place is turned by its row so that neither 16 rows' same unit nor, transposed,
// two units of eight rows meet in a bank.
template <int UNITS, bool F32>
struct Tile {
    static constexpr int BYTES = UNITS * 16;
    static __device__ __forceinline__ int place(int row, int unit) {
        int f;
        if constexpr (UNITS == 8) f = (row & 6) | (row >> 3 & 1);
        else if constexpr (F32) f = row & 15;
        else f = (row & 7) << 1 | (row >> 3 & 1);
        return row * BYTES + (unit ^ f) * 16;
    }
};

// Four values of one column of a bf16 tile: lane i of 16 gives the place of four values of row i/4, and gets column i.
__device__ __forceinline__ bf16x4_t read_turned(const char* p) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4bf16((__attribute__((address_space(3))) bf16x4_t*)const_cast<char*>(p));
}

template <int DA, int DC, bool F32, bool ROWS>
struct LinTile {
    static constexpr int C = F32 ? 32 : 64;      // tokens of a chunk
    static constexpr int ES = F32 ? 4 : 2;
    static constexpr int UA = DA * ES / 16, UC = DC * ES / 16;  // units of a row
    static constexpr int NA = C * UA / kThreads, NC = C * UC / kThreads;  // units a thread moves
    static constexpr int ND = DC / 64;           // 16-column tiles of a wave
    static constexpr int KS = C / 32, RB = C / 16, AS = DA / 32, CT = DA / 16;
    static constexpr int PL = F32 ? 1 : 2;       // planes of scores and of the state
    static constexpr int VL = F32 ? 1 : 3;       // planes of the weighted values
    static constexpr int PU = C * ES / 16;       // units of a row of scores
    static constexpr int KB = C * UA * 16, VB = C * UC * 16, PB = C * PU * 16;
    static constexpr int TAB = (C + 4) * 4;
    static constexpr int LDS = KB + VB + TAB + (ROWS ? KB + PL * PB : 0);
};

template <int DA, int DC, bool F32, bool ROWS>
__global__ __launch_bounds__(kThreads, 2) void linattn_chunk_kernel(LinOp op0, LinOp op1, LinOp op2, int ops, Segs segs,
                                                                    const float* g) {
    using G = LinTile<DA, DC, F32, ROWS>;
    using TA = Tile<G::UA, F32>;
    using TC = Tile<G::UC, F32>;
    using TP = Tile<G::PU, F32>;
    constexpr int C = G::C, ND = G::ND;
    __shared__ __align__(16) char lds[G::LDS];
    char* const ldsK = lds;
    char* const ldsV = lds + G::KB;
    float* const tab = reinterpret_cast<float*>(lds + G::KB + G::VB);  // a^0 .. a^C, and what a^C is rounded off by
    char* const ldsQ = lds + G::KB + G::VB + G::TAB;
    char* const ldsP = ldsQ + G::KB;

    // the operations of a segment and head in workgroups of one XCD, next to one another
    const int64_t id = (int64_t)(blockIdx.x / (8 * ops)) * 8 + blockIdx.x % 8;
    const int which = blockIdx.x / 8 % ops;
    const LinOp op = which == 0 ? op0 : which == 1 ? op1 : op2;
    const int H = segs.H, h = id % H;
    const Where w = where_of(segs, id / H);
    if (w.count < 0) return;
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, m = lane & 15, grp = lane >> 4;
    const bool first = op.back ? w.j == w.count - 1 : w.j == 0, last = op.back ? w.j == 0 : w.j + 1 >= w.count;
    if (w.count == 0) {
        if (ROWS && op.fin) {
            const int64_t at = (w.n * H + h) * (int64_t)DA * DC;
            for (int i = tid; i < DA * DC; i += kThreads) op.fin[at + i] = op.x0 ? op.x0[at + i] : 0.f;
        }
        return;
    }
    if (!ROWS && last) return;

    // a column of a wave's 16-column tile d: eight columns of a lane side by side in rows
    auto col = [&](int i, int d) { return ND == 2 ? 32 * wave + 8 * (i >> 2) + 4 * d + (i & 3) : 16 * wave + i; };

    const double lg = log_decay(g[h]);
    for (int i = tid; i <= C; i += kThreads) tab[i] = (float)exp(lg * i);
    if (tid == 0) tab[C + 1] = (float)(exp(lg * C) - (double)(float)exp(lg * C));

    f32x4_t S[G::CT][ND];
#pragma unroll
    for (int ct = 0; ct < G::CT; ++ct)
#pragma unroll
        for (int d = 0; d < ND; ++d) S[ct][d] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    if constexpr (ROWS) {
        const float* x = first ? op.x0 : op.states;
        if (x) {
            x += ((first ? w.n : op.back ? w.slot + 1 : w.slot - 1) * H + h) * (int64_t)DA * DC;
#pragma unroll
            for (int ct = 0; ct < G::CT; ++ct)
#pragma unroll
                for (int d = 0; d < ND; ++d) {
                    const int c = col(m, d), r = 16 * ct + 4 * grp;
                    if (op.turned) S[ct][d] = *reinterpret_cast<const f32x4_t*>(x + (int64_t)c * DA + r);
                    else
#pragma unroll
                        for (int j = 0; j < 4; ++j) S[ct][d][j] = x[(r + j) * DC + c];
                }
        }
    }

    const int64_t tokens = w.end - w.begin, chunks = (tokens + C - 1) / C;
    // row r of chunk c, in the order of the recurrence
    auto token = [&](int64_t c, int r) { return op.back ? w.end - 1 - (c * C + r) : w.begin + c * C + r; };

    uint4 ra[ROWS ? G::NA : 1], rb[G::NA], rc[G::NC];
    auto fetch = [&](int64_t c) {
        const uint4 zero = make_uint4(0, 0, 0, 0);
        const int n = tokens - c * C < C ? (int)(tokens - c * C) : C;
#pragma unroll
        for (int x = 0; x < G::NA; ++x) {
            const int u = tid + x * kThreads, row = u / G::UA;
            const int64_t at = ((token(c, row < n ? row : 0) * H + h) * DA) * G::ES / 16 + u % G::UA;
            if constexpr (ROWS) {
                ra[x] = static_cast<const uint4*>(op.a)[at];
                if (row >= n) ra[x] = zero;
            }
            rb[x] = static_cast<const uint4*>(op.b)[at];
            if (row >= n) rb[x] = zero;
        }
#pragma unroll
        for (int x = 0; x < G::NC; ++x) {
            const int u = tid + x * kThreads, row = u / G::UC;
            rc[x] = static_cast<const uint4*>(op.c)[((token(c, row < n ? row : 0) * H + h) * DC) * G::ES / 16 + u % G::UC];
            if (row >= n) rc[x] = zero;
        }
    };
    // Contracted channels are taken in the order in which two 16-row tiles of a product lie in a lane: group g holds 4g .. +3
    // and 16 + 4g .. +3 of each 32.  Rows of `a` are stored in that order.
    auto stage = [&]() {
#pragma unroll
        for (int x = 0; x < G::NA; ++x) {
            const int u = tid + x * kThreads, row = u / G::UA, v = u % G::UA;
            *reinterpret_cast<uint4*>(ldsK + TA::place(row, v)) = rb[x];
            if constexpr (ROWS && F32) {
                *reinterpret_cast<uint4*>(ldsQ + TA::place(row, (v & ~7) + 2 * (v & 3) + (v >> 2 & 1))) = ra[x];
            } else if constexpr (ROWS) {
                const int to = (v & ~3) + 2 * (v & 1), half = (v >> 1 & 1) * 8;
                *reinterpret_cast<uint2*>(ldsQ + TA::place(row, to) + half) = make_uint2(ra[x].x, ra[x].y);
                *reinterpret_cast<uint2*>(ldsQ + TA::place(row, to + 1) + half) = make_uint2(ra[x].z, ra[x].w);
            }
        }
#pragma unroll
        for (int x = 0; x < G::NC; ++x) {
            const int u = tid + x * kThreads;
            *reinterpret_cast<uint4*>(ldsV + TC::place(u / G::UC, u % G::UC)) = rc[x];
        }
    };

    // fragments: eight contracted values of row (or column) m
    auto frag_a = [&](int row, int s) {
        LFrag<F32> f;
        if constexpr (F32) {
            const f32x4_t x = *reinterpret_cast<const f32x4_t*>(ldsQ + TA::place(row, 8 * s + 2 * grp));
            const f32x4_t y = *reinterpret_cast<const f32x4_t*>(ldsQ + TA::place(row, 8 * s + 2 * grp + 1));
#pragma unroll
            for (int j = 0; j < 4; ++j) f.v[j] = x[j], f.v[4 + j] = y[j];
        } else {
            f.v = *reinterpret_cast<const bf16x8_t*>(ldsQ + TA::place(row, 4 * s + grp));
        }
        return f;
    };
    auto frag_b = [&](int row, int s) {
        LFrag<F32> f;
        if constexpr (F32) {
            const f32x4_t x = *reinterpret_cast<const f32x4_t*>(ldsK + TA::place(row, 8 * s + grp));
            const f32x4_t y = *reinterpret_cast<const f32x4_t*>(ldsK + TA::place(row, 8 * s + 4 + grp));
#pragma unroll
            for (int j = 0; j < 4; ++j) f.v[j] = x[j], f.v[4 + j] = y[j];
        } else {
            const bf16x4_t x = *reinterpret_cast<const bf16x4_t*>(ldsK + TA::place(row, 4 * s + (grp >> 1)) + 8 * (grp & 1));
            const bf16x4_t y = *reinterpret_cast<const bf16x4_t*>(ldsK + TA::place(row, 4 * s + 2 + (grp >> 1)) + 8 * (grp & 1));
            f.v = __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
        }
        return f;
    };
    // columns of a tile over 32 tokens, in the same order
    auto frag_bt = [&](int ct, int ks) {
        LFrag<F32> f;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int row = 32 * ks + 16 * half + 4 * grp;
            if constexpr (F32) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    f.v[4 * half + j] = *reinterpret_cast<const float*>(ldsK + TA::place(row + j, 4 * ct + (m >> 2)) + 4 * (m & 3));
            } else {
                const bf16x4_t x = read_turned(ldsK + TA::place(row + (m >> 2), 2 * ct + (m >> 1 & 1)) + 8 * (m & 1));
#pragma unroll
                for (int j = 0; j < 4; ++j) f.v[4 * half + j] = x[j];
            }
        }
        return f;
    };
    auto frag_ct = [&](int d, int ks) {
        LFrag<F32> f;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int row = 32 * ks + 16 * half + 4 * grp;
            if constexpr (F32) {
                const int c = col(m, d);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    f.v[4 * half + j] = *reinterpret_cast<const float*>(ldsV + TC::place(row + j, c >> 2) + 4 * (c & 3));
            } else {
                const int c = ND == 2 ? 32 * wave + 8 * (m & 3) + 4 * d : 16 * wave + 4 * (m & 3);
                const bf16x4_t x = read_turned(ldsV + TC::place(row + (m >> 2), c >> 3) + (c & 4) * 2);
#pragma unroll
                for (int j = 0; j < 4; ++j) f.v[4 * half + j] = x[j];
            }
        }
        return f;
    };

    fetch(0);
    __syncthreads();
    float into[G::RB];  // what a row takes of the state
#pragma unroll
    for (int r = 0; r < G::RB; ++r) into[r] = op.so * tab[16 * r + m + (op.back ? 0 : 1)];
    const float sp = op.su * op.so;

    for (int64_t c = 0; c < chunks; ++c) {
        const int n = tokens - c * C < C ? (int)(tokens - c * C) : C;
        stage();
        lds_barrier();
        if (c + 1 < chunks) fetch(c + 1);

        f32x4_t O[G::RB][ND];
        if constexpr (ROWS) {
            f32x4_t P[G::RB];
#pragma unroll
            for (int r = 0; r < G::RB; ++r) {
                P[r] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int d = 0; d < ND; ++d) O[r][d] = f32x4_t{0.f, 0.f, 0.f, 0.f};
            }
#pragma unroll
            for (int s = 0; s < G::AS; ++s) {
                LFrag<F32> st[ND][G::PL];
#pragma unroll
                for (int d = 0; d < ND; ++d) {
                    float x[8];
#pragma unroll
                    for (int j = 0; j < 4; ++j) x[j] = S[2 * s][d][j], x[4 + j] = S[2 * s + 1][d][j];
                    split<G::PL, F32>(x, st[d]);
                }
                LFrag<F32> kf;
                if (wave < G::RB) kf = frag_b(16 * wave + m, s);
#pragma unroll
                for (int r = 0; r < G::RB; ++r) {
                    const LFrag<F32> qf = frag_a(16 * r + m, s);
                    if (wave <= r) P[r] = mma(kf, qf, P[r]);
#pragma unroll
                    for (int d = 0; d < ND; ++d)
#pragma unroll
                        for (int p = 0; p < G::PL; ++p) O[r][d] = mma(st[d][p], qf, O[r][d]);
                }
            }
            // scores of rows 16r + m against tokens 16 wave + 4 grp + j
#pragma unroll
            for (int r = 0; r < G::RB; ++r) {
                if (wave <= r) {
                    float x[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int apart = 16 * (r - wave) + m - 4 * grp - j;
                        x[j] = apart >= 0 ? P[r][j] * (sp * tab[apart >= 0 ? apart : 0]) : 0.f;
                    }
                    const int unit8 = 4 * (wave >> 1) + grp, half = wave & 1;  // of eight values
                    if constexpr (F32) {
                        *reinterpret_cast<f32x4_t*>(ldsP + TP::place(16 * r + m, 2 * unit8 + half)) = f32x4_t{x[0], x[1], x[2], x[3]};
                    } else {
                        bf16x4_t hi, lo;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            hi[j] = (__bf16)x[j];
                            lo[j] = (__bf16)(x[j] - (float)hi[j]);
                        }
                        char* to = ldsP + TP::place(16 * r + m, unit8) + 8 * half;
                        *reinterpret_cast<bf16x4_t*>(to) = hi;
                        *reinterpret_cast<bf16x4_t*>(to + G::PB) = lo;
                    }
                }
#pragma unroll
                for (int d = 0; d < ND; ++d)
#pragma unroll
                    for (int j = 0; j < 4; ++j) O[r][d][j] *= into[r];
            }
            // the tiles above the diagonal that the products reach
            if (wave & 1) {
                const int r = wave - 1;
                if (r < G::RB) {
                    const int unit8 = 4 * (wave >> 1) + grp;
                    if constexpr (F32) {
                        *reinterpret_cast<f32x4_t*>(ldsP + TP::place(16 * r + m, 2 * unit8 + 1)) = f32x4_t{0.f, 0.f, 0.f, 0.f};
                    } else {
                        char* to = ldsP + TP::place(16 * r + m, unit8) + 8;
                        *reinterpret_cast<uint2*>(to) = make_uint2(0, 0);
                        *reinterpret_cast<uint2*>(to + G::PB) = make_uint2(0, 0);
                    }
                }
            }
            lds_barrier();
        }

        LFrag<F32> vf[G::KS][ND];
#pragma unroll
        for (int ks = 0; ks < G::KS; ++ks)
#pragma unroll
            for (int d = 0; d < ND; ++d) vf[ks][d] = frag_ct(d, ks);

        if constexpr (ROWS) {
            // A value that is not finite must not meet the zeros of earlier rows: such values are left out of the product, and
            // its column is made NaN from that token on.
            int bad[ND];
            bool any = false;
#pragma unroll
            for (int d = 0; d < ND; ++d) {
                bad[d] = C;
#pragma unroll
                for (int ks = G::KS - 1; ks >= 0; --ks)
#pragma unroll
                    for (int j = 7; j >= 0; --j)
                        if (!(fabsf((float)vf[ks][d].v[j]) < __builtin_inff())) bad[d] = 32 * ks + 16 * (j >> 2) + 4 * grp + (j & 3);
                any |= bad[d] < C;
            }
            const bool marked = __ballot(any) != 0;
            LFrag<F32> clean[G::KS][ND];
#pragma unroll
            for (int ks = 0; ks < G::KS; ++ks)
#pragma unroll
                for (int d = 0; d < ND; ++d) clean[ks][d] = vf[ks][d];
            if (marked) {
#pragma unroll
                for (int d = 0; d < ND; ++d) {
                    bad[d] = min(bad[d], __shfl_xor(bad[d], 16));
                    bad[d] = min(bad[d], __shfl_xor(bad[d], 32));
#pragma unroll
                    for (int ks = 0; ks < G::KS; ++ks)
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (!(fabsf((float)clean[ks][d].v[j]) < __builtin_inff())) clean[ks][d].v[j] = 0.f;
                }
            }
#pragma unroll
            for (int r = 0; r < G::RB; ++r) {
#pragma unroll
                for (int ks = 0; ks <= r / 2; ++ks)
#pragma unroll
                    for (int p = 0; p < G::PL; ++p) {
                        LFrag<F32> pf;
                        if constexpr (F32) {
                            const f32x4_t x = *reinterpret_cast<const f32x4_t*>(ldsP + TP::place(16 * r + m, 8 * ks + 2 * grp));
                            const f32x4_t y = *reinterpret_cast<const f32x4_t*>(ldsP + TP::place(16 * r + m, 8 * ks + 2 * grp + 1));
#pragma unroll
                            for (int j = 0; j < 4; ++j) pf.v[j] = x[j], pf.v[4 + j] = y[j];
                        } else {
                            pf.v = *reinterpret_cast<const bf16x8_t*>(ldsP + p * G::PB + TP::place(16 * r + m, 4 * ks + grp));
                        }
#pragma unroll
                        for (int d = 0; d < ND; ++d) O[r][d] = mma(clean[ks][d], pf, O[r][d]);
                    }
                if (marked) {
#pragma unroll
                    for (int d = 0; d < ND; ++d)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (16 * r + m >= __shfl(bad[d], 4 * grp + j)) O[r][d][j] = __builtin_nanf("");
                }
                const int row = 16 * r + m;
                if (row < n) {
                    const int64_t at = (token(c, row) * H + h) * DC + col(4 * grp, 0);
                    if constexpr (F32) {
#pragma unroll
                        for (int d = 0; d < ND; ++d)
                            *reinterpret_cast<f32x4_t*>(static_cast<float*>(op.out) + at + 4 * d) = O[r][d];
                    } else if constexpr (ND == 2) {
                        bf16x8_t x;
#pragma unroll
                        for (int j = 0; j < 4; ++j) x[j] = (__bf16)O[r][0][j], x[4 + j] = (__bf16)O[r][1][j];
                        *reinterpret_cast<bf16x8_t*>(static_cast<__bf16*>(op.out) + at) = x;
                    } else {
                        bf16x4_t x;
#pragma unroll
                        for (int j = 0; j < 4; ++j) x[j] = (__bf16)O[r][0][j];
                        *reinterpret_cast<bf16x4_t*>(static_cast<__bf16*>(op.out) + at) = x;
                    }
                }
            }
        }

        // the state: decayed in 32 bits and what the power is rounded off by, so that thousands of chunks do not add up to more
        // than a rounding each; the weighted values as sums of three bf16 values, which hold all of their 24 bits
        {
            const float dec = tab[n], rest = n == C ? tab[C + 1] : 0.f;
#pragma unroll
            for (int ct = 0; ct < G::CT; ++ct)
#pragma unroll
                for (int d = 0; d < ND; ++d)
#pragma unroll
                    for (int j = 0; j < 4; ++j) S[ct][d][j] = fmaf(S[ct][d][j], rest, S[ct][d][j] * dec);
        }
#pragma unroll
        for (int ks = 0; ks < G::KS; ++ks) {
            LFrag<F32> vb[ND][G::VL];
#pragma unroll
            for (int d = 0; d < ND; ++d) {
                float x[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int left = n - 1 - (32 * ks + 16 * (j >> 2) + 4 * grp + (j & 3));
                    x[j] = (float)vf[ks][d].v[j] * (op.su * tab[(left > 0 ? left : 0) + (op.back ? 1 : 0)]);
                }
                split<G::VL, F32>(x, vb[d]);
            }
#pragma unroll
            for (int ct = 0; ct < G::CT; ++ct) {
                const LFrag<F32> kt = frag_bt(ct, ks);
#pragma unroll
                for (int d = 0; d < ND; ++d)
#pragma unroll
                    for (int p = 0; p < G::VL; ++p) S[ct][d] = mma(kt, vb[d][p], S[ct][d]);
            }
        }
        lds_barrier();
    }

    float* to = nullptr;
    if constexpr (ROWS) {
        if (last && op.fin) to = op.fin + (w.n * H + h) * (int64_t)DA * DC;
    } else {
        to = static_cast<float*>(op.out) + (w.slot * H + h) * (int64_t)DA * DC;
    }
    if (to) {
#pragma unroll
        for (int ct = 0; ct < G::CT; ++ct)
#pragma unroll
            for (int d = 0; d < ND; ++d)
#pragma unroll
                for (int j = 0; j < 4; ++j) to[(16 * ct + 4 * grp + j) * DC + col(m, d)] = S[ct][d][j];
    }
}

// The states behind (with `back` before) each segment from the segments' own ones, in place: X_j = a^length X_(j-1) + U_j.
// A thread holds four values of a head's state through all segments.
struct FoldOp {
    float* states;
    const float* x0;
    bool back;
};
__global__ __launch_bounds__(kThreads) void linattn_fold_kernel(FoldOp op0, FoldOp op1, Segs segs, const float* g, int size) {
    const FoldOp op = blockIdx.y ? op1 : op0;
    const int per = size / (4 * kThreads);
    const int64_t nh = blockIdx.x / per, n = nh / segs.H;
    const int h = nh % segs.H, at = (blockIdx.x % per) * 4 * kThreads + 4 * threadIdx.x;
    const int64_t slot0 = segs.cu ? seq_begin(segs, n) / segs.L + n : n * segs.per_seq;
    const Where w = where_of(segs, slot0);
    if (w.n != n || w.count < 2) return;
    const int64_t length = segs.cu ? seq_begin(segs, n + 1) - seq_begin(segs, n) : segs.T_fixed;
    const double lg = log_decay(g[h]);
    const float whole = (float)exp(lg * segs.L), tail = (float)exp(lg * (length - (w.count - 1) * segs.L));
    f32x4_t x = {0.f, 0.f, 0.f, 0.f};
    if (op.x0) x = *reinterpret_cast<const f32x4_t*>(op.x0 + nh * size + at);
    const int64_t step = (int64_t)segs.H * size;
    f32x4_t* p = reinterpret_cast<f32x4_t*>(op.states + (slot0 * segs.H + h) * (int64_t)size + at);
    constexpr int AHEAD = 8;
    for (int64_t j0 = 0; j0 < w.count - 1; j0 += AHEAD) {
        f32x4_t u[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int64_t j = j0 + i < w.count - 1 ? j0 + i : w.count - 2;
            u[i] = p[(op.back ? w.count - 1 - j : j) * (step / 4)];
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int64_t j = j0 + i;
            if (j >= w.count - 1) break;
            const float f = op.back && j == 0 ? tail : whole;
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = fmaf(f, x[e], u[i][e]);
            p[(op.back ? w.count - 1 - j : j) * (step / 4)] = x;
        }
    }
}

// ------------------------------------------------------------------------------------------------ one token

// A workgroup holds one head's state, four columns of RPT rows a thread, and reads and writes it once.
template <int DK, int DV, bool F32>
__global__ __launch_bounds__(256) void linattn_step_kernel(const void* q, const void* k, const void* v, const float* g,
                                                           const float* s_in, float* s_out, void* o, int H, float scale) {
    constexpr int C4 = DV / 4, RG = 256 / C4, RPT = DK / RG;
    __shared__ float sq[DK], sk[DK];
    __shared__ f32x4_t part[RG][C4];
    const int64_t bh = blockIdx.x;
    const int tid = threadIdx.x, c4 = tid % C4, rg = tid / C4;
    const int ti = tid % DK;
    const float qr = load1<F32>(q, bh * DK + ti), kr = load1<F32>(k, bh * DK + ti);
    float x[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = load1<F32>(v, bh * DV + 4 * c4 + j);
    const float decay = expf(log_decay(g[bh % H]));
    const f32x4_t* S = reinterpret_cast<const f32x4_t*>(s_in + bh * (int64_t)DK * DV);
    f32x4_t* So = reinterpret_cast<f32x4_t*>(s_out + bh * (int64_t)DK * DV);
    f32x4_t s[RPT];
#pragma unroll
    for (int i = 0; i < RPT; ++i) s[i] = __builtin_nontemporal_load(&S[(rg + RG * i) * C4 + c4]);
    sq[ti] = qr;
    sk[ti] = kr;
    __syncthreads();
    f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const int r = rg + RG * i;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            s[i][j] = fmaf(decay, s[i][j], sk[r] * x[j]);
            acc[j] = fmaf(sq[r], s[i][j], acc[j]);
        }
        __builtin_nontemporal_store(s[i], &So[r * C4 + c4]);
    }
    part[rg][c4] = acc;
    __syncthreads();
    if (tid < DV) {
        float sum = 0.f;
#pragma unroll
        for (int r = 0; r < RG; ++r) sum += part[r][tid / 4][tid % 4];
        store1<F32>(o, bh * DV + tid, scale * sum);
    }
}

// ------------------------------------------------------------------------------------------------ launches

// Tokens of a segment.  Two workgroups fit on a CU: with 512 segments every place has one.  A segment's state is written,
// folded and read, four times its size, which 256 tokens outweigh.
int64_t segment_tokens(int64_t total, int H) {
    const int64_t even = (total * H + 511) / 512, up = (even + 63) / 64 * 64;
    return up < 256 ? 256 : up;
}

Segs segs_of(const LinArgs& a) {
    Segs s{a.cu, a.T_fixed, a.N, a.total, segment_tokens(a.total, a.H), 1, a.H};
    if (!a.cu && a.T_fixed > s.L) s.per_seq = (a.T_fixed + s.L - 1) / s.L;
    return s;
}

int64_t slots_of(const Segs& s) { return s.cu ? s.total / s.L + s.N : s.N * s.per_seq; }

// Whether a sequence may have more than one segment.
bool is_split(const Segs& s) { return s.cu ? s.total > s.L : s.per_seq > 1; }

using I64 = std::integral_constant<int, 64>;
using I128 = std::integral_constant<int, 128>;

template <bool ROWS>
void chunks(const LinArgs& a, const Segs& s, std::initializer_list<LinOp> ops, int DA, int DC, hipStream_t st) {
    LinOp op[3] = {};
    int count = 0;
    for (const LinOp& o : ops) op[count++] = o;
    const int64_t each = (slots_of(s) * a.H + 7) / 8 * 8;  // workgroups behind the last segment find none
    auto run = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3((unsigned)(each * count)), dim3(kThreads), 0, st, op[0], op[1], op[2], count, s, a.g);
    };
    auto types = [&](auto da, auto dc) {
        constexpr int A = decltype(da)::value, B = decltype(dc)::value;
        a.f32 ? run(linattn_chunk_kernel<A, B, true, ROWS>) : run(linattn_chunk_kernel<A, B, false, ROWS>);
    };
    if (DA == 64) DC == 64 ? types(I64(), I64()) : types(I64(), I128());
    else DC == 64 ? types(I128(), I64()) : types(I128(), I128());
}

void fold(const LinArgs& a, const Segs& s, FoldOp one, const FoldOp* two, hipStream_t st) {
    const int size = a.Dk * a.Dv;
    hipLaunchKernelGGL(linattn_fold_kernel, dim3((unsigned)(a.N * a.H * (size / (4 * kThreads))), two ? 2 : 1), dim3(kThreads), 0,
                       st, one, two ? *two : one, s, a.g, size);
}

}  // namespace

int64_t linattn_workspace_bytes(const LinArgs& a, bool backward) {
    const int64_t L = segment_tokens(a.total, a.H);
    if (a.total <= L) return 0;
    return (a.total / L + a.N) * a.H * a.Dk * (int64_t)a.Dv * 4 * (backward ? 2 : 1);
}

int64_t linattn_groups(const LinArgs& a, bool backward) {
    const Segs s = segs_of(a);
    const int64_t chunk = (slots_of(s) * a.H + 8) * (backward ? 3 : 1), folds = a.N * a.H * (a.Dk * a.Dv / (4 * kThreads));
    return chunk > folds ? chunk : folds;
}

hipError_t launch_linattn_fwd(const LinArgs& a, hipStream_t st) {
    const Segs s = segs_of(a);
    float* states = static_cast<float*>(a.ws);
    if (is_split(s)) {
        chunks<false>(a, s, {LinOp{nullptr, a.k, a.v, states, nullptr, nullptr, nullptr, false, false, 1.f, 1.f}}, a.Dk, a.Dv, st);
        fold(a, s, FoldOp{states, a.s0, false}, nullptr, st);
    }
    chunks<true>(a, s, {LinOp{a.q, a.k, a.v, a.o, a.s0, states, a.s_final, false, false, 1.f, a.scale}}, a.Dk, a.Dv, st);
    return hipGetLastError();
}

hipError_t launch_linattn_bwd(const LinArgs& a, hipStream_t st) {
    const Segs s = segs_of(a);
    float* states = static_cast<float*>(a.ws);
    float* grads = states + slots_of(s) * a.H * a.Dk * a.Dv;
    if (is_split(s)) {
        chunks<false>(a, s, {LinOp{nullptr, a.k, a.v, states, nullptr, nullptr, nullptr, false, false, 1.f, 1.f},
                             LinOp{nullptr, a.q, a.d_o, grads, nullptr, nullptr, nullptr, false, true, a.scale, 1.f}},
                      a.Dk, a.Dv, st);
        const FoldOp two{grads, a.d_sfinal, true};
        fold(a, s, FoldOp{states, a.s0, false}, &two, st);
    }
    const LinOp dq{a.d_o, a.v, a.k, a.dq, a.s0, states, nullptr, true, false, 1.f, a.scale};
    const LinOp dk{a.v, a.d_o, a.q, a.dk, a.d_sfinal, grads, nullptr, true, true, a.scale, 1.f};
    const LinOp dv{a.k, a.q, a.d_o, a.dv, a.d_sfinal, grads, a.ds0, false, true, a.scale, 1.f};
    if (a.Dk == a.Dv) {
        chunks<true>(a, s, {dq, dk, dv}, a.Dk, a.Dv, st);
    } else {
        chunks<true>(a, s, {dq, dk}, a.Dv, a.Dk, st);
        chunks<true>(a, s, {dv}, a.Dk, a.Dv, st);
    }
    return hipGetLastError();
}

hipError_t launch_linattn_step(const LinArgs& a, const float* s_in, float* s_out, hipStream_t st) {
    const dim3 grid((unsigned)(a.N * a.H));
    auto run = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid, dim3(256), 0, st, a.q, a.k, a.v, a.g, s_in, s_out, a.o, a.H, a.scale);
    };
    auto types = [&](auto dk, auto dv) {
        constexpr int DK = decltype(dk)::value, DV = decltype(dv)::value;
        a.f32 ? run(linattn_step_kernel<DK, DV, true>) : run(linattn_step_kernel<DK, DV, false>);
    };
    if (a.Dk == 64) a.Dv == 64 ? types(I64(), I64()) : types(I64(), I128());
    else a.Dv == 64 ? types(I128(), I64()) : types(I128(), I128());
    return hipGetLastError();
}

}  // namespace kda
