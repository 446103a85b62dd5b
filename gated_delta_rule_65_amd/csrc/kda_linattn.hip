// Linear attention with a decay for each head, forward and backward (mathematics and layouts: include/kda_layer.h).
//
// Over a chunk of C tokens that begins with state S (rows r, i of the chunk from 0; a the decay):
//     o_r = scale (a^(r+1) S^T q_r + sum over i <= r of a^(r-i) (q_r . k_i) v_i)
//     S'  = a^n S + sum over i of a^(n-1-i) k_i v_i^T                                   (n tokens in the chunk)
// The backward pass is three recurrences of the same shape: dq_t = scale S_t d_o_t is the forward one of S^T with d_o, v, k in
// the places of q, k, v.  dk_t = dS_t v_t and dv_t = dS_t^T k_t run from the last token back, on dS^T with v, d_o, q and on dS
// with k, q, d_o; their state is carried as dL/dS of the token before (decayed already), so that a decay of zero divides
// nothing: row r (from the end) takes a^r of it, and a token leaves a^(n-i) of its product.  One kernel does all four.
//
// Two passes over a sequence's segments: the first makes what each segment adds to the state (reads k and v), the second
// starts every segment from the state before it.  One pass from begin to end would read k and v once, but has one workgroup
// for a sequence and head, 64 for B=4 H=16: 620 us where two passes take 215.
//
// bf16: products of bf16 on the matrix units, with what is not bf16 (the state, the scores, the weighted values) as the sum of three
// bf16 values, which hold all of its 24 bits: a result that is small beside its terms is as exact as in fp32.  Two planes, 16 bits,
// would take 189 us instead of 215 and 233 instead of 281 for dq, dk, dv of T=4096, with errors of 2^-17 of the terms.  fp32: products of fp32 (16x16x4).
//
// B=4 T=8192 H=16 D=128 bf16: 59 us for the segments' states and 145 for the outputs, 215 the call; reading q, k, v and writing o
// once takes 86 at a copy's rate, k and v twice 129.  What bounds the outputs' pass is that vector and matrix instructions
// of a SIMD's two waves do not overlap well: the vector units are busy for 48% of the time, the matrix units for 43%
// (one product and four vector instructions take 26 to 29 cycles together, 17.5 and 18.6 alone).
#include <type_traits>

#include "kda_device.h"
#include "kda_layer_launch.h"

namespace kda {

namespace {

constexpr int kThreads = 256;  // of the fold's workgroups
#define KDA_INLINE __attribute__((always_inline))  // a state that a call is given by reference would lie in memory

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
    int64_t base;           // the sequence's first place among the states
    int64_t j, count;       // segment j of count; count 0: a sequence without tokens
    int64_t tail;           // tokens of the sequence's last segment
};

__device__ __forceinline__ int64_t seq_begin(const Segs& s, int64_t n) {
    const int64_t x = s.cu[n];
    return x < 0 ? 0 : x > s.total ? s.total : x;
}

// The last packed sequence n whose begin is below what is looked for; 64 sequences are looked at together.
template <typename Below>
__device__ __forceinline__ int64_t last_below(const Segs& s, Below below) {
    int64_t lo = 0, hi = s.N;
    while (hi - lo > 1) {
        const int64_t step = (hi - lo + 63) / 64, at = lo + (int64_t)(threadIdx.x & 63) * step;
        const uint64_t found = __ballot(at < hi && below(seq_begin(s, at < hi ? at : lo), at));
        if (!found) break;
        lo += (63 - __builtin_clzll(found)) * step;
        hi = lo + step < hi ? lo + step : hi;
    }
    return lo;
}

__device__ __forceinline__ Where sequence(const Segs& s, int64_t n) {
    Where w;
    w.n = n;
    if (!s.cu) {
        w.begin = n * s.T_fixed;
        w.end = w.begin + s.T_fixed;
    } else {
        w.begin = seq_begin(s, n);
        const int64_t e = seq_begin(s, n + 1);
        w.end = e < w.begin ? w.begin : e;
    }
    w.j = 0;
    w.count = (w.end - w.begin + s.L - 1) / s.L;
    w.tail = w.end - w.begin - (w.count - 1) * s.L;
    w.base = w.begin / s.L;
    return w;
}

// The segment of a slot; count < 0: there is none.  For the outputs packed sequence n takes the slots from floor(begin / L) + n
// on: no two the same, and one at least for each sequence.
//
// States are kept between segments only, one fewer than a sequence has segments, from floor(begin / L) on: forward that behind
// segment j has place j of them, backward that before it place j - 1.  Sequences with one segment need none, and all of them
// lie below total / L: the next sequence begins behind all but the last segment.  The pass for the segments' states has these
// places for slots, so that many short sequences cost it nothing.
template <bool ROWS>
__device__ __forceinline__ Where where_of(const Segs& s, int64_t slot, bool back) {
    const int64_t each = s.per_seq - (ROWS ? 0 : 1);
    const int64_t n = s.cu ? last_below(s, [&](int64_t begin, int64_t at) { return begin / s.L + (ROWS ? at : 0) <= slot; }) : slot / each;
    if (n >= s.N) {
        Where w{};
        w.count = -1;
        return w;
    }
    Where w = sequence(s, n);
    w.j = slot - (s.cu ? w.base + (ROWS ? n : 0) : n * each);
    if (w.j < 0 || w.j >= (ROWS ? (w.count ? w.count : 1) : w.count - 1)) {
        w.count = -1;
        return w;
    }
    if (!ROWS && back) ++w.j;
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

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));

// Two values as bf16, the nearest ones; and what they stand for.
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{a, b}, bf16x2_t));
}
__device__ __forceinline__ float low_of(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float high_of(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }

// x less the low, the high half of u: one dot product of two pairs, with -1 and 0, instead of taking the half out and
// subtracting.  It is exact: the difference of a value and its nearest bf16 has few enough bits.  The pair of ones has to be
// in registers: the instruction takes a literal otherwise than it says.
struct Ones {
    uint32_t low = 0x0000bf80u, high = 0xbf800000u;
};
__device__ __forceinline__ float less_low(float x, uint32_t u, const Ones& k) {
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2_t, u), __builtin_bit_cast(bf16x2_t, k.low), x, false);
}
__device__ __forceinline__ float less_high(float x, uint32_t u, const Ones& k) {
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2_t, u), __builtin_bit_cast(bf16x2_t, k.high), x, false);
}

// x as a sum of PLANES bf16 values, each the nearest to what the ones before leave; in fp32 x itself.
template <int PLANES>
__device__ __forceinline__ void split(const float x[8], LFrag<false> f[PLANES], const Ones& k) {
    uint4 u[PLANES];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float a = x[2 * j], b = x[2 * j + 1];
#pragma unroll
        for (int p = 0; p < PLANES; ++p) {
            const uint32_t h = pack2(a, b);
            (&u[p].x)[j] = h;
            if (p + 1 < PLANES) {
                a = less_low(a, h, k);
                b = less_high(b, h, k);
            }
        }
    }
#pragma unroll
    for (int p = 0; p < PLANES; ++p) f[p].v = __builtin_bit_cast(bf16x8_t, u[p]);
}
template <int PLANES>
__device__ __forceinline__ void split(const float x[8], LFrag<true> f[PLANES], const Ones&) {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[0].v[j] = x[j];
}

__device__ __forceinline__ void values(const LFrag<false>& f, float x[8]) {
    const uint4 u = __builtin_bit_cast(uint4, f.v);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        x[2 * j] = low_of((&u.x)[j]);
        x[2 * j + 1] = high_of((&u.x)[j]);
    }
}
__device__ __forceinline__ void values(const LFrag<true>& f, float x[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = f.v[j];
}

// Whether one of a lane's values is not finite: the largest of their bits without sign.
typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
template <int COUNT>
__device__ __forceinline__ bool any_not_finite(const LFrag<false>* f) {
    u16x2_t most = {0, 0};
#pragma unroll
    for (int i = 0; i < COUNT; ++i) {
        const uint4 u = __builtin_bit_cast(uint4, f[i].v);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            most = __builtin_elementwise_max(most, __builtin_bit_cast(u16x2_t, (&u.x)[j] & 0x7fff7fffu));
    }
    return most[0] >= 0x7f80 || most[1] >= 0x7f80;
}
template <int COUNT>
__device__ __forceinline__ bool any_not_finite(const LFrag<true>* f) {
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < COUNT; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) most = max(most, __float_as_uint(f[i].v[j]) & 0x7fffffffu);
    return most >= 0x7f800000u;
}

// Rows of UNITS 16-byte units in LDS.  A unit's place is turned by its row so that neither 16 rows' same unit nor, transposed,
// two units of eight rows meet in a bank.
template <int UNITS, bool F32>
__device__ __forceinline__ int turn(int row) {
    if constexpr (UNITS == 4) return row >> 2 & 3;
    else if constexpr (UNITS == 8) return (row & 6) | (row >> 3 & 1);
    else if constexpr (F32) return row & 15;
    else return (row & 7) << 1 | (row >> 3 & 1);
}
template <int UNITS, bool F32>
__device__ __forceinline__ int place(int row, int unit) {
    return (row * UNITS + (unit ^ turn<UNITS, F32>(row))) * 16;
}

// Four values of one column of a bf16 tile: lane i of 16 gives the place of four values of row i/4, and gets column i.
__device__ __forceinline__ bf16x4_t read_turned(const char* p) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4bf16((__attribute__((address_space(3))) bf16x4_t*)const_cast<char*>(p));
}

// The count of s_waitcnt that lets `vm` requests of memory be under way, and none of LDS.
constexpr int waitcnt(int vm) { return (vm & 15) | (vm >> 4) << 14 | 7 << 4; }

// 16 bytes for each lane of a wave from memory to LDS, where they lie one after another from `to` on.
__device__ __forceinline__ void load_to_lds(const void* from, char* to) {
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) uint32_t*)(uintptr_t)from,
                                     (__attribute__((address_space(3))) uint32_t*)to, 16, 0, 0);
}

template <int DA, int DC, bool F32>
struct LinTile {
    // A wave for 32 columns in 16 bits: what all waves read of `a` and `b` is read half as often as with 16, and each wave has the
    // registers of two (prefill batch 215 against 336 us).  In fp32 products take most of the time, and 16 columns give twice the waves.
    static constexpr int ND = !F32 && DC == 128 ? 2 : 1, WAVES = DC / 16 / ND, THREADS = 64 * WAVES;
    static constexpr int C = F32 ? 32 : 64;      // tokens of a chunk
    static constexpr int ES = F32 ? 4 : 2;
    static constexpr int UA = DA * ES / 16, UC = DC * ES / 16;  // units of a row
    static constexpr int KB = C * UA * 16, VB = C * UC * 16;
    static constexpr int KS = C / 32, RB = C / 16, AS = DA / 32, CT = DA / 16;
    static constexpr int STORES = RB;            // that a wave makes at least at the end of a whole chunk, behind its loads
    // Planes of the state, of the scores and of the weighted values: three bf16 hold all 24 bits of each.
    static constexpr int PL = F32 ? 1 : 3;
    static constexpr int PB = F32 ? 32 * 128 : 5120;  // a plane of scores: rows up to their diagonal's tile
};

// The state's rows are dealt over tiles of 16 so that a lane's rows of two tiles' products are eight side by side: what the next
// product contracts lies in a row of `a` as it is.  Row i of tile ct:
__host__ __device__ constexpr int state_row(int ct, int i) { return 32 * (ct >> 1) + 8 * (i >> 2) + 4 * (ct & 1) + (i & 3); }
// Scores of 16 rows against 32 tokens in a plane: a block of 64 bytes a row, or of 32 where the second 16 tokens lie above the
// diagonal (half_block), which are zeros and not kept: with three whole planes two workgroups would not fit on a CU.
__host__ __device__ constexpr int score_block(int r, int ks) { return r == 0 ? 0 : 1024 * (r + ks) - (r < 3 ? 512 : 0); }
__host__ __device__ constexpr bool half_block(int r, int ks) { return r == 2 * ks; }
static_assert(score_block(1, 0) == score_block(0, 0) + 512 && score_block(2, 0) == score_block(1, 0) + 1024 &&
                  score_block(2, 1) == score_block(2, 0) + 1024 && score_block(3, 0) == score_block(2, 1) + 512 &&
                  score_block(3, 1) == score_block(3, 0) + 1024 && score_block(3, 1) + 1024 == 5120,
              "blocks lie one behind another");
// A wave's columns likewise, for what is stored in a row of the outputs: column i of its tile d.
template <int ND>
__host__ __device__ constexpr int state_col(int wave, int i, int d) {
    return ND == 2 ? 32 * wave + 8 * (i >> 2) + 4 * d + (i & 3) : 16 * wave + i;
}
// Segments' states lie as tiles of 16 rows and 16 columns, in a tile as lanes hold a product: 64 times four rows.  The place of
// four rows from `row` on (a multiple of 4) in column c of a state of DA rows; column tiles go by columns / 16.
template <int DA>
__device__ __forceinline__ int state_at(int row, int c) {
    const int ct = 2 * (row >> 5) + (row >> 2 & 1), grp = row >> 3 & 3;
    return (((c >> 4) * (DA / 16) + ct) * 64 + grp * 16 + (c & 15)) * 4;
}

// Sequences of up to so many segments: a segment's workgroup folds those before it by itself.  Beyond, the last one would read more
// states of 64 KB than a kernel for it costs (8 segments each: prefill of B=4 T=8192 H=16 D=128 216 us against 225 with the kernel, the
// backward call of T=4096 281 against 292; up to 16 by themselves the same, packed 40011 tokens 194 against 198).
constexpr int kOwnFold = 8;

// Two of a lane's values and two of another's as a matrix, transposed: a lane of the upper half gives its first value for the other's
// second.  CTRL: where the other lane is, of four.
template <int CTRL>
__device__ __forceinline__ void across(float& a, float& b, bool upper) {
    const float give = upper ? a : b;
    const float take = __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(give), CTRL, 0xf, 0xf, true));
    if (upper) a = take;
    else b = take;
}

template <int DC, bool F32>
constexpr int kLinThreads = !F32 && DC == 128 ? 256 : 4 * DC;

// A workgroup's way through its segment: a wave has all rows of the state for its columns.  Two workgroups on a CU.
template <int DA, int DC, bool F32, bool ROWS>
__global__ __launch_bounds__((kLinThreads<DC, F32>), (kLinThreads<DC, F32> / 128)) void linattn_chunk_kernel(
    LinOp op0, LinOp op1, LinOp op2, int ops, Segs segs, const float* g) {
    using G = LinTile<DA, DC, F32>;
    constexpr int C = G::C, ND = G::ND, UA = G::UA, UC = G::UC, THREADS = G::THREADS;
    static_assert(THREADS == kLinThreads<DC, F32>, "the launch's");
    __shared__ __align__(16) char ldsK0[G::KB], ldsK1[G::KB];
    __shared__ __align__(16) char ldsV0[G::VB], ldsV1[ROWS ? 16 : G::VB];
    __shared__ __align__(16) char ldsQ[ROWS ? G::KB : 16], ldsP[ROWS ? G::PL * G::PB : 16];
    __shared__ __align__(16) float weights[2][C];  // what a token's product keeps at the chunk's end, whole or the last one
    __shared__ float powers[C + 1];                // of the decay
    __shared__ float lefts[ROWS ? 1 : THREADS];    // of it over so many chunks

    // the operations of a segment and head in workgroups of one XCD, next to one another
    const int64_t id = (int64_t)(blockIdx.x / (8 * ops)) * 8 + blockIdx.x % 8;
    const int which = blockIdx.x / 8 % ops;
    const LinOp op = which == 0 ? op0 : which == 1 ? op1 : op2;
    const int H = segs.H, h = id % H;
    const Where w = where_of<ROWS>(segs, id / H, op.back);
    if (w.count < 0) return;
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, m = lane & 15, grp = lane >> 4;
    const bool last = op.back ? w.j == 0 : w.j + 1 >= w.count;
    if (w.count == 0) {
        if (op.fin) {
            const int64_t at = (w.n * H + h) * (int64_t)DA * DC;
            for (int i = tid; i < DA * DC; i += THREADS) op.fin[at + i] = op.x0 ? op.x0[at + i] : 0.f;
        }
        return;
    }

    const int tokens = (int)(w.end - w.begin), chunks = (tokens + C - 1) / C;
    // Rows of a chunk, in the order of the recurrence, to LDS, 64 units a wave at a time: for a whole chunk, a lane's offset from
    // an address that the wave shares.  Rows behind the last one repeat it and weigh nothing: as many requests for every chunk.
    // A segment's own state may be summed in any order: from where the outputs' pass ends to where it begins, which leaves in the
    // caches what that pass reads first.
    const bool back = op.back == ROWS;
    const int64_t row0 = back ? w.end - 1 : w.begin;
    auto offset_of = [&](auto units) KDA_INLINE {
        constexpr int U = decltype(units)::value;
        const int r = tid / U;
        return (uint32_t)((back ? C - 1 - r : r) * H * U + (tid % U ^ turn<U, F32>(r))) * 16u;
    };
    auto fetch = [&](const void* from, char* to, int c, auto units, uint32_t offset) KDA_INLINE {
        constexpr int U = decltype(units)::value, N = C * U / THREADS, STEP = THREADS / U;
        static_assert(N * THREADS == C * U && (STEP % 16 == 0 || (F32 && STEP == 8)), "a row's turn is that of 16 rows before");
        constexpr int other = STEP == 8 ? 8 : 0;
        if (tokens - c * C >= C) {
            const char* base = static_cast<const char*>(from) +
                               ((back ? row0 - c * C - (C - 1) : row0 + c * C) * H * U + (int64_t)h * U) * 16;
            const int64_t step = (int64_t)(back ? -STEP : STEP) * H * U * 16;
#pragma unroll
            for (int x = 0; x < N; ++x)
                load_to_lds(base + x * step + (x % 2 ? offset ^ (other * 16) : offset), to + (x * G::WAVES + wave) * 1024);
        } else {
            const int top = tokens - c * C - 1;
            const uint4* base = static_cast<const uint4*>(from) + (back ? row0 - c * C - top : row0 + c * C) * H * U + (int64_t)h * U;
            int mine = tid / U;
            __asm__ volatile("" : "+v"(mine));  // made here, for the last chunk alone
#pragma unroll
            for (int x = 0; x < N; ++x) {
                const int r = mine + x * STEP, t = r > top ? top : r;
                load_to_lds(base + (uint32_t)(__mul24(back ? top - t : t, H * U) + (tid % U ^ turn<U, F32>(r))),
                            to + (x * G::WAVES + wave) * 1024);
            }
        }
    };
    using UnitsA = std::integral_constant<int, UA>;
    using UnitsC = std::integral_constant<int, UC>;
    const uint32_t offset_a = offset_of(UnitsA()), offset_c = offset_of(UnitsC());
    fetch(op.b, ldsK0, 0, UnitsA(), offset_a);
    fetch(op.c, ldsV0, 0, UnitsC(), offset_c);
    if constexpr (ROWS) fetch(op.a, ldsQ, 0, UnitsA(), offset_a);

    const double lg = log_decay(g[h]);
    if (tid <= C) powers[tid] = (float)exp(lg * tid);
    if constexpr (!ROWS) lefts[tid] = (float)exp(lg * C * tid);
    const double whole = exp(lg * C);
    const float whole32 = (float)whole, rest = whole > 0 ? (float)((whole - (double)whole32) / whole) : 0.f;

    // The state before the segment: what there is before the sequence, and the segments' before this one, or these folded already.
    // Turned states are summed as they lie, four lanes with each other's columns, and change places in the end.
    f32x4_t S[G::CT][ND];
#pragma unroll
    for (int ct = 0; ct < G::CT; ++ct)
#pragma unroll
        for (int d = 0; d < ND; ++d) S[ct][d] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    if constexpr (ROWS) {
        const int64_t before = op.back ? w.count - 1 - w.j : w.j;
        const bool folded = before > 0 && w.count > kOwnFold;
        auto each = [&](auto f) KDA_INLINE {
#pragma unroll
            for (int ct = 0; ct < G::CT; ++ct)
#pragma unroll
                for (int d = 0; d < ND; ++d) f(S[ct][d], state_row(ct, 4 * grp), state_col<ND>(wave, m, d));
        };
        if (op.x0 && !folded) {
            const float* x = op.x0 + (w.n * H + h) * (int64_t)DA * DC;
            each([&](f32x4_t& to, int r, int c) KDA_INLINE {
#pragma unroll
                for (int j = 0; j < 4; ++j) to[j] = op.turned ? x[((c & ~3) + j) * DA + r + (c & 3)] : x[(r + j) * DC + c];
            });
        }
        const float f = before > 0 ? (float)exp(lg * segs.L) : 0.f;
        for (int64_t i = folded ? before - 1 : 0; i < before; ++i) {
            // segments in the order of the recurrence; the first one of it may be the sequence's last, with fewer tokens
            const float* x = op.states + ((w.base + (op.back ? w.count - 2 - i : i)) * H + h) * (int64_t)DA * DC;
            const float fi = folded ? 0.f : op.back && i == 0 ? (float)exp(lg * w.tail) : f;
            auto add = [&](f32x4_t& to, const float* from) KDA_INLINE {
                const f32x4_t u = *reinterpret_cast<const f32x4_t*>(from);
#pragma unroll
                for (int j = 0; j < 4; ++j) to[j] = folded ? u[j] : fmaf(fi, to[j], u[j]);
            };
            if (op.turned) each([&](f32x4_t& to, int r, int c) KDA_INLINE { add(to, x + state_at<DC>(c & ~3, r + (c & 3))); });
            else each([&](f32x4_t& to, int r, int c) KDA_INLINE { add(to, x + state_at<DA>(r, c)); });
        }
        if (op.turned)
            each([&](f32x4_t& to, int, int) KDA_INLINE {
                float u[4] = {to[0], to[1], to[2], to[3]};
                across<0xb1>(u[0], u[1], m & 1);  // the neighbour's
                across<0xb1>(u[2], u[3], m & 1);
                across<0x4e>(u[0], u[2], m & 2);  // the other pair's
                across<0x4e>(u[1], u[3], m & 2);
                to = f32x4_t{u[0], u[1], u[2], u[3]};
            });
    }

    __syncthreads();
    const float sp = op.su * op.so;
    float owed = 0.f;
    Ones ones;
    if (tid < 2 * C) {
        const int i = tid % C, n = tid < C ? C : tokens - (chunks - 1) * C;
        weights[tid / C][i] = i < n ? op.su * powers[(ROWS ? n - 1 - i : i) + (op.back ? 1 : 0)] : 0.f;
    }

    // Fragments: eight contracted values of row (or column) m.  A lane's first place in a tile; the others are it with some bits
    // of the unit turned over, or whole rows behind it.
    constexpr int RA = UA * 16, RC = UC * 16;
    int at_row, at_turned, at_col;
    if constexpr (F32) {
        at_row = place<UA, true>(m, 2 * grp);
        at_turned = place<UA, true>(4 * grp, 2 * (m >> 2)) + 4 * (m & 3);
        at_col = place<UC, true>(4 * grp, 4 * wave + (m >> 2)) + 4 * (m & 3);
        static_assert(!F32 || ND == 1, "a lane's column");
    } else {
        at_row = place<UA, false>(m, grp);
        at_turned = place<UA, false>(4 * grp + (m >> 2), m & 3);
        at_col = ND == 2 ? place<UC, false>(4 * grp + (m >> 2), 4 * wave + (m & 3))
                         : place<UC, false>(4 * grp + (m >> 2), 2 * wave + (m >> 1 & 1)) + 8 * (m & 1);
    }
    // scores, read by row: a lane's place in a whole block and in a half one; in fp32 one tile of 32
    int at_score = F32 ? place<8, true>(m, 2 * grp) : place<4, false>(m, grp);
    int at_half = F32 ? 0 : 32 * m + 8 * grp;
    int at_power = m, at_far = 16 - 4 * grp;  // of the decay's powers
    auto frag = [&](const char* tile, int r, int s) KDA_INLINE {
        LFrag<F32> f;
        if constexpr (F32) {
            const f32x4_t x = *reinterpret_cast<const f32x4_t*>(tile + (at_row ^ (128 * s)) + 16 * RA * r);
            const f32x4_t y = *reinterpret_cast<const f32x4_t*>(tile + (at_row ^ (128 * s + 16)) + 16 * RA * r);
#pragma unroll
            for (int j = 0; j < 4; ++j) f.v[j] = x[j], f.v[4 + j] = y[j];
        } else {
            f.v = *reinterpret_cast<const bf16x8_t*>(tile + (at_row ^ (64 * s)) + 16 * RA * r);
        }
        return f;
    };
    // the channels of a tile of the state over 32 tokens: group g holds tokens 4g .. +3 and 16 + 4g .. +3
    auto frag_bt = [&](const char* tile, int ct, int ks) KDA_INLINE {
        LFrag<F32> f;
        if constexpr (F32) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                f.v[j] = *reinterpret_cast<const float*>(tile + (at_turned ^ (128 * (ct >> 1) + 16 * ((ct & 1) ^ (j & 3)))) +
                                                         (32 * ks + 16 * (j >> 2) + (j & 3)) * RA);
        } else {
            const char* p = tile + (at_turned ^ (64 * (ct >> 1))) + 8 * (ct & 1) + 32 * ks * RA;
            f.v = __builtin_shufflevector(read_turned(p), read_turned(p + 16 * RA), 0, 1, 2, 3, 4, 5, 6, 7);
        }
        return f;
    };
    auto frag_ct = [&](const char* tile, int d, int ks) KDA_INLINE {
        LFrag<F32> f;
        if constexpr (F32) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                f.v[j] = *reinterpret_cast<const float*>(tile + (at_col ^ (16 * (j & 3))) + (32 * ks + 16 * (j >> 2) + (j & 3)) * RC);
        } else {
            const char* p = tile + at_col + 8 * d + 32 * ks * RC;
            f.v = __builtin_shufflevector(read_turned(p), read_turned(p + 16 * RC), 0, 1, 2, 3, 4, 5, 6, 7);
        }
        return f;
    };

    // One chunk with its keys in K; those of the next one go to Kn, if there is one: only the last chunk may have fewer tokens
    // than C.  Which requests are under way is the same on every path, so that the compiler sees what has been waited for.
    auto chunk = [&](int c, char* K, char* Kn, char* V, char* Vn, auto ends) KDA_INLINE {
        constexpr bool LAST = decltype(ends)::value;
        const int n = LAST ? tokens - c * C : C;
        // the places of a chunk's fragments are made again from these few: kept, they would take most of the registers
        __asm__ volatile("" : "+v"(ones.low), "+v"(ones.high), "+v"(at_row), "+v"(at_turned), "+v"(at_col), "+v"(at_score), "+v"(at_half),
                         "+v"(at_power), "+v"(at_far));
        // Of two workgroups on a CU one goes first in these products and the other in the state's, else the elder in all of them
        // (without: packed 40011 tokens 209 us for 198, prefill batch 225 for 216).
        __builtin_amdgcn_s_setprio(1);
        // The chunk's rows have come.  Requests end in the order in which they were made, and the last ones are the stores of the
        // chunk before: they are not waited for.
        __builtin_amdgcn_s_waitcnt(waitcnt(ROWS ? G::STORES : 0));
        __asm__ volatile("s_barrier" ::: "memory");
        if constexpr (!LAST) {
            fetch(op.b, Kn, c + 1, UnitsA(), offset_a);
            if constexpr (!ROWS) fetch(op.c, Vn, c + 1, UnitsC(), offset_c);
        }
        // The state's decay, in 32 bits: what a power's rounding owes is paid in the next ones, so that thousands of chunks do
        // not add up.  A segment's own state needs none on the way: its tokens are weighed by what is left at the segment's end.
        float dec = powers[n], left = 1.f;
        if constexpr (!ROWS) {
            left = c < THREADS ? lefts[c] : (float)exp(lg * c * C);
        } else if (n == C) {
            dec = fmaf(whole32, owed, whole32);
            owed += rest - (whole32 > 0.f ? (dec - whole32) / whole32 : 0.f);
        }

        LFrag<F32> vf[G::KS * ND];
        auto read_values = [&]() KDA_INLINE {
#pragma unroll
            for (int ks = 0; ks < G::KS; ++ks)
#pragma unroll
                for (int d = 0; d < ND; ++d) vf[ks * ND + d] = frag_ct(V, d, ks);
        };
        int bad[ND];  // a column's first token whose value is not finite
        bool marked = false;
        if constexpr (ROWS) {
            // The scores are the first waves' (every SIMD has one of them), with the products of the state where all waves are.
            constexpr bool TOGETHER = G::WAVES == G::RB;
            f32x4_t O[G::RB][ND], P[G::RB];
            auto scores = [&]() KDA_INLINE {
                // Of row 16r + m against token 16i + 4 grp + j with i = wave: a^(16(r-i)-4 grp-j) a^m above the diagonal's tile; in
                // it a^(m-4 grp-j) and nothing above the diagonal; rows of the products' 32 tokens behind it: zeros.
                float part = sp * powers[at_power];
                const float step16 = powers[16];
#pragma unroll
                for (int r = 0; r < G::RB; ++r) {
                    if (wave > (F32 ? r | 1 : r)) continue;
                    float x[4];
                    if (wave == r) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int apart = at_power - 16 + at_far - j;
                            x[j] = apart >= 0 ? P[r][j] * (sp * powers[apart >= 0 ? apart : 0]) : 0.f;
                        }
                    } else if (wave < r) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) x[j] = P[r][j] * (powers[at_far - j] * part);
                        part *= step16;
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; ++j) x[j] = 0.f;
                    }
                    if constexpr (F32) {
                        *reinterpret_cast<f32x4_t*>(ldsP + (at_score ^ (16 * wave)) + 2048 * r) = f32x4_t{x[0], x[1], x[2], x[3]};
                    } else {
                        char* to = ldsP + (wave == r && r % 2 == 0 ? score_block(r, r / 2) + at_half
                                                                   : score_block(r, wave >> 1) + at_score + 8 * (wave & 1));
#pragma unroll
                        for (int p = 0; p < G::PL; ++p) {
                            const uint32_t h0 = pack2(x[0], x[1]), h1 = pack2(x[2], x[3]);
                            *reinterpret_cast<uint2*>(to + p * G::PB) = make_uint2(h0, h1);
                            if (p + 1 < G::PL) {
                                x[0] = less_low(x[0], h0, ones), x[1] = less_high(x[1], h0, ones);
                                x[2] = less_low(x[2], h1, ones), x[3] = less_high(x[3], h1, ones);
                            }
                        }
                    }
                }
            };
#pragma unroll
            for (int r = 0; r < G::RB; ++r) {
                P[r] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int d = 0; d < ND; ++d) O[r][d] = f32x4_t{0.f, 0.f, 0.f, 0.f};
            }
            if (!TOGETHER && wave < G::RB) {
#pragma unroll
                for (int s = 0; s < G::AS; ++s) {
                    const LFrag<F32> kf = frag(K, wave, s);
#pragma unroll
                    for (int r = 0; r < G::RB; ++r) P[r] = mma(kf, frag(ldsQ, r, s), P[r]);
                }
                scores();
            }
#pragma unroll
            for (int s = 0; s < G::AS; ++s) {
                LFrag<F32> qf[G::RB], kf;
#pragma unroll
                for (int r = 0; r < G::RB; ++r) qf[r] = frag(ldsQ, r, s);
                if constexpr (TOGETHER) kf = frag(K, wave, s);
#pragma unroll
                for (int d = 0; d < ND; ++d) {
                    LFrag<F32> st[G::PL];
                    float x[8];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        x[j] = S[2 * s][d][j];
                        x[4 + j] = S[2 * s + 1][d][j];
                        S[2 * s][d][j] *= dec;
                        S[2 * s + 1][d][j] *= dec;
                    }
                    split<G::PL>(x, st, ones);
#pragma unroll
                    for (int p = 0; p < G::PL; ++p)
#pragma unroll
                        for (int r = 0; r < G::RB; ++r) O[r][d] = mma(st[p], qf[r], O[r][d]);
                }
                if constexpr (TOGETHER)
#pragma unroll
                    for (int r = 0; r < G::RB; ++r) P[r] = mma(kf, qf[r], P[r]);
            }
            read_values();
            if constexpr (TOGETHER) scores();
#pragma unroll
            for (int r = 0; r < G::RB; ++r) {
                const float into = op.so * powers[16 * r + at_power + (op.back ? 0 : 1)];
#pragma unroll
                for (int d = 0; d < ND; ++d)
#pragma unroll
                    for (int j = 0; j < 4; ++j) O[r][d][j] *= into;
            }
            lds_barrier();
            if constexpr (!LAST) {
                fetch(op.a, ldsQ, c + 1, UnitsA(), offset_a);
                fetch(op.c, Vn, c + 1, UnitsC(), offset_c);
            }

            LFrag<F32> pf[G::KS][G::PL][G::RB];
#pragma unroll
            for (int ks = 0; ks < G::KS; ++ks)
#pragma unroll
                for (int p = 0; p < G::PL; ++p)
#pragma unroll
                    for (int r = 2 * ks; r < G::RB; ++r) {
                        LFrag<F32>& f = pf[ks][p][r];
                        if constexpr (F32) {
                            const f32x4_t x = *reinterpret_cast<const f32x4_t*>(ldsP + at_score + 2048 * r);
                            const f32x4_t y = *reinterpret_cast<const f32x4_t*>(ldsP + (at_score ^ 16) + 2048 * r);
#pragma unroll
                            for (int j = 0; j < 4; ++j) f.v[j] = x[j], f.v[4 + j] = y[j];
                        } else {
                            const char* from = ldsP + p * G::PB + score_block(r, ks);
                            if (half_block(r, ks))
                                f.v = __builtin_shufflevector(*reinterpret_cast<const bf16x4_t*>(from + at_half), bf16x4_t{},
                                                              0, 1, 2, 3, 4, 5, 6, 7);
                            else f.v = *reinterpret_cast<const bf16x8_t*>(from + at_score);
                        }
                    }
            // A value that is not finite must not meet the zeros of earlier rows: such values are left out of the products, and
            // their column is made NaN from their token on, here and in the state.
            marked = __ballot(any_not_finite<G::KS * ND>(vf)) != 0;
            if (marked) {
#pragma unroll
                for (int d = 0; d < ND; ++d) {
                    bad[d] = C;
#pragma unroll
                    for (int ks = G::KS - 1; ks >= 0; --ks)
#pragma unroll
                        for (int j = 7; j >= 0; --j)
                            if (!(fabsf((float)vf[ks * ND + d].v[j]) < __builtin_inff())) {
                                bad[d] = 32 * ks + 16 * (j >> 2) + 4 * grp + (j & 3);
                                vf[ks * ND + d].v[j] = 0.f;
                            }
                    bad[d] = min(bad[d], __shfl_xor(bad[d], 16));
                    bad[d] = min(bad[d], __shfl_xor(bad[d], 32));
                }
            }
#pragma unroll
            for (int ks = 0; ks < G::KS; ++ks)
#pragma unroll
                for (int p = 0; p < G::PL; ++p)
#pragma unroll
                    for (int d = 0; d < ND; ++d)
#pragma unroll
                        for (int r = 2 * ks; r < G::RB; ++r) O[r][d] = mma(vf[ks * ND + d], pf[ks][p][r], O[r][d]);
            if (marked) {
#pragma unroll
                for (int d = 0; d < ND; ++d)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int from = __shfl(bad[d], 4 * grp + j);
#pragma unroll
                        for (int r = 0; r < G::RB; ++r)
                            if (16 * r + m >= from) O[r][d][j] = __builtin_nanf("");
                    }
            }
            // a lane's first row of the chunk; the others are 16 rows apart
            char* to = static_cast<char*>(op.out) + ((row0 + (op.back ? -c * C : c * C)) * H + h) * (int64_t)(DC * G::ES);
            const int pitch = (op.back ? -H : H) * DC * G::ES, mine = m * pitch + state_col<ND>(wave, 4 * grp, 0) * G::ES;
            __asm__ volatile("" ::: "memory");  // behind the chunk's loads, all of them
            static_assert(G::STORES == G::RB && 4 * ND * G::ES <= 16, "one store for each of a lane's rows");
#pragma unroll
            for (int r = 0; r < G::RB; ++r)
                if (!LAST || 16 * r + m < n) {
                    char* p = to + (int64_t)(16 * r * pitch) + mine;
                    if constexpr (F32) *reinterpret_cast<f32x4_t*>(p) = O[r][0];
                    else if constexpr (ND == 2)
                        *reinterpret_cast<uint4*>(p) = make_uint4(pack2(O[r][0][0], O[r][0][1]), pack2(O[r][0][2], O[r][0][3]),
                                                                  pack2(O[r][1][0], O[r][1][1]), pack2(O[r][1][2], O[r][1][3]));
                    else *reinterpret_cast<uint2*>(p) = make_uint2(pack2(O[r][0][0], O[r][0][1]), pack2(O[r][0][2], O[r][0][3]));
                }
            __asm__ volatile("" ::: "memory");
        } else {
            read_values();
        }

        __builtin_amdgcn_s_setprio(0);
#pragma unroll
        for (int ks = 0; ks < G::KS; ++ks) {
            f32x4_t w0 = *reinterpret_cast<const f32x4_t*>(weights[LAST] + 32 * ks + 4 * grp);
            f32x4_t w1 = *reinterpret_cast<const f32x4_t*>(weights[LAST] + 32 * ks + 16 + 4 * grp);
            if constexpr (!ROWS)
#pragma unroll
                for (int j = 0; j < 4; ++j) w0[j] *= left, w1[j] *= left;
            constexpr int TOGETHER = F32 ? 2 : 4;  // tiles of the state: as many as the registers hold
            LFrag<F32> vb[ND][G::PL], kt[TOGETHER];
#pragma unroll
            for (int ct = 0; ct < TOGETHER; ++ct) kt[ct] = frag_bt(K, ct, ks);
#pragma unroll
            for (int d = 0; d < ND; ++d) {
                float x[8];
                values(vf[ks * ND + d], x);
#pragma unroll
                for (int j = 0; j < 4; ++j) x[j] *= w0[j], x[4 + j] *= w1[j];
                split<G::PL>(x, vb[d], ones);
            }
#pragma unroll
            for (int first = 0; first < G::CT; first += TOGETHER) {
                if (first > 0)
#pragma unroll
                    for (int ct = 0; ct < TOGETHER; ++ct) kt[ct] = frag_bt(K, first + ct, ks);
#pragma unroll
                for (int p = 0; p < G::PL; ++p)
#pragma unroll
                    for (int ct = 0; ct < TOGETHER; ++ct)
#pragma unroll
                        for (int d = 0; d < ND; ++d) S[first + ct][d] = mma(kt[ct], vb[d][p], S[first + ct][d]);
            }
        }
        if (ROWS && marked) {
#pragma unroll
            for (int d = 0; d < ND; ++d)
                if (bad[d] < n)
#pragma unroll
                    for (int ct = 0; ct < G::CT; ++ct)
#pragma unroll
                        for (int j = 0; j < 4; ++j) S[ct][d][j] = __builtin_nanf("");
        }
    };

    char* const ldsVn = ROWS ? ldsV0 : ldsV1;
    __builtin_amdgcn_s_waitcnt(waitcnt(0));
    int c = 0;
    while (true) {
        if (c + 1 >= chunks) break;
        chunk(c++, ldsK0, ldsK1, ldsV0, ldsVn, std::false_type());
        if (c + 1 >= chunks) break;
        chunk(c++, ldsK1, ldsK0, ldsVn, ldsV0, std::false_type());
    }
    chunk(c, c % 2 ? ldsK1 : ldsK0, nullptr, c % 2 ? ldsVn : ldsV0, nullptr, std::true_type());

    if constexpr (ROWS) {
        if (last && op.fin) {
            float* to = op.fin + (w.n * H + h) * (int64_t)DA * DC;
#pragma unroll
            for (int ct = 0; ct < G::CT; ++ct)
#pragma unroll
                for (int d = 0; d < ND; ++d)
#pragma unroll
                    for (int j = 0; j < 4; ++j) to[state_row(ct, 4 * grp + j) * DC + state_col<ND>(wave, m, d)] = S[ct][d][j];
        }
    } else {
        float* to = static_cast<float*>(op.out) + ((w.base + w.j - (op.back ? 1 : 0)) * H + h) * (int64_t)DA * DC;
#pragma unroll
        for (int ct = 0; ct < G::CT; ++ct)
#pragma unroll
            for (int d = 0; d < ND; ++d)
                *reinterpret_cast<f32x4_t*>(to + state_at<DA>(state_row(ct, 4 * grp), state_col<ND>(wave, m, d))) = S[ct][d];
    }
}

// The states behind (with `back` before) each segment from the segments' own ones, in place, for sequences of many segments:
// X_j = a^length X_(j-1) + U_j.  A thread holds four values of a head's state through all segments.  A packed sequence of more
// than kOwnFold segments holds a token whose number is a multiple of kOwnFold L: its first such token stands for it in the grid.
struct FoldOp {
    float* states;
    const float* x0;
    bool back;
};
template <int DA>
__global__ __launch_bounds__(kThreads) void linattn_fold_kernel(FoldOp op0, FoldOp op1, Segs segs, const float* g, int DC) {
    const FoldOp op = blockIdx.y ? op1 : op0;
    const int size = DA * DC, per = size / (4 * kThreads);
    const int64_t sh = blockIdx.x / per, token = sh / segs.H * kOwnFold * segs.L;
    const int h = sh % segs.H, at = (int)(blockIdx.x % per) * 4 * kThreads + 4 * threadIdx.x;
    const Where w = sequence(segs, segs.cu ? last_below(segs, [&](int64_t begin, int64_t) { return begin <= token; }) : sh / segs.H);
    if (w.count <= kOwnFold || (segs.cu && (token < w.begin || token - w.begin >= kOwnFold * segs.L))) return;
    const double lg = log_decay(g[h]);
    const float whole = (float)exp(lg * segs.L), tail = (float)exp(lg * w.tail);
    f32x4_t x = {0.f, 0.f, 0.f, 0.f};
    if (op.x0) {
        const int lane = at / 4 % 64, ct = at / 256 % (DA / 16), c = at / (256 * (DA / 16)) * 16 + lane % 16;
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = op.x0[(w.n * segs.H + h) * size + state_row(ct, lane / 16 * 4 + j) * DC + c];
    }
    const int64_t step = (int64_t)segs.H * size;
    f32x4_t* p = reinterpret_cast<f32x4_t*>(op.states + (w.base * segs.H + h) * (int64_t)size + at);
    constexpr int AHEAD = 8;
    for (int64_t j0 = 0; j0 < w.count - 1; j0 += AHEAD) {
        f32x4_t u[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int64_t j = j0 + i < w.count - 1 ? j0 + i : w.count - 2;
            u[i] = p[(op.back ? w.count - 2 - j : j) * (step / 4)];
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int64_t j = j0 + i;
            if (j >= w.count - 1) break;
            const float f = op.back && j == 0 ? tail : whole;
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = fmaf(f, x[e], u[i][e]);
            p[(op.back ? w.count - 2 - j : j) * (step / 4)] = x;
        }
    }
}

// ------------------------------------------------------------------------------------------------ one token

// A workgroup holds one head's state, four columns of RPT rows a thread, and reads and writes it once, past the caches: 256 x 32
// states of 128 x 128 in 179 us, 6.0 TB/s (a copy of as many bytes takes 174).
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

// Tokens of a segment, about `many`.  A segment's state is written and read, several times its size, which 256 tokens outweigh; fewer
// only where every CU has no segment otherwise.
int64_t segment_tokens(int64_t many, int64_t total, int H) {
    auto whole = [](int64_t x) { return (x + 63) / 64 * 64; };
    const int64_t one = whole((total * H + 255) / 256);
    many = whole(many);
    return many > 256 ? many : one < 64 ? 64 : one < 256 ? one : 256;
}
// Packed sequences end anywhere, so that half of the segments are shorter: with 768 of them the 512 places, two on a CU, even out
// (40011 tokens of 16 heads in 32 sequences 198 us, with 512 206; their backward call 480 and 474).
int64_t packed_segment(const LinArgs& a) { return segment_tokens((a.total * a.H + 767) / 768, a.total, a.H); }
// Equal lengths are cut in equal parts, as many as there are places for, and not at all where that is one part: the first pass costs
// more than empty places.  Against segments as of packed sequences: B=4 T=8192 H=16 D=128 bf16 218 us for 264, B=30 T=1500 222 for 296
// (fp32 537 for 823), B=10 T=3000 185 for 220.
int64_t equal_segment(const LinArgs& a) {
    const int64_t parts = a.N * a.H >= 512 ? 1 : 512 / (a.N * a.H);
    return segment_tokens((a.T_fixed + parts - 1) / parts, a.total, a.H);
}

Segs segs_of(const LinArgs& a) {
    Segs s{a.cu, a.T_fixed, a.N, a.total, a.cu ? packed_segment(a) : equal_segment(a), 1, a.H};
    if (!a.cu && a.T_fixed > s.L) s.per_seq = (a.T_fixed + s.L - 1) / s.L;
    return s;
}

int64_t slots_of(const Segs& s, bool rows) {
    return s.cu ? s.total / s.L + (rows ? s.N : 0) : s.N * (s.per_seq - (rows ? 0 : 1));
}

// Whether a sequence may have more than one segment.
bool is_split(const Segs& s) { return s.cu ? s.total > s.L : s.per_seq > 1; }

using I64 = std::integral_constant<int, 64>;
using I128 = std::integral_constant<int, 128>;

template <bool ROWS>
void chunks(const LinArgs& a, const Segs& s, std::initializer_list<LinOp> ops, int DA, int DC, hipStream_t st) {
    LinOp op[3] = {};
    int count = 0;
    for (const LinOp& o : ops) op[count++] = o;
    const int64_t each = (slots_of(s, ROWS) * a.H + 7) / 8 * 8;  // workgroups behind the last segment find none
    auto run = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3((unsigned)(each * count)), dim3(a.f32 || DC == 64 ? 4 * DC : 256), 0, st, op[0], op[1],
                           op[2], count, s, a.g);
    };
    auto types = [&](auto da, auto dc) {
        constexpr int A = decltype(da)::value, B = decltype(dc)::value;
        a.f32 ? run(linattn_chunk_kernel<A, B, true, ROWS>) : run(linattn_chunk_kernel<A, B, false, ROWS>);
    };
    if (DA == 64) DC == 64 ? types(I64(), I64()) : types(I64(), I128());
    else DC == 64 ? types(I128(), I64()) : types(I128(), I128());
}

// Workgroups of the fold for one operation; 0: no sequence can have so many segments.
int64_t fold_groups(const LinArgs& a, const Segs& s) {
    if ((s.cu ? (s.total + s.L - 1) / s.L : s.per_seq) <= kOwnFold) return 0;
    return (s.cu ? (s.total - 1) / (kOwnFold * s.L) + 1 : s.N) * a.H * (a.Dk * a.Dv / (4 * kThreads));
}

void fold(const LinArgs& a, const Segs& s, FoldOp one, const FoldOp* two, hipStream_t st) {
    const int64_t groups = fold_groups(a, s);
    if (groups == 0) return;
    const dim3 grid((unsigned)groups, two ? 2 : 1);
    auto run = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, st, one, two ? *two : one, s, a.g, a.Dv); };
    a.Dk == 64 ? run(linattn_fold_kernel<64>) : run(linattn_fold_kernel<128>);
}

}  // namespace

// For either way of giving the sequences: packed ones have the shorter segments, since a part of an equal length has a 512th of
// all tokens at least.
int64_t linattn_workspace_bytes(const LinArgs& a, bool backward) {
    const int64_t L = packed_segment(a);
    if (a.total <= L) return 0;
    return a.total / L * a.H * a.Dk * (int64_t)a.Dv * 4 * (backward ? 2 : 1);
}

// Of the outputs' launch, or of the fold's where that has more: 16 workgroups for 8 segments of 128 x 128, twice in a backward call
// (forward, a sequence of 768 segments and one head: 1536 against 769).
int64_t linattn_threads(const LinArgs& a, bool backward) {
    const Segs s = segs_of(a);
    const int64_t D = a.Dk > a.Dv ? a.Dk : a.Dv, rows = (slots_of(s, true) * a.H + 8) * (backward ? 3 : 1) * (a.f32 ? 4 * D : 256);
    const int64_t folds = fold_groups(a, s) * kThreads * (backward ? 2 : 1);
    return rows > folds ? rows : folds;
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
    float* grads = states + s.total / s.L * a.H * a.Dk * a.Dv;
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
