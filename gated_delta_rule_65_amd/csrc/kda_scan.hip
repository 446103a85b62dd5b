// Gated scan over channels: h_t = a_t h_{t-1} + w_t x_t, its gradients and its single-token step
// (mathematics and layouts: include/kda_layer.h).
//
// A step of the scan is the map s -> A s + b of the state; steps compose to (A2 A1, A2 b1 + b2), so a run of tokens is
// one such pair per channel.  Time is cut into segments of 64 tokens, a segment and 64 * CPL channels to a workgroup:
//   1. each wave takes 8 of the tokens, reads its rows (all loads in flight at once), and folds them to its pair;
//   2. the waves' pairs meet in LDS and give the segment's pair, which is published in the workspace;
//   3. the state before the segment is folded from what the earlier segments of the sequence published: the pairs of
//      the up to 7 segments of its own group of 8, of the up to 7 whole groups before in its own block of 64, and
//      the state at the end of the block before.  The last segment of a group publishes the group's pair, the
//      last of a block the state behind it;
//   4. each wave runs its tokens again from its own state, with the gates and inputs still in registers.
// Every input is read once and every output written once; the pairs add 8 bytes for 64 tokens of a channel, and
// are read about 8 times, from the cache behind the L2s.  What waits is a chain of one hop for each 4096 tokens.
// All sums are in a fixed order, so results do not depend on the timing.
//
// Why every wait ends: a workgroup takes its place in the order of work from a counter when it starts, and only waits for
// segments whose places were taken earlier, by workgroups that are therefore running or done.  The one
// with the lowest place among those not done waits for nobody.
//
// The backward pass is the same scan with time reversed, of e_t = a_t (dy_t + e_{t+1}).
#include <type_traits>

#include "kda_ckpt8.h"
#include "kda_layer_launch.h"

namespace kda {

namespace {

typedef unsigned long long u64;

constexpr int kWaves = 8, kRows = 8, kThreads = kWaves * 64;
static_assert(kWaves * kRows == kScanSeg, "a wave's rows");
constexpr int kGroup = 8, kBlock = 64;  // segments of a group and of a block

// ---------------------------------------------------------------------------- rows in registers
// CPL consecutive elements of a row as they come from memory.
template <bool F32, int CPL>
struct Raw {
    static constexpr int WORDS = F32 ? CPL : (CPL + 1) / 2;
    uint32_t w[WORDS];
};
// Rows are read once and written once: past the caches.  (B = 4, T = 8192, D = 2048 in bf16, rows moved in this pattern and
// nothing else: 90 us, and 84 non-temporal.)
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
template <int WORDS>
__device__ __forceinline__ void load_words(const void* p, uint32_t* w) {
    if constexpr (WORDS == 4) {
        const u32x4 v = __builtin_nontemporal_load(static_cast<const u32x4*>(p));
        w[0] = v[0]; w[1] = v[1]; w[2] = v[2]; w[3] = v[3];
    } else if constexpr (WORDS == 2) {
        const u32x2 v = __builtin_nontemporal_load(static_cast<const u32x2*>(p));
        w[0] = v[0]; w[1] = v[1];
    } else {
        w[0] = __builtin_nontemporal_load(static_cast<const uint32_t*>(p));
    }
}
template <bool F32, int CPL>
__device__ __forceinline__ Raw<F32, CPL> load_raw(const void* base, int64_t i) {
    Raw<F32, CPL> r;
    if constexpr (F32) load_words<CPL>(static_cast<const float*>(base) + i, r.w);
    else if constexpr (CPL == 1) r.w[0] = static_cast<const uint16_t*>(base)[i];
    else load_words<CPL / 2>(static_cast<const uint16_t*>(base) + i, r.w);
    return r;
}
template <bool F32, int CPL>
__device__ __forceinline__ float raw_get(const Raw<F32, CPL>& r, int k, uint32_t shift = 16, uint32_t mask = 0xffff0000u) {
    if constexpr (F32) return __uint_as_float(r.w[k]);
    else return __uint_as_float(k % 2 ? r.w[k / 2] & mask : r.w[k / 2] << shift);
}
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
    typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
    const bf2 v = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, v);
}
template <bool F32, int CPL>
__device__ __forceinline__ void store_row(void* base, int64_t i, const float v[CPL]) {
    if constexpr (F32) {
        float* p = static_cast<float*>(base) + i;
        if constexpr (CPL == 4) __builtin_nontemporal_store(f32x4{v[0], v[1], v[2], v[3]}, reinterpret_cast<f32x4*>(p));
        else *p = v[0];
    } else {
        uint16_t* p = static_cast<uint16_t*>(base) + i;
        if constexpr (CPL == 4)
            __builtin_nontemporal_store(u32x2{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])}, reinterpret_cast<u32x2*>(p));
        else *reinterpret_cast<__bf16*>(p) = (__bf16)v[0];
    }
}

// ---------------------------------------------------------------------------- gates
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
// The constants of one run over a wave's rows.  A later run takes the same ones through again(), where the compiler cannot
// see that they are the same: it would keep every decay and input of the first run in registers otherwise.
struct Run {
    uint32_t shift = 16, mask = 0xffff0000u;
    float low = -5.f, edge = kLogitEdge, log2e = 1.4426950408889634f;
};
__device__ __forceinline__ Run again() {
    Run r;
    __asm__ volatile("" : "+s"(r.shift), "+s"(r.mask), "+s"(r.low), "+s"(r.edge), "+s"(r.log2e));
    return r;
}
template <bool LOGIT, bool REST>
__device__ __forceinline__ Gate gate_of(float g, const Run& run) {
    if constexpr (LOGIT) {
        const float t = __builtin_amdgcn_exp2f(__builtin_elementwise_minimum(g, run.edge) * run.log2e);
        const float a = __builtin_amdgcn_rcpf(1.f + t);
        return {a, t * a};
    }
    const float l = __builtin_elementwise_minimum(__builtin_elementwise_maximum(g, run.low), 0.f);
    const float a = __builtin_amdgcn_exp2f(l * run.log2e);
    return {a, REST ? one_minus_exp(l, a) : 0.f};
}
// The derivative of l by g: 1 inside the clamp (ends included) and 0 outside; with logits -sigmoid(g) = -(1 - a).
template <bool LOGIT>
__device__ __forceinline__ float gate_slope(float g, float rest) {
    if constexpr (LOGIT) return g > kLogitEdge ? 0.f : -rest;
    return (g < -5.f || g > 0.f) ? 0.f : 1.f;
}

// ---------------------------------------------------------------------------- places in the order of work
struct ScanPlan {
    uint32_t cols;      // groups of 64 * CPL channels
    uint32_t chains;    // sequences with segments of their own; 1 for packed rows
    uint32_t per_chain; // segments of a chain
    uint32_t* counter;  // nullptr: no chain is longer than a segment
    u64 *pairs, *groups, *states;
};

struct Tile {
    int64_t chain, at;   // segment `at` of its chain, in the direction of the scan
    int64_t id;          // index of the segment
    int64_t row0;        // its first row, and how many rows it has
    int rows;
    int64_t col;
};

template <bool FLAT, bool BACK>
__device__ __forceinline__ Tile tile_of(const ScanArgs& a, const ScanPlan& p, uint32_t place, int64_t total) {
    Tile t;
    t.col = place % p.cols;
    const uint32_t s = place / p.cols;
    t.chain = FLAT ? 0 : s % p.chains;
    t.at = FLAT ? s : s / p.chains;
    const int64_t q = BACK ? (int64_t)p.per_chain - 1 - t.at : t.at;
    t.id = t.chain * p.per_chain + q;
    t.row0 = t.chain * a.T_fixed + q * kScanSeg;
    const int64_t end = FLAT ? total : (t.chain + 1) * a.T_fixed;
    const int64_t left = end - t.row0;
    t.rows = left < 0 ? 0 : left < kScanSeg ? (int)left : kScanSeg;
    return t;
}

// The place of this workgroup, the same in all its threads.
__device__ __forceinline__ uint32_t take_place(uint32_t* counter, uint32_t* shared) {
    if (!counter) return blockIdx.x;
    if (threadIdx.x == 0)
        *shared = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    return (uint32_t)__builtin_amdgcn_readfirstlane((int)*shared);
}

// An offset of packed rows, read through the scalar cache (the kernels do not write them).
__device__ __forceinline__ int64_t offset_of(const int32_t* cu, int64_t n) {
    typedef const __attribute__((address_space(4))) int32_t* scalar;
    return ((scalar)cu)[__builtin_amdgcn_readfirstlane((int)n)];
}
// The sequence that holds row r of packed rows: the last n with cu[n] <= r.
__device__ __forceinline__ int64_t seq_of(const int32_t* cu, int64_t N, int64_t r) {
    int lo = 0, hi = (int)N - 1;
    while (lo < hi) {
        const int mid = lo + (hi - lo + 1) / 2;
        if (offset_of(cu, mid) <= r) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// ---------------------------------------------------------------------------- published words
// A pair (A, b) in one 64-bit word that is valid as a whole: kEmpty until it is written, so that neither a flag nor
// a fence is needed.  A word that happens to look empty is written with another NaN.  A = -0 says that a sequence
// begins inside: whatever the state before is, even infinite, it has no part in what follows.
constexpr u64 kEmpty = ~0ull;
constexpr uint32_t kBegins = 0x80000000u;

struct Pair {
    float A, b;
};
__device__ __forceinline__ Pair then(Pair first, Pair second) {
    if (__float_as_uint(second.A) == kBegins) return second;
    const bool begun = __float_as_uint(first.A) == kBegins;
    return {begun ? first.A : first.A * second.A, fmaf(second.A, first.b, second.b)};
}
__device__ __forceinline__ float apply(Pair p, float s) {
    return __float_as_uint(p.A) == kBegins ? p.b : fmaf(p.A, s, p.b);
}
__device__ __forceinline__ void publish(u64* at, Pair p) {
    u64 w = (u64)__float_as_uint(p.A) << 32 | __float_as_uint(p.b);
    if (w == kEmpty) w ^= 1;
    __hip_atomic_store(at, w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ u64 peek(const u64* at) {
    return __hip_atomic_load(const_cast<u64*>(at), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// Waits for a word that an earlier place publishes.  The bound (some seconds) is never reached by the argument above; behind
// it the word reads as NaN, so that a broken promise shows and does not hang.
__device__ __forceinline__ Pair await(const u64* at, u64 w) {
    for (int i = 0; w == kEmpty && i < (1 << 22); ++i) {
        __builtin_amdgcn_s_sleep(1);
        w = peek(at);
    }
    return {__uint_as_float((uint32_t)(w >> 32)), __uint_as_float((uint32_t)w)};
}

// The pair of the segments of t.at's group before it, for channel c; the group's last segment publishes the group's.
__device__ __forceinline__ Pair group_before(const ScanArgs& a, const ScanPlan& p, const Tile& t, int64_t c, Pair own) {
    const int n = (int)(t.at % kGroup);
    const u64* at = p.pairs + (t.chain * p.per_chain + t.at - n) * a.D + c;
    u64 w[kGroup - 1];
#pragma unroll
    for (int i = 0; i < kGroup - 1; ++i) w[i] = i < n ? peek(at + i * a.D) : 0;
    Pair group = {1.f, 0.f};
#pragma unroll
    for (int i = 0; i < kGroup - 1; ++i)
        if (i < n) group = then(group, await(at + i * a.D, w[i]));
    if (n == kGroup - 1) {
        const int64_t groups = (p.per_chain + kGroup - 1) / kGroup;
        publish(p.groups + (t.chain * groups + t.at / kGroup) * a.D + c, then(group, own));
    }
    return group;
}

// The state of channel c before t.at's group, from the groups of its block and the state before the block; `reach` segments
// back at most have a part in it (packed rows: those from the sequence's first on).
__device__ __forceinline__ float state_before_group(const ScanArgs& a, const ScanPlan& p, const Tile& t, int64_t c,
                                                    int64_t reach) {
    constexpr int most = kBlock / kGroup - 1;
    const int64_t groups = (p.per_chain + kGroup - 1) / kGroup, blocks = (p.per_chain + kBlock - 1) / kBlock;
    const int n = (int)(t.at / kGroup % (most + 1));
    const bool further = t.at >= kBlock && t.at - reach < t.at / kBlock * kBlock;
    const u64* at = p.groups + (t.chain * groups + t.at / kGroup - n) * a.D + c;
    const u64* state = p.states + (t.chain * blocks + t.at / kBlock - 1) * a.D + c;
    u64 w[most], ws = 0;
    if (further) ws = peek(state);
#pragma unroll
    for (int i = 0; i < most; ++i) w[i] = i < n ? peek(at + i * a.D) : 0;
    Pair before = {1.f, 0.f};
#pragma unroll
    for (int i = 0; i < most; ++i)
        if (i < n) before = then(before, await(at + i * a.D, w[i]));
    return apply(before, further ? await(state, ws).b : 0.f);
}

// What the waves of a workgroup tell one another of its channels: their pairs, then the states before them, and
// the state before the segment's group.
template <int CPL>
struct Exchange {
    float A[kWaves][64 * CPL], b[kWaves][64 * CPL], before[64 * CPL];
};
// Half of what a lane keeps of its rows in the backward pass, so that two workgroups' registers fit a CU.
constexpr int kKept = kRows / 2;
template <int CPL, bool USED>
struct Kept {
    float rows[USED ? kKept : 1][USED ? kWaves : 1][USED ? 64 * CPL : 1];
};
template <int CPL>
__device__ __forceinline__ void put(float* row, const float v[CPL]) {
    if constexpr (CPL % 4 == 0) {
#pragma unroll
        for (int k = 0; k < CPL; k += 4)
            *reinterpret_cast<float4*>(row + k) = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
    } else {
#pragma unroll
        for (int k = 0; k < CPL; ++k) row[k] = v[k];
    }
}
template <int CPL>
__device__ __forceinline__ void take(const float* row, float v[CPL]) {
    if constexpr (CPL % 4 == 0) {
#pragma unroll
        for (int k = 0; k < CPL; k += 4) {
            const float4 u = *reinterpret_cast<const float4*>(row + k);
            v[k] = u.x; v[k + 1] = u.y; v[k + 2] = u.z; v[k + 3] = u.w;
        }
    } else {
#pragma unroll
        for (int k = 0; k < CPL; ++k) v[k] = row[k];
    }
}

// From the waves' pairs (taken in the scan's direction) to the state before each wave, in x.b.  `start`: the state before the
// chain's first segment, where reach < 0 names it.  A thread of the first part has a channel of its own and folds
// its group, one of the second part folds what lies before the group at the same time.
template <bool BACK, int CPL>
__device__ __forceinline__ void join_waves(const ScanArgs& a, const ScanPlan& p, const Tile& t, Exchange<CPL>& x,
                                           const float* start, int64_t reach, float* carry) {
    constexpr int C = 64 * CPL;
    static_assert(2 * C <= kThreads, "two threads a channel");
    const int part = __builtin_amdgcn_readfirstlane(threadIdx.x / C), ch = threadIdx.x % C;
    const int64_t c = t.col * C + ch;
    const bool mine = c < a.D;
    Pair own = {1.f, 0.f}, group = {1.f, 0.f};
    if (part == 0 && mine) {
#pragma unroll
        for (int i = 0; i < kWaves; ++i) {
            const int w = BACK ? kWaves - 1 - i : i;
            own = then(own, Pair{x.A[w][ch], x.b[w][ch]});
        }
        // before the chain's first segment the state is known: its pair holds for any
        if (reach < 0) own = {__uint_as_float(kBegins), apply(own, start ? start[c] : 0.f)};
        if (p.counter) {
            publish(p.pairs + (t.chain * p.per_chain + t.at) * a.D + c, own);
            group = group_before(a, p, t, c, own);
        }
    }
    if (part == 1 && mine && p.counter) x.before[ch] = state_before_group(a, p, t, c, reach);
    if (p.counter) __syncthreads();
    if (part != 0 || !mine) return;
    float s;
    if (reach < 0) s = start ? start[c] : 0.f;
    else s = p.counter ? apply(group, x.before[ch]) : 0.f;
    if (p.counter && t.at % kBlock == kBlock - 1) {
        const int64_t blocks = (p.per_chain + kBlock - 1) / kBlock;
        publish(p.states + (t.chain * blocks + t.at / kBlock) * a.D + c, Pair{0.f, apply(own, s)});
    }
    if (carry) carry[t.id * a.D + c] = s;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) {
        const int w = BACK ? kWaves - 1 - i : i;
        const Pair q = {x.A[w][ch], x.b[w][ch]};
        x.b[w][ch] = s;
        s = apply(q, s);
    }
}

// Where sequences begin or end among a wave's rows of packed rows (bit i: row i), and their numbers.
struct Marks {
    uint32_t begins, ends;
    int n[kRows];
};
__device__ __forceinline__ Marks marks_of(const ScanArgs& a, int64_t r0, int rows) {
    Marks m{0, 0, {}};
    if (rows <= 0) return m;
    int64_t n = seq_of(a.cu, a.N, r0);
    int64_t next = offset_of(a.cu, n + 1);
    bool begins = offset_of(a.cu, n) == r0;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        if (i < rows) {
            while (r0 + i >= next && n + 1 < a.N) {
                ++n;
                next = offset_of(a.cu, n + 1);
                begins = true;
            }
            m.n[i] = (int)n;
            if (begins) m.begins |= 1u << i;
            if (r0 + i + 1 == next) m.ends |= 1u << i;
            begins = false;
        }
    }
    return m;
}

// ---------------------------------------------------------------------------- forward
// The rows of a wave with what a row gives: its decay and its input's share.  The gates are made again in the second run
// rather than kept: as they come, in 16 bits, the rows of a wave take half the registers of decays and inputs in 32,
// and twice the workgroups are on a CU while they wait for memory and for one another.
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

// The state before a sequence, or zeros.
template <int CPL>
__device__ __forceinline__ void state_of(const float* h0, int64_t at, bool in, float h[CPL]) {
#pragma unroll
    for (int k = 0; k < CPL; ++k) h[k] = h0 && in ? h0[at + k] : 0.f;
}

template <bool LOGIT, bool MIX, bool XF, bool GF, int CPL, bool FLAT, bool PACK>
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
            state_of<CPL>(a.h0, m.n[i] * a.D + c, in, h);
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
        if (FLAT && (m.begins >> i & 1)) state_of<CPL>(a.h0, m.n[i] * a.D + c, in, h);
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
#pragma unroll
                    for (int k = 0; k < CPL; k += 4) *reinterpret_cast<uint32_t*>(codes + k) = ckpt_code4(u + k, inv, any);
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
        if (in) store_row<XF, CPL>(a.y, r * a.D + c, h);
        if (a.h_final && in) {
            bool ends;
            int64_t n;
            if constexpr (FLAT) ends = m.ends >> i & 1, n = m.n[i];
            else ends = r + 1 == (t.chain + 1) * a.T_fixed, n = t.chain;
            if (ends) store_row<true, CPL>(a.h_final, n * a.D + c, h);
        }
    }
}

// Rows in use: all of them, or those up to the last sequence's end.
template <bool FLAT>
__device__ __forceinline__ int64_t rows_used(const ScanArgs& a) {
    if constexpr (!FLAT) return a.total;
    const int64_t used = offset_of(a.cu, a.N);
    return used < 0 ? 0 : used < a.total ? used : a.total;
}
// Of the segment's rows, how many are the wave's.
__device__ __forceinline__ int rows_of_wave(const Tile& t, int wave) {
    const int left = t.rows - wave * kRows;
    return left < 0 ? 0 : left < kRows ? left : kRows;
}

// `f` with the form of the gates, the same in all threads.
template <class F>
__device__ __forceinline__ void by_form(const ScanArgs& a, F f) {
    if (a.logit) {
        if (a.complement) f(std::true_type(), std::true_type());
        else f(std::true_type(), std::false_type());
    } else {
        if (a.complement) f(std::false_type(), std::true_type());
        else f(std::false_type(), std::false_type());
    }
}

// Waves of a SIMD that the registers are cut to: two to a workgroup.
constexpr int fwd_waves(bool xf, bool gf) { return xf && gf ? 4 : xf || gf ? 5 : 7; }
constexpr int bwd_waves(bool xf, bool gf, bool packed) { return packed && !xf && !gf ? 5 : 4; }

template <bool XF, bool GF, int CPL, bool FLAT, bool PACK>
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
        raw.g[i] = load_raw<GF, CPL>(a.g, at);
        raw.x[i] = load_raw<XF, CPL>(a.x, at);
    }
    Marks m{0, 0, {}};
    int64_t reach = t.at > 0 ? t.at : -1;
    if constexpr (FLAT) {
        m = marks_of(a, r0, rows);
        // segments back to the one where the sequence of the first row begins
        reach = 0;
        if (t.rows > 0) {
            const int64_t begin = offset_of(a.cu, seq_of(a.cu, a.N, t.row0));
            reach = begin < t.row0 ? t.at - (begin < 0 ? 0 : begin) / kScanSeg : 0;
        }
    }
    by_form(a, [&](auto logit, auto mix) {
        fwd_body<decltype(logit)::value, decltype(mix)::value, XF, GF, CPL, FLAT, PACK>(a, p, t, m, raw, rows, r0, c, in,
                                                                                       reach, x);
    });
}

// ---------------------------------------------------------------------------- backward
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

template <bool LOGIT, bool MIX, bool XF, bool GF, int CPL, bool FLAT, bool PACKED>
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
                state_of<CPL>(a.h0, m.n[i] * a.D + c, in, s);
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
            if (FLAT && (m.begins >> i & 1)) state_of<CPL>(a.h0, m.n[i] * a.D + c, in, s);
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
            state_of<CPL>(a.dh_final, m.n[i] * a.D + c, in, s);
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
        if (FLAT && (m.ends >> i & 1)) state_of<CPL>(a.dh_final, m.n[i] * a.D + c, in, s);
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
            store_row<XF, CPL>(a.dx, r * a.D + c, dx);
            store_row<GF, CPL>(a.dg, r * a.D + c, dg);
            if (a.dh0) {
                bool begins;
                int64_t n;
                if constexpr (FLAT) begins = m.begins >> i & 1, n = m.n[i];
                else begins = r == t.chain * a.T_fixed, n = t.chain;
                if (begins) store_row<true, CPL>(a.dh0, n * a.D + c, s);
            }
        }
    }
}

template <bool XF, bool GF, int CPL, bool FLAT, bool PACKED>
__global__ __launch_bounds__(kThreads, bwd_waves(XF, GF, PACKED)) void scan_bwd_kernel(ScanArgs a, ScanPlan p) {
    __shared__ __align__(16) Exchange<CPL> x;
    __shared__ __align__(16) Kept<CPL, !PACKED> kept;
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
        raw.g[i] = load_raw<GF, CPL>(a.g, at);
        raw.dy[i] = load_raw<XF, CPL>(a.dy, at);
        if constexpr (PACKED) {
            if constexpr (CPL == 1) raw.code[i][0] = a.u[at];
            else load_words<CPL / 4>(a.u + at, raw.code[i]);
            scales[i] = a.us[r * blocks + cc / kCkptBlock];
        } else {
            raw.x[i] = load_raw<XF, CPL>(a.x, at);
        }
    }
    if constexpr (PACKED) {
#pragma unroll
        for (int i = 0; i < kRows; i += 4)
            raw.scale[i / 4] = scales[i] | scales[i + 1] << 8 | scales[i + 2] << 16 | scales[i + 3] << 24;
    }
    Marks m{0, 0, {}};
    int64_t reach = t.at > 0 ? t.at : -1;
    if constexpr (FLAT) {
        m = marks_of(a, r0, rows);
        reach = 0;
        if (t.rows == kScanSeg) {  // segments on to the one where the sequence of the last row ends
            const int64_t next = offset_of(a.cu, seq_of(a.cu, a.N, last) + 1), end = next < total ? next : total;
            reach = end > last ? (end - 1) / kScanSeg - t.id : 0;
        }
    }
    by_form(a, [&](auto logit, auto mix) {
        bwd_body<decltype(logit)::value, decltype(mix)::value, XF, GF, CPL, FLAT, PACKED>(a, p, t, m, raw, rows, r0, c, in,
                                                                                         reach, x, kept);
    });
}

// Empties the published words and the counter; sequences without tokens pass their state through.
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

// ---------------------------------------------------------------------------- launches
int64_t words_of(int64_t chains, int64_t per_chain, int64_t D) {
    return chains * D * (per_chain + (per_chain + kGroup - 1) / kGroup + (per_chain + kBlock - 1) / kBlock);
}

// The plan, with the workspace emptied; `from` and `to`: the states that sequences without tokens pass through.
template <int CPL>
ScanPlan plan_of(const ScanArgs& a, const float* from, float* to, hipStream_t st) {
    ScanPlan p{};
    p.cols = (uint32_t)((a.D + 64 * CPL - 1) / (64 * CPL));
    p.chains = a.cu ? 1 : (uint32_t)a.N;
    p.per_chain = (uint32_t)(a.cu ? scan_segments(a) : (a.T_fixed + kScanSeg - 1) / kScanSeg);
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

template <bool XF, bool GF, int CPL>
void fwd(const ScanArgs& a, hipStream_t st) {
    const ScanPlan p = plan_of<CPL>(a, a.h0, a.h_final, st);
    if (a.total == 0) return;
    const dim3 grid(p.cols * p.chains * p.per_chain), block(kThreads);
    if (a.u_out && a.cu) hipLaunchKernelGGL((scan_fwd_kernel<XF, GF, CPL, true, true>), grid, block, 0, st, a, p);
    else if (a.u_out) hipLaunchKernelGGL((scan_fwd_kernel<XF, GF, CPL, false, true>), grid, block, 0, st, a, p);
    else if (a.cu) hipLaunchKernelGGL((scan_fwd_kernel<XF, GF, CPL, true, false>), grid, block, 0, st, a, p);
    else hipLaunchKernelGGL((scan_fwd_kernel<XF, GF, CPL, false, false>), grid, block, 0, st, a, p);
}

template <bool XF, bool GF, int CPL>
void bwd(const ScanArgs& a, hipStream_t st) {
    const ScanPlan p = plan_of<CPL>(a, a.dh_final, a.dh0, st);
    if (a.total == 0) return;
    const dim3 grid(p.cols * p.chains * p.per_chain), block(kThreads);
    if (a.u && a.cu) hipLaunchKernelGGL((scan_bwd_kernel<XF, GF, CPL, true, true>), grid, block, 0, st, a, p);
    else if (a.u) hipLaunchKernelGGL((scan_bwd_kernel<XF, GF, CPL, false, true>), grid, block, 0, st, a, p);
    else if (a.cu) hipLaunchKernelGGL((scan_bwd_kernel<XF, GF, CPL, true, false>), grid, block, 0, st, a, p);
    else hipLaunchKernelGGL((scan_bwd_kernel<XF, GF, CPL, false, false>), grid, block, 0, st, a, p);
}

template <bool XF, bool GF, int CPL>
void step(const ScanArgs& a, const float* h_in, float* h_out, hipStream_t st) {
    const int64_t count = a.N * a.D;
    const dim3 grid((unsigned)((count + 256 * CPL - 1) / (256 * CPL)));
    hipLaunchKernelGGL((scan_step_kernel<XF, GF, CPL>), grid, dim3(256), 0, st, a, h_in, h_out, count);
}

// `f` with the types of x and g.
template <class F>
void by_type(const ScanArgs& a, F f) {
    if (a.x_f32 && a.g_f32) f(std::true_type(), std::true_type());
    else if (a.x_f32) f(std::true_type(), std::false_type());
    else if (a.g_f32) f(std::false_type(), std::true_type());
    else f(std::false_type(), std::false_type());
}

}  // namespace

int64_t scan_places(const ScanArgs& a) {
    const int64_t wide = a.D % 4 == 0 ? 256 : 64;
    return (a.D + wide - 1) / wide * scan_segments(a);
}

// For N sequences and total tokens, packed or of equal lengths: at most total/64 + N segments in all, each group and
// block started anew for each sequence.
int64_t scan_workspace_bytes(int64_t N, int64_t total, int64_t D) {
    if (total <= kScanSeg) return 0;
    const int64_t s = total / kScanSeg + N;
    return 256 + 8 * D * (s + s / kGroup + N + s / kBlock + N);
}

hipError_t launch_scan_fwd(const ScanArgs& a, hipStream_t st) {
    by_type(a, [&](auto xf, auto gf) {
        if (a.D % 4 == 0) fwd<decltype(xf)::value, decltype(gf)::value, 4>(a, st);
        else fwd<decltype(xf)::value, decltype(gf)::value, 1>(a, st);
    });
    return hipGetLastError();
}

hipError_t launch_scan_bwd(const ScanArgs& a, hipStream_t st) {
    by_type(a, [&](auto xf, auto gf) {
        if (a.D % 4 == 0) bwd<decltype(xf)::value, decltype(gf)::value, 4>(a, st);
        else bwd<decltype(xf)::value, decltype(gf)::value, 1>(a, st);
    });
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
