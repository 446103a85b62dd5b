// Gated scan over channels, h_t = a_t h_{t-1} + w_t x_t: what its kernels share
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
// Why this size: 64 tokens give 4096 workgroups at B = 4, T = 8192, D = 2048, several to each place on the card, and 64
// pairs of 8 bytes against 64 rows of 2 or 4 each way; a workgroup that goes on over several segments and asks for the next
// one's rows early was slower (152 us against 98), since those who wait for its tiles wait for tiles not begun.  256
// channels a row (CPL = 4: 8 or 16 bytes a lane) and 512 do the same (98.1 and 98.9 us).
// What bounds it: memory and the vector units, each busy most of the time, and the waits between.  Of the 92 us of that call
// the vector units work 69% (each gate takes an exponential and, from logits, a reciprocal, in both runs); its rows
// moved by the same workgroups and nothing else take 77 us, of a plain copy's 64.  Its waves spend half of their
// cycles waiting, for rows and for earlier segments.  fp32 rows leave the vector units idle (20%) and are bound by memory.
// Before the kernel comes the emptying of the words, 4 to 8 us.
//
// Why every wait ends: a workgroup takes its place in the order of work from a counter when it starts, and only waits for
// segments whose places were taken earlier, by workgroups that are therefore running or done.  The one
// with the lowest place among those not done waits for nobody.
//
// The backward pass is the same scan with time reversed, of e_t = a_t (dy_t + e_{t+1}).
#pragma once
#include <type_traits>

#include "kda_ckpt8.h"
#include "kda_layer_launch.h"

namespace kda {

typedef unsigned long long u64;

struct ScanPlan {
    uint32_t cols;      // groups of 64 * CPL channels
    uint32_t chains;    // sequences with segments of their own; 1 for packed rows
    uint32_t per_chain; // segments of a chain
    uint32_t* counter;  // nullptr: no chain is longer than a segment
    u64 *pairs, *groups, *states;
};

namespace {

constexpr int kWaves = 8, kRows = 8, kThreads = kScanThreads;
static_assert(kWaves * kRows == kScanSeg && kWaves * 64 == kThreads, "a wave's rows");
constexpr int kGroup = 8, kBlock = 64;  // segments of a group and of a block

// ---------------------------------------------------------------------------- rows in registers
// CPL consecutive elements of a row as they come from memory.
template <bool F32, int CPL>
struct Raw {
    static constexpr int WORDS = F32 ? CPL : (CPL + 1) / 2;
    uint32_t w[WORDS];
};
// Rows are read once and written once, past the caches where `stream` says so.  (One sequence of 131072 tokens of 1024 bf16
// channels: 240 us through the caches, 228 past them; B = 4, T = 8192, D = 2048: 98.5 and 97.7.)
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
template <class T, bool STREAM>
__device__ __forceinline__ T load_as(const void* p) {
    if constexpr (STREAM) return __builtin_nontemporal_load(static_cast<const T*>(p));
    else return *static_cast<const T*>(p);
}
template <bool STREAM, class T>
__device__ __forceinline__ void store_as(void* p, T v) {
    if constexpr (STREAM) __builtin_nontemporal_store(v, static_cast<T*>(p));
    else *static_cast<T*>(p) = v;
}
template <int WORDS, bool STREAM>
__device__ __forceinline__ void load_words(const void* p, uint32_t* w) {
    if constexpr (WORDS == 4) {
        const u32x4 v = load_as<u32x4, STREAM>(p);
        w[0] = v[0]; w[1] = v[1]; w[2] = v[2]; w[3] = v[3];
    } else if constexpr (WORDS == 2) {
        const u32x2 v = load_as<u32x2, STREAM>(p);
        w[0] = v[0]; w[1] = v[1];
    } else {
        w[0] = load_as<uint32_t, STREAM>(p);
    }
}
template <bool F32, int CPL, bool STREAM = false>
__device__ __forceinline__ Raw<F32, CPL> load_raw(const void* base, int64_t i) {
    Raw<F32, CPL> r;
    if constexpr (F32) load_words<CPL, STREAM>(static_cast<const float*>(base) + i, r.w);
    else if constexpr (CPL == 1) r.w[0] = static_cast<const uint16_t*>(base)[i];
    else load_words<CPL / 2, STREAM>(static_cast<const uint16_t*>(base) + i, r.w);
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
template <bool F32, int CPL, bool STREAM = false>
__device__ __forceinline__ void store_row(void* base, int64_t i, const float v[CPL]) {
    if constexpr (F32) {
        float* p = static_cast<float*>(base) + i;
        if constexpr (CPL == 4) store_as<STREAM>(p, f32x4{v[0], v[1], v[2], v[3]});
        else *p = v[0];
    } else {
        uint16_t* p = static_cast<uint16_t*>(base) + i;
        if constexpr (CPL == 4) store_as<STREAM>(p, u32x2{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])});
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

// Where sequence n of packed rows begins; offsets are read through the scalar cache (the kernels do not write them).
__device__ __forceinline__ int64_t offset_of(const ScanArgs& a, int64_t n) {
    typedef const __attribute__((address_space(4))) int32_t* scalar;
    return a.cu ? (int64_t)((scalar)a.cu)[__builtin_amdgcn_readfirstlane((int)n)] : n * a.T_fixed;
}
// The sequence that holds row r of packed rows: the last n that begins at r or before, of lo .. hi.
__device__ __forceinline__ int search(const ScanArgs& a, int64_t r, int lo, int hi) {
    while (lo < hi) {
        const int mid = lo + (hi - lo + 1) / 2;
        if (offset_of(a, mid) <= r) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}
__device__ __forceinline__ int64_t seq_of(const ScanArgs& a, int64_t r) {
    return a.cu ? search(a, r, 0, (int)a.N - 1) : r / a.T_fixed;
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

// What earlier segments have published for a channel, as far as a thread folds it: the pairs of the segments before t.at in
// its group, or (OUTER) the pairs of the groups before it in its block and the state before the block.
constexpr int kPeeked = kGroup - 1;
static_assert(kBlock / kGroup - 1 == kPeeked, "as many groups in a block as segments in a group");
struct Peeked {
    const u64 *at, *state;  // state nullptr: none has a part in it
    int n;
    u64 w[kPeeked], ws;
};
// Reads what is there so far.  `reach` segments back at most have a part in the state (packed rows: those from the sequence's
// first on).
template <bool OUTER>
__device__ __forceinline__ void peek_before(const ScanArgs& a, const ScanPlan& p, const Tile& t, int64_t c, int64_t reach,
                                            Peeked& k) {
    k.state = nullptr;
    if constexpr (OUTER) {
        const int64_t groups = (p.per_chain + kGroup - 1) / kGroup, blocks = (p.per_chain + kBlock - 1) / kBlock;
        k.n = (int)(t.at / kGroup % (kPeeked + 1));
        k.at = p.groups + (t.chain * groups + t.at / kGroup - k.n) * a.D + c;
        if (t.at >= kBlock && t.at - reach < t.at / kBlock * kBlock)
            k.state = p.states + (t.chain * blocks + t.at / kBlock - 1) * a.D + c;
        k.ws = k.state ? peek(k.state) : 0;
    } else {
        k.n = (int)(t.at % kGroup);
        k.at = p.pairs + (t.chain * p.per_chain + t.at - k.n) * a.D + c;
    }
#pragma unroll
    for (int i = 0; i < kPeeked; ++i) k.w[i] = i < k.n ? peek(k.at + i * a.D) : 0;
}
__device__ __forceinline__ Pair fold(const ScanArgs& a, const Peeked& k) {
    Pair all = {1.f, 0.f};
#pragma unroll
    for (int i = 0; i < kPeeked; ++i)
        if (i < k.n) all = then(all, await(k.at + i * a.D, k.w[i]));
    return all;
}
// The state before the group; the group's last segment publishes the group's pair.
__device__ __forceinline__ float state_before_group(const ScanArgs& a, const Peeked& k) {
    return apply(fold(a, k), k.state ? await(k.state, k.ws).b : 0.f);
}
__device__ __forceinline__ Pair group_before(const ScanArgs& a, const ScanPlan& p, const Tile& t, int64_t c, const Peeked& k,
                                             Pair own) {
    const Pair group = fold(a, k);
    if (k.n == kPeeked) {
        const int64_t groups = (p.per_chain + kGroup - 1) / kGroup;
        publish(p.groups + (t.chain * groups + t.at / kGroup) * a.D + c, then(group, own));
    }
    return group;
}

// What the waves of a workgroup tell one another of its channels: their pairs, then the states before them, and
// the state before the segment's group.  put() and take() move 16 bytes at a time.
template <int CPL>
struct alignas(16) Exchange {
    float A[kWaves][64 * CPL], b[kWaves][64 * CPL], before[64 * CPL];
};
// Half of what a lane keeps of its rows in the backward pass, so that two workgroups' registers fit a CU.
constexpr int kKept = kRows / 2;
template <int CPL, bool USED>
struct alignas(16) Kept {
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
            Peeked k;
            peek_before<false>(a, p, t, c, reach, k);
            group = group_before(a, p, t, c, k, own);
        }
    }
    if (part == 1 && mine && p.counter) {
        Peeked k;
        peek_before<true>(a, p, t, c, reach, k);
        x.before[ch] = state_before_group(a, k);
    }
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

// Where sequences begin or end among a wave's rows of packed rows (bit i: row i), and their numbers, row i's in lane i (in
// scalar registers they cost more than they give: the few places that ask are where sequences begin or end).
struct Marks {
    uint32_t begins, ends;
    int n;
    __device__ __forceinline__ int64_t seq(int i) const { return __builtin_amdgcn_readlane(n, i); }
};
// A turn of the loop for each sequence that has rows here.  The next one is most often the one behind; past more empty ones
// the steps double, and a search between the last two ends them, so that any number of them costs a few loads.
__device__ __forceinline__ Marks marks_of(const ScanArgs& a, int64_t r0, int rows) {
    Marks m{0, 0, 0};
    if (rows <= 0) return m;
    const int last = (int)a.N - 1, lane = threadIdx.x & 63;
    int n = (int)seq_of(a, r0);
    int64_t from = offset_of(a, n), next = offset_of(a, n + 1);
#pragma unroll 1
    for (int i = 0;;) {
        const int64_t left = next - r0;
        const int end = n == last || left >= rows ? rows : left <= i ? i + 1 : (int)left;
        if (from == r0 + i) m.begins |= 1u << i;
        if (left == end) m.ends |= 1u << (end - 1);
        m.n = lane >= i ? n : m.n;
        if (end == rows) return m;
        i = end;  // n < last
        from = next;
        next = offset_of(a, ++n + 1);
        if (next <= r0 + i && n < last) {
            int step = 1;
            while (step <= last - n && offset_of(a, n + step) <= r0 + i) {
                n += step;
                step *= 2;
            }
            n = search(a, r0 + i, n, step - 1 < last - n ? n + step - 1 : last);
            from = offset_of(a, n);
            next = offset_of(a, n + 1);
        }
    }
}

// Rows in use: all of them, or those up to the last sequence's end.
template <bool FLAT>
__device__ __forceinline__ int64_t rows_used(const ScanArgs& a) {
    if constexpr (!FLAT) return a.total;
    const int64_t used = offset_of(a, a.N);
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

// The state before a sequence, or zeros.
template <int CPL>
__device__ __forceinline__ void state_of(const float* h0, int64_t at, bool in, float h[CPL]) {
#pragma unroll
    for (int k = 0; k < CPL; ++k) h[k] = h0 && in ? h0[at + k] : 0.f;
}

// ---------------------------------------------------------------------------- launches
// `f` with packed rows or batches, with or without 8-bit factors, past the caches or through them (kStreamBytes).
template <int CPL, class F>
void by_kind(bool flat, bool packed, bool stream, F f) {
    typedef std::true_type Y;
    typedef std::false_type N;
    const auto with = [&](auto s) {
        if (flat) packed ? f(Y(), Y(), s) : f(Y(), N(), s);
        else packed ? f(N(), Y(), s) : f(N(), N(), s);
    };
    if constexpr (CPL > 1) {
        if (stream) return with(Y());
    }
    with(N());
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

// The plan of a call whose lanes take cpl channels, with its workspace emptied; `from` and `to`: the states that sequences
// without tokens pass through.
ScanPlan scan_plan(const ScanArgs& a, int cpl, const float* from, float* to, hipStream_t st);

// The kernels of x's type, in a file of each.
template <bool XF>
void scan_fwd_of(const ScanArgs& a, hipStream_t st);
template <bool XF>
void scan_bwd_of(const ScanArgs& a, hipStream_t st);

}  // namespace kda
