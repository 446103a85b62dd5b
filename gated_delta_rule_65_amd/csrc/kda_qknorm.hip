// Norm of queries and keys per head with the position rotation in the same pass, forward and backward
// (mathematics and layouts: include/kda_layer.h).
//
// A row (token, head) of D channels goes to D/16 lanes of 16 channels, both channels of a turned pair in one lane, so that
// only the row's sums cross lanes.  A workgroup takes a few whole tokens with all their heads: the angles, 64-bit products
// with a sine and a cosine each, are made once a token and shared by its heads through LDS, while the first rows'
// loads are in flight.  Both passes move their bytes once; what bounds them is HBM.
//
// The gradient, with z^ = r x the normed row, d the outputs' gradient turned back and times w: dx = r (d - s (d . z^) z^),
// dw = the sum over rows of (d turned back) z^.
//
// Measured (q and k of 16 heads of 128 bf16 channels, 32768 tokens): forward, half of the channels turned, columns of one
// projection, 537 MB in 93 us (5.8 TB/s; 101 without the exchange of chunks, since
// half lines at a time do not go past the caches); forward with the raw rows packed in 8 bits beside, 675 MB in 110 us (6.1
// TB/s); backward from the packed rows with the weights' gradients, 675 MB in 123 us (5.5 TB/s; its three workgroups a CU
// stop at each tile's tables) and 5 us for the weights' sums.  4099 tokens of 12 + 2 heads of 64 fp32 channels: 10
// us forward and 14 backward for 74 MB in all; 32 tokens: 4.8 us, one pass of latency.
#include <type_traits>

#include "kda_ckpt8.h"
#include "kda_layer_launch.h"

namespace kda {

namespace {

constexpr int kThreads = 256;
constexpr int kAngles = 2048;  // pairs of a workgroup's tokens at most: 16 KiB of cosines and sines

// The two chunks of eight channels that a lane of a row holds, such that both channels of every pair that is turned are in
// one lane: lane j of D/16 holds channels first .. +7 and second .. +7.
//   Spread (adjacent pairs, no rotation, or halves of the whole head): 8j and D/2 + 8j.  Pairs (2i, 2i + 1) lie in a
//     chunk, pairs (i, i + D/2) in the two of a lane, and the lanes' chunks are side by side: whole lines at a time.
//   Else (halves of part of the head, pairs (i, i + rot/2)): 8j and rot/2 + 8j for the lanes j < rot/16, and the channels
//     behind in the same way for those after them.
//   Halves of half of the head lie in whole lines too once lanes exchange a chunk: lane j of the lower half and lane
//     LANES - 1 - j load and store as if spread (so that a line takes one instruction) and each keeps what the other
//     needs: (8j, D/2 + 8j) and (D/4 + 8j, 3D/4 + 8j) in memory, (8j, D/4 + 8j) and (D/2 + 8j, 3D/4 + 8j) in use.
struct Place {
    int first, second;
    bool turned0, turned1;  // the chunks lie in the turned channels
    int mem_first, mem_second;
    bool exchange, low;     // chunks are exchanged; the lane is of the lower half
};
__host__ __device__ __forceinline__ bool is_spread(int D, int rot, bool interleaved) { return interleaved || rot == 0 || rot == D; }
__host__ __device__ __forceinline__ bool is_exchanged(int D, int rot, bool interleaved) { return !interleaved && 2 * rot == D; }
template <int D>
__device__ __forceinline__ Place place_of(int j, int rot, bool interleaved) {
    const bool spread = is_spread(D, rot, interleaved), half = spread || j < rot / 16;
    const int first = 8 * j + (half ? 0 : rot / 2), apart = spread ? D / 2 : half ? rot / 2 : (D - rot) / 2;
    if (!is_exchanged(D, rot, interleaved)) return {first, first + apart, first < rot, first + apart < rot, first, first + apart, false, half};
    const int m = half ? j : D / 16 - 1 - j, in_use = 8 * m + (half ? 0 : D / 2), in_memory = 8 * m + (half ? 0 : D / 4);
    return {in_use, in_use + D / 4, half, half, in_memory, in_memory + D / 2, true, half};
}

// From chunks a and b as they lie in memory to those in use, and back: the same exchange.
template <int D, int WORDS>
__device__ __forceinline__ void exchange(uint32_t* a, uint32_t* b, bool low) {
#pragma unroll
    for (int k = 0; k < WORDS; ++k) {
        const int send = (int)(low ? b[k] : a[k]);
        const uint32_t got = (uint32_t)(D == 128 ? __builtin_amdgcn_update_dpp(0, send, 0x141, 0xf, 0xf, true)   // 7 - lane
                                                 : __builtin_amdgcn_update_dpp(0, send, 0x1B, 0xf, 0xf, true));  // 3 - lane
        a[k] = low ? a[k] : got;
        b[k] = low ? got : b[k];
    }
}

// The sum over the lanes of a row (4 or 8 neighbours), the same bits in each of them.
template <int LANES>
__device__ __forceinline__ float row_sum(float v) {
    static_assert(LANES == 4 || LANES == 8, "lanes of a row");
    const auto from = [](float x, auto ctrl) {
        return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), decltype(ctrl)::value, 0xf, 0xf, true));
    };
    v += from(v, std::integral_constant<int, 0xB1>());  // lane ^ 1
    v += from(v, std::integral_constant<int, 0x4E>());  // lane ^ 2
    if constexpr (LANES == 8) v += from(v, std::integral_constant<int, 0x141>());  // the other quad
    return v;
}

// (s |x|^2 + eps)^(-1/2) of a row, 0 where that is 0.  Rows whose sum of squares leaves float32's comfortable
// range are summed again at a power of two of their own size.  A root beyond 2^66 would have a reciprocal near or below the
// smallest normal float (2^-132 at worst): such a row is scaled down by 2^64 in place, `unit` says by what (else 1), and
// what is returned is the root's reciprocal for the row as it then is.
template <int LANES>
__device__ __forceinline__ float row_rsqrt(float x[16], float s, float eps, float& unit) {
    unit = 1.f;
    float ss = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) ss = fmaf(x[k], x[k], ss);
    ss = row_sum<LANES>(ss);
    if (ss > 0x1p-100f && ss < 0x1p100f) return __builtin_amdgcn_rsqf(fmaf(ss, s, eps));
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < 16; ++k) top = max(top, abs_bits(x[k]));
    top = lanes_max<LANES>(top);
    if (top >= kInfBits) return __uint_as_float(0x7fc00000u);  // a row that holds infinity or NaN has no norm
    if (top == 0) return eps > 0.f ? rsqrtf(eps) : 0.f;
    int e;
    frexpf(__uint_as_float(top), &e);
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        const float u = ldexpf(x[k], -e);
        sum = fmaf(u, u, sum);
    }
    sum = row_sum<LANES>(sum);
    const double total = (double)sum * s * ldexp(1.0, 2 * e) + eps;
    if (total > 0x1p132) {
        unit = 0x1p-64f;
#pragma unroll
        for (int k = 0; k < 16; ++k) x[k] *= unit;
        return (float)(0x1p64 / sqrt(total));
    }
    return total < 0x1p-252 ? 0.f : (float)(1.0 / sqrt(total));
}

// Sixteen channels of a row as they come from memory: two chunks of eight.
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
template <bool F32, bool PACKED>
struct Chunks {
    u32x4 a[F32 ? 2 : 1], b[F32 ? 2 : 1];
};
template <bool F32>
struct Chunks<F32, true> {
    u32x2 a, b;
    uint8_t sa, sb;
};
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
template <bool STREAM, bool F32, bool PACKED>
__device__ __forceinline__ void load_chunks(const void* p, const uint8_t* scales, int64_t row, const Place& at,
                                            Chunks<F32, PACKED>& c) {
    if constexpr (PACKED) {
        const uint8_t* s = static_cast<const uint8_t*>(p) + row;
        c.a = load_as<u32x2, STREAM>(s + at.mem_first);
        c.b = load_as<u32x2, STREAM>(s + at.mem_second);
        c.sa = scales[(row + at.first) / kCkptBlock];
        c.sb = scales[(row + at.second) / kCkptBlock];
    } else {
        const char* s = static_cast<const char*>(p) + row * (F32 ? 4 : 2);
#pragma unroll
        for (int i = 0; i < (F32 ? 2 : 1); ++i) {
            c.a[i] = load_as<u32x4, STREAM>(s + at.mem_first * (F32 ? 4 : 2) + 16 * i);
            c.b[i] = load_as<u32x4, STREAM>(s + at.mem_second * (F32 ? 4 : 2) + 16 * i);
        }
    }
}
template <bool F32>
__device__ __forceinline__ void chunk_values(const uint32_t* c, float x[8]) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        if constexpr (F32) x[k] = __uint_as_float(c[k]);
        else x[k] = __uint_as_float(k % 2 ? c[k / 2] & 0xffff0000u : c[k / 2] << 16);
    }
}
template <int D, bool F32, bool PACKED>
__device__ __forceinline__ void values_of(const Chunks<F32, PACKED>& c, const Place& at, float x[16]) {
    if constexpr (PACKED) {
        uint32_t a[2] = {c.a[0], c.a[1]}, b[2] = {c.b[0], c.b[1]};
        if (at.exchange) exchange<D, 2>(a, b, at.low);
        const float ua = ckpt_unit(c.sa), ub = ckpt_unit(c.sb);
        ckpt_value4(a[0], ua, x);
        ckpt_value4(a[1], ua, x + 4);
        ckpt_value4(b[0], ub, x + 8);
        ckpt_value4(b[1], ub, x + 12);
    } else {
        constexpr int N = F32 ? 2 : 1;
        uint32_t a[4 * N], b[4 * N];
#pragma unroll
        for (int k = 0; k < 4 * N; ++k) a[k] = c.a[k / 4][k % 4], b[k] = c.b[k / 4][k % 4];
        if (at.exchange) exchange<D, 4 * N>(a, b, at.low);
        chunk_values<F32>(a, x);
        chunk_values<F32>(b, x + 8);
    }
}
template <int D, bool STREAM, bool F32>
__device__ __forceinline__ void store_chunks(void* p, int64_t row, const Place& at, const float x[16]) {
    if constexpr (F32) {
        uint32_t a[8], b[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) a[k] = __float_as_uint(x[k]), b[k] = __float_as_uint(x[8 + k]);
        if (at.exchange) exchange<D, 8>(a, b, at.low);
        float* d = static_cast<float*>(p) + row;
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
            store_as<STREAM>(d + at.mem_first + i, u32x4{a[i], a[i + 1], a[i + 2], a[i + 3]});
            store_as<STREAM>(d + at.mem_second + i, u32x4{b[i], b[i + 1], b[i + 2], b[i + 3]});
        }
    } else {
        typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
        bf8 u, v;
#pragma unroll
        for (int k = 0; k < 8; ++k) u[k] = (__bf16)x[k], v[k] = (__bf16)x[8 + k];
        const u32x4 pu = __builtin_bit_cast(u32x4, u), pv = __builtin_bit_cast(u32x4, v);
        uint32_t a[4] = {pu[0], pu[1], pu[2], pu[3]}, b[4] = {pv[0], pv[1], pv[2], pv[3]};
        if (at.exchange) exchange<D, 4>(a, b, at.low);
        uint16_t* d = static_cast<uint16_t*>(p) + row;
        store_as<STREAM>(d + at.mem_first, u32x4{a[0], a[1], a[2], a[3]});
        store_as<STREAM>(d + at.mem_second, u32x4{b[0], b[1], b[2], b[3]});
    }
}

// Cosine and sine of pos * freq radians.  Only the fraction of a turn counts, and pos * freq / 2 pi may be many turns: freq / 2 pi
// is taken as a sum hi + lo of two 64-bit numbers and each product with the position as its rounded value and what that
// leaves, so that of 2^k turns the fraction keeps 2^(k - 106): angles below 2^80 radians are as good as small ones, for
// any position (64-bit ones go in two parts, each a whole number of at most 40 bits).  Contraction off: the rounded
// product has to be the same number in both of its uses.
__device__ __forceinline__ double turn_part(double p, double hi, double lo) {
#pragma clang fp contract(off)
    const double t = p * hi, e = fma(p, lo, fma(p, hi, -t));
    return (t - rint(t)) + (e - rint(e));
}
__device__ __forceinline__ void angle(int64_t pos, double freq, bool wide, float& c, float& s) {
#pragma clang fp contract(off)
    constexpr double inv_hi = 0x1.45f306dc9c883p-3, inv_lo = -0x1.6b01ec5417056p-57;  // 1 / 2 pi
    const double hi = freq * inv_hi, lo = fma(freq, inv_lo, fma(freq, inv_hi, -hi));
    double t;
    if (wide) t = turn_part((double)(pos >> 24) * 0x1p24, hi, lo) + turn_part((double)(int32_t)(pos & 0xffffff), hi, lo);
    else t = turn_part((double)(int32_t)pos, hi, lo);
    sincospif(2.f * (float)(t - rint(t)), &s, &c);
}

// The tables of a workgroup's tokens in LDS, in the order in which lanes read them: a lane's eight values of a token as two
// 16-byte reads, the lanes of a row side by side.  With adjacent pairs that is the pairs' own order.
template <int D>
struct Tables {
    static constexpr int LANES = D / 16;
    float c[kAngles], s[kAngles];
    float w[2][D];

    // value `pair` of a token, rot/2 to a token
    static __device__ __forceinline__ int slot(int token, int pair, int rot, bool interleaved) {
        const int lanes = rot / 16;
        return token * lanes * 8 + (interleaved ? pair : (pair & 4) * lanes + (pair >> 3) * 4 + (pair & 3));
    }
    // What the tables are made from is asked for before the rows, and used while those are on their way: loads come
    // back in order.
    struct Source {
        int64_t pos;
        double freq;
        float w;
    };
    static __device__ __forceinline__ int64_t position(const QkArgs& a, int64_t t) {
        return a.pos64 ? static_cast<const int64_t*>(a.pos)[t] : static_cast<const int32_t*>(a.pos)[t];
    }
    static __device__ __forceinline__ Source first_of(const QkArgs& a, int64_t t0, int tokens, bool weighted) {
        Source s{0, 0.0, 1.f};
        const int pairs = a.rot / 2, i = threadIdx.x;
        if (i < tokens * pairs) {
            const int t = (uint32_t)i / (uint32_t)pairs;
            s.pos = position(a, t0 + t);
            s.freq = a.freqs[i - t * pairs];
        }
        if (weighted && i < 2 * D) s.w = weight_at(a, i);
        return s;
    }
    static __device__ __forceinline__ float weight_at(const QkArgs& a, int i) {
        const int side = i / D, at = i % D, m = at / (4 * LANES), j = at / 4 % LANES, k = (m & 1) * 4 + at % 4;
        const Place p = place_of<D>(j, a.rot, a.interleaved);
        const int first = p.first, second = p.second;
        const float* src = side ? a.wk : a.wq;
        return src ? src[(m < 2 ? first : second) + k] : 1.f;
    }
    __device__ __forceinline__ void fill_weights(float first) {
        static_assert(2 * D <= kThreads, "a weight a thread");
        if (threadIdx.x < 2 * D) (&w[0][0])[threadIdx.x] = first;
    }
    __device__ __forceinline__ void fill_angles(const QkArgs& a, int64_t t0, int tokens, const Source& first) {
        const int pairs = a.rot / 2;
        int64_t pos = first.pos;
        double freq = first.freq;
        for (int i = threadIdx.x; i < tokens * pairs; i += kThreads) {
            const int t = (uint32_t)i / (uint32_t)pairs, q = i - t * pairs;
            if (i != (int)threadIdx.x) {
                pos = position(a, t0 + t);
                freq = a.freqs[q];
            }
            const int at = slot(t, q, a.rot, a.interleaved);
            angle(pos, freq, a.pos64, c[at], s[at]);
        }
    }
    __device__ __forceinline__ void weight(int side, int j, float v[16]) const {
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const float4 u = *reinterpret_cast<const float4*>(&w[side][m * 4 * LANES + 4 * j]);
            v[4 * m] = u.x; v[4 * m + 1] = u.y; v[4 * m + 2] = u.z; v[4 * m + 3] = u.w;
        }
    }
    __device__ __forceinline__ void four(int at, float cv[4], float sv[4]) const {
        const float4 u = *reinterpret_cast<const float4*>(c + at), v = *reinterpret_cast<const float4*>(s + at);
        cv[0] = u.x; cv[1] = u.y; cv[2] = u.z; cv[3] = u.w;
        sv[0] = v.x; sv[1] = v.y; sv[2] = v.z; sv[3] = v.w;
    }
    // The four adjacent pairs of a chunk.
    __device__ __forceinline__ void adjacent(float* x, int at, float sign) const {
        float cv[4], sv[4];
        four(at, cv, sv);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float u = x[2 * k], v = x[2 * k + 1], t = sign * sv[k];
            x[2 * k] = u * cv[k] - v * t;
            x[2 * k + 1] = v * cv[k] + u * t;
        }
        __asm__ volatile("; a chunk of adjacent pairs");
    }
    // z = (x0 c - x1 s, x1 c + x0 s) on the lane's pairs; sign -1 turns back.
    __device__ __forceinline__ void turn(float x[16], int token, int j, const Place& p, int rot, bool interleaved,
                                         float sign) const {
        const int lanes = rot / 16, base = token * lanes * 8;
        if (interleaved) {
            if (p.turned0) adjacent(x, base + p.first / 2, sign);
            if (p.turned1) adjacent(x + 8, base + p.second / 2, sign);
            __asm__ volatile("; adjacent pairs");  // keeps the two forms' ends apart: joined, they would put x into memory
        } else if (p.turned0) {
            float cv[8], sv[8];
            four(base + 4 * j, cv, sv);
            four(base + 4 * lanes + 4 * j, cv + 4, sv + 4);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float u = x[k], v = x[8 + k], t = sign * sv[k];
                x[k] = u * cv[k] - v * t;
                x[8 + k] = v * cv[k] + u * t;
            }
            __asm__ volatile("; halves");
        }
    }
};

// The row's channels packed in 8 bits, from the raw values.  The lanes of a block: the quad of each chunk where chunks are
// spread or halves are whole blocks; other halves exchange each block's largest over the whole row.
template <int D>
__device__ __forceinline__ void pack_row(const float x[16], const Place& p, int j, int rot, bool interleaved,
                                         uint8_t* codes, uint8_t* scales) {
    constexpr int LANES = D / 16, BLOCKS = D / kCkptBlock;
    int s0, s1;
    bool any0, any1;
    if (is_spread(D, rot, interleaved) || rot % 64 == 0) {
        uint32_t t0 = lanes_max<4>(ckpt_amax<8>(x)), t1 = lanes_max<4>(ckpt_amax<8>(x + 8));
        any0 = t0 > kCkptTopBits;
        any1 = t1 > kCkptTopBits;
        if (__any(any0 || any1)) {
            t0 = lanes_max<4>(ckpt_amax_finite<8>(x));
            t1 = lanes_max<4>(ckpt_amax_finite<8>(x + 8));
        }
        s0 = ckpt_scale(t0);
        s1 = ckpt_scale(t1);
    } else {
        const uint32_t m0 = ckpt_amax_finite<8>(x), m1 = ckpt_amax_finite<8>(x + 8);
        s0 = s1 = 0;
        any0 = any1 = true;
#pragma unroll
        for (int b = 0; b < BLOCKS; ++b) {
            const bool in0 = p.first / kCkptBlock == b, in1 = p.second / kCkptBlock == b;
            const int s = ckpt_scale(lanes_max<LANES>(max(in0 ? m0 : 0u, in1 ? m1 : 0u)));
            if (in0) s0 = s;
            if (in1) s1 = s;
        }
    }
    const float i0 = ckpt_inverse(s0), i1 = ckpt_inverse(s1);
    *reinterpret_cast<u32x2*>(codes + p.first) = u32x2{ckpt_code4(x, i0, any0), ckpt_code4(x + 4, i0, any0)};
    *reinterpret_cast<u32x2*>(codes + p.second) = u32x2{ckpt_code4(x + 8, i1, any1), ckpt_code4(x + 12, i1, any1)};
    // a block's first channels are the start of some lane's chunk
    if (p.first % kCkptBlock == 0) scales[p.first / kCkptBlock] = (uint8_t)s0;
    if (p.second % kCkptBlock == 0) scales[p.second / kCkptBlock] = (uint8_t)s1;
}

// `per` tokens to a workgroup, their rows (queries, then keys, of a token) by passes of 256 / LANES; PASSES passes are
// loaded before the first of them is used.
template <int D, bool F32, bool PACKED, bool STREAM>
__global__ __launch_bounds__(kThreads, 4) void qknorm_fwd_kernel(QkArgs a, int per) {
    constexpr int LANES = D / 16, ROWS = kThreads / LANES, PASSES = F32 ? 2 : 4;
    __shared__ __align__(16) Tables<D> tab;
    const int H = a.Hq + a.Hk, j = threadIdx.x % LANES;
    const Place p = place_of<D>(j, a.rot, a.interleaved);
    const int64_t t0 = (int64_t)blockIdx.x * per;
    const int tokens = a.tokens - t0 < per ? (int)(a.tokens - t0) : per, rows = tokens * H;
    const bool weighted = a.wq || a.wk;
    const typename Tables<D>::Source source = Tables<D>::first_of(a, t0, tokens, weighted);
    for (int base = 0; base < rows; base += PASSES * ROWS) {
        Chunks<F32, PACKED> c[PASSES];
        int tok[PASSES], head[PASSES];
#pragma unroll
        for (int i = 0; i < PASSES; ++i) {
            int r = base + i * ROWS + threadIdx.x / LANES;
            r = r < rows ? r : rows - 1;
            tok[i] = (uint32_t)r / (uint32_t)H;
            head[i] = r - tok[i] * H;
            const bool key = head[i] >= a.Hq;
            const int64_t t = t0 + tok[i];
            if (key) load_chunks<STREAM>(a.k, a.ks, t * a.k_stride + (head[i] - a.Hq) * D, p, c[i]);
            else load_chunks<STREAM>(a.q, a.qs, t * a.q_stride + head[i] * D, p, c[i]);
        }
        if (base == 0) {
            if (weighted) tab.fill_weights(source.w);
            tab.fill_angles(a, t0, tokens, source);
            __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < PASSES; ++i) {
            if (base + i * ROWS + (int)threadIdx.x / LANES >= rows) continue;
            const bool key = head[i] >= a.Hq;
            const int64_t out = key ? ((t0 + tok[i]) * a.Hk + head[i] - a.Hq) * D : ((t0 + tok[i]) * a.Hq + head[i]) * D;
            float x[16];
            values_of<D>(c[i], p, x);
            if constexpr (!PACKED) {
                if (a.q8)
                    pack_row<D>(x, p, j, a.rot, a.interleaved, (key ? a.k8 : a.q8) + out,
                                (key ? a.k8s : a.q8s) + out / kCkptBlock);
            }
            float unit;
            const float r = row_rsqrt<LANES>(x, a.rms ? 1.f / D : 1.f, a.eps, unit);
#pragma unroll
            for (int k = 0; k < 16; ++k) x[k] *= r;
            if (weighted) {
                float w[16];
                tab.weight(key, j, w);
#pragma unroll
                for (int k = 0; k < 16; ++k) x[k] *= w[k];
            }
            tab.turn(x, tok[i], j, p, a.rot, a.interleaved, 1.f);
            store_chunks<D, STREAM, F32>(key ? a.k_out : a.q_out, out, p, x);
        }
    }
}

// The tokens' queries by tiles of per[0] tokens, then their keys by tiles of per[1].
struct Sides {
    int per[2];
    int64_t tiles[2];
};

// Gradients of the rows.  With weights, a workgroup goes on over the tiles with its lanes' sums in registers and writes them,
// added up in LDS, to its line of the workspace: queries' when it comes to the keys, keys' at the end.  One side's sums at a
// time and as many workgroups as fit at once: with both sides' sums the registers spilled, and of 1024 workgroups
// the last 256 ran alone (145 us against 121 for the call below; tiles of 2, 4, 8 or 16 passes: 124, 121, 122 and 130).
template <int D, bool F32, bool PACKED, bool GF32, bool STREAM>
__global__ __launch_bounds__(kThreads, 3) void qknorm_bwd_kernel(QkArgs a, Sides sides) {
    constexpr int LANES = D / 16, ROWS = kThreads / LANES, PASSES = 2;
    __shared__ __align__(16) Tables<D> tab;
    __shared__ __align__(16) float part[ROWS][D];
    const int j = threadIdx.x % LANES;
    const Place p = place_of<D>(j, a.rot, a.interleaved);
    const float sc = a.rms ? 1.f / D : 1.f;
    const bool weighted = a.wq || a.wk || a.dwq;
    float* line = static_cast<float*>(a.ws) + (int64_t)blockIdx.x * 2 * D;
    float dw[16] = {};
    int at = 0;  // the side whose sums dw holds
    const auto flush = [&] {
        if (a.dwq) {
            __syncthreads();
            float* mine = part[threadIdx.x / LANES];
#pragma unroll
            for (int m = 0; m < 4; ++m)
                *reinterpret_cast<float4*>(mine + (m < 2 ? p.first : p.second) + 4 * (m & 1)) =
                    make_float4(dw[4 * m], dw[4 * m + 1], dw[4 * m + 2], dw[4 * m + 3]);
            __syncthreads();
            if (threadIdx.x < D) {
                float sum = 0.f;
                for (int i = 0; i < ROWS; ++i) sum += part[i][threadIdx.x];
                line[at * D + threadIdx.x] = sum;
            }
        }
#pragma unroll
        for (int k = 0; k < 16; ++k) dw[k] = 0.f;
        ++at;
    };
    for (int64_t tile = blockIdx.x; tile < sides.tiles[0] + sides.tiles[1]; tile += gridDim.x) {
        const int side = tile >= sides.tiles[0];
        if (side != at) flush();
        const int per = sides.per[side], Hs = side ? a.Hk : a.Hq;
        const int64_t t0 = (tile - (side ? sides.tiles[0] : 0)) * per;
        const int tokens = a.tokens - t0 < per ? (int)(a.tokens - t0) : per, rows = tokens * Hs;
        const typename Tables<D>::Source source = Tables<D>::first_of(a, t0, tokens, weighted);
        const void *src = side ? a.k : a.q, *grad = side ? a.d_k : a.d_q;
        const uint8_t* scales = side ? a.ks : a.qs;
        void* to = side ? a.dk : a.dq;
        const int64_t stride = side ? a.k_stride : a.q_stride;
        for (int base = 0; base < rows; base += PASSES * ROWS) {
            Chunks<F32, PACKED> c[PASSES];
            Chunks<GF32, false> g[PASSES];
            int tok[PASSES];
            int64_t out[PASSES];
#pragma unroll
            for (int i = 0; i < PASSES; ++i) {
                int r = base + i * ROWS + threadIdx.x / LANES;
                r = r < rows ? r : rows - 1;
                tok[i] = (uint32_t)r / (uint32_t)Hs;
                out[i] = (t0 * Hs + r) * D;
                load_chunks<STREAM>(src, scales, (t0 + tok[i]) * stride + (r - tok[i] * Hs) * D, p, c[i]);
                load_chunks<STREAM>(grad, nullptr, out[i], p, g[i]);
            }
            if (base == 0) {
                __syncthreads();  // the tables of the tile before are done with
                if (weighted) tab.fill_weights(source.w);
                tab.fill_angles(a, t0, tokens, source);
                __syncthreads();
            }
#pragma unroll
            for (int i = 0; i < PASSES; ++i) {
                if (base + i * ROWS + (int)threadIdx.x / LANES >= rows) continue;
                float x[16], d[16];
                values_of<D>(c[i], p, x);
                values_of<D>(g[i], p, d);
                float unit;
                const float r = row_rsqrt<LANES>(x, sc, a.eps, unit);
                tab.turn(d, tok[i], j, p, a.rot, a.interleaved, -1.f);
#pragma unroll
                for (int k = 0; k < 16; ++k) x[k] *= r;
                if (weighted) {
                    float w[16];
                    tab.weight(side, j, w);
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        dw[k] = fmaf(d[k], x[k], dw[k]);
                        d[k] *= w[k];
                    }
                }
                float dot = 0.f;
#pragma unroll
                for (int k = 0; k < 16; ++k) dot = fmaf(d[k], x[k], dot);
                dot = row_sum<LANES>(dot) * sc;
#pragma unroll
                for (int k = 0; k < 16; ++k) x[k] = r * fmaf(-dot, x[k], d[k]);
                if (unit != 1.f) {
#pragma unroll
                    for (int k = 0; k < 16; ++k) x[k] *= unit;
                }
                store_chunks<D, STREAM, F32>(to, out[i], p, x);
            }
        }
    }
    while (at < 2) flush();
}

// The workgroups' lines added up in a fixed order: 32 threads to a column, each every 32nd line, then those in their
// order.  Columns in groups of 32.
__global__ __launch_bounds__(1024) void qknorm_dw_kernel(const float* __restrict__ lines, int count, int D,
                                                         float* __restrict__ dwq, float* __restrict__ dwk) {
    __shared__ float part[32][33];
    const int col = threadIdx.x % 32, at = threadIdx.x / 32, c = blockIdx.x * 32 + col;
    float sum = 0.f;
#pragma unroll 8
    for (int i = at; i < count; i += 32) sum += lines[(int64_t)i * 2 * D + c];
    part[at][col] = sum;
    __syncthreads();
    if (at == 0) {
        float all = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) all += part[i][col];
        if (c < D) dwq[c] = all;
        else dwk[c - D] = all;
    }
}

// Workgroups that the card holds at once: four a CU of the forward kernel, three of the backward kernel.
constexpr int kFwdGroups = 1024, kBwdGroups = 768;

// Tokens of a tile of H heads: enough rows to fill `passes` passes, as far as their angles fit and the card is filled, all
// the tokens' `heads` taken together (4099 tokens of 12 + 2 fp32 heads, forward: 15 us in 216 workgroups, 13 us in 820; 10 us
// there since the tables' sources are asked for before the rows).
int tokens_of(int64_t tokens, int H, int heads, int D, int rot, int passes, int groups) {
    const int most = passes * kThreads / (D / 16);
    const int64_t share = (tokens * heads + groups - 1) / groups;
    const int rows = most < share ? most : (int)share;
    const int per = (rows + H - 1) / H;
    return rot && per > kAngles / (rot / 2) ? kAngles / (rot / 2) : per;
}

}  // namespace

// At most as many lines as workgroups, and a tile holds a token or more of a side.
int64_t qknorm_bwd_workspace_bytes(int64_t tokens, int, int, int D) {
    return (2 * tokens < kBwdGroups ? 2 * tokens : kBwdGroups) * 2 * D * 4;
}

// Whether a call's rows go past the caches: many bytes, and whole lines at a time (a line that two instructions share
// is written in two parts: 108 us past the caches and 101 through them for the call above before its lanes
// exchanged chunks, 92 and 102 since).
static bool streams(const QkArgs& a, int64_t bytes_per_channel) {
    return a.tokens * (a.Hq + a.Hk) * a.D * bytes_per_channel > kStreamBytes &&
           (is_spread(a.D, a.rot, a.interleaved) || is_exchanged(a.D, a.rot, a.interleaved));
}

template <int D, bool F32, bool PACKED, bool STREAM>
static void fwd(const QkArgs& a, hipStream_t st, int64_t tiles, int per) {
    hipLaunchKernelGGL((qknorm_fwd_kernel<D, F32, PACKED, STREAM>), dim3((unsigned)tiles), dim3(kThreads), 0, st, a, per);
}
template <int D, bool F32, bool PACKED, bool STREAM>
static void bwd(const QkArgs& a, hipStream_t st, const Sides& sides, int groups) {
    const dim3 grid((unsigned)groups), block(kThreads);
    if (a.grad_f32)
        hipLaunchKernelGGL((qknorm_bwd_kernel<D, F32, PACKED, true, STREAM>), grid, block, 0, st, a, sides);
    else hipLaunchKernelGGL((qknorm_bwd_kernel<D, F32, PACKED, false, STREAM>), grid, block, 0, st, a, sides);
}
// `f` with D, the rows' type, whether they are packed and whether they go past the caches.
template <class F>
static void by_kind(const QkArgs& a, bool stream, F f) {
    typedef std::true_type Y;
    typedef std::false_type N;
    const auto with = [&](auto d, auto f32, auto packed) { stream ? f(d, f32, packed, Y()) : f(d, f32, packed, N()); };
    const auto of = [&](auto d) {
        if (a.f32) a.qs ? with(d, Y(), Y()) : with(d, Y(), N());
        else a.qs ? with(d, N(), Y()) : with(d, N(), N());
    };
    if (a.D == 128) of(std::integral_constant<int, 128>());
    else of(std::integral_constant<int, 64>());
}

hipError_t launch_qknorm_fwd(const QkArgs& a, hipStream_t st) {
    const int per = tokens_of(a.tokens, a.Hq + a.Hk, a.Hq + a.Hk, a.D, a.rot, 4, kFwdGroups);
    const int64_t tiles = (a.tokens + per - 1) / per;
    if (tiles > kMaxThreads / kThreads) return hipErrorInvalidConfiguration;
    by_kind(a, streams(a, a.f32 ? 8 : 4), [&](auto d, auto f32, auto packed, auto stream) {
        fwd<decltype(d)::value, decltype(f32)::value, decltype(packed)::value, decltype(stream)::value>(a, st, tiles, per);
    });
    return hipGetLastError();
}

hipError_t launch_qknorm_bwd(const QkArgs& a, hipStream_t st) {
    Sides sides;
    for (int i = 0; i < 2; ++i) {
        sides.per[i] = tokens_of(a.tokens, i ? a.Hk : a.Hq, a.Hq + a.Hk, a.D, a.rot, 4, kBwdGroups);
        sides.tiles[i] = a.tokens ? (a.tokens + sides.per[i] - 1) / sides.per[i] : 0;
    }
    const int64_t tiles = sides.tiles[0] + sides.tiles[1], most = a.dwq ? kBwdGroups : kMaxThreads / kThreads;
    const int groups = (int)(tiles < most ? tiles : most);
    if (groups > 0)  // without tokens only the weights' zero gradients are written
        by_kind(a, streams(a, (a.f32 ? 8 : 4) + (a.grad_f32 ? 4 : 2)), [&](auto d, auto f32, auto packed, auto stream) {
            bwd<decltype(d)::value, decltype(f32)::value, decltype(packed)::value, decltype(stream)::value>(a, st, sides,
                                                                                                          groups);
        });
    if (a.dwq)
        hipLaunchKernelGGL(qknorm_dw_kernel, dim3((unsigned)(2 * a.D / 32)), dim3(1024), 0, st,
                           static_cast<const float*>(a.ws), groups, a.D, a.dwq, a.dwk);
    return hipGetLastError();
}

}  // namespace kda
