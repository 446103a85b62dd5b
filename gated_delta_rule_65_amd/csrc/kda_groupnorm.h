// Group norm with an activation over channels-last rows (mathematics and layouts: include/kda_layer.h): the kernel of both
// passes, for rows that a few lanes hold.
//
// A group of a token goes to P lanes of ITER pieces of CPL channels each, held in registers between the mean, the sum of
// squares around it and the outputs, so that memory is read and written once.  A thread keeps its channels over the tokens
// of its workgroup: weights are read once, and the weights' gradients are sums in registers until the workgroup's end.
//
// Memory bounds it: 32768 x 16 x 128 with weights and a gate, from fp32 to bf16 in 92 us (5.8 TB/s; a copy of as many bytes
// takes 86), in bf16 62 us forward (6.4 TB/s) and 122 backward (5.5 TB/s), in fp32 148 and 263 (5.5 and 5.1 TB/s).
#pragma once
#include <type_traits>

#include "kda_device.h"
#include "kda_layer_launch.h"

namespace kda {

// Blocks of tokens in whose sums the weights' gradients are added up: of 8 tokens at least, so that they are small beside the
// rows (4099 x 12 x 90 fp32, backward call: 18.5 us with 8, 21.6 with 16, 18.5 with 4), and two workgroups for a CU where there is one
// for each (32768 x 16 x 128 in bf16, backward call: 141 us with 512, 148 with 256, 155 with 768 and 164 with 1024).
constexpr int64_t kGnBlocks = 512, kGnBlockTokens = 8;
// the sums of the workspace's blocks
void groupnorm_sums(const GroupNormArgs& a, int64_t blocks, hipStream_t st);

namespace {

constexpr int kGnThreads = 256;

// How a call's tokens and groups lie over workgroups: `groups` groups and `tokens` tokens of each at a time, `block` tokens
// in all, `blocks` of those.
struct GnPlan {
    int groups, tokens;
    int64_t block, blocks;
    bool stream;  // outputs go past the caches
};

typedef uint32_t gn_u32x4 __attribute__((ext_vector_type(4)));
// The empty statements keep the compiler from making one plain store of the two.
template <typename V>
__device__ __forceinline__ void gn_put(void* p, V v, bool stream) {
    if (stream) {
        __asm__ volatile("");
        __builtin_nontemporal_store(v, static_cast<V*>(p));
        __asm__ volatile("");
    } else {
        *static_cast<V*>(p) = v;
    }
}

typedef __bf16 gn_bf16x2 __attribute__((ext_vector_type(2)));
typedef float gn_f32x2 __attribute__((ext_vector_type(2)));

template <int N, bool F32>
struct GnRaw {
    static constexpr int BYTES = N * (F32 ? 4 : 2);
    using Word = std::conditional_t<BYTES >= 16, uint4,
                                    std::conditional_t<BYTES == 8, uint2, std::conditional_t<BYTES == 4, uint32_t, uint16_t>>>;
    Word w[BYTES >= 16 ? BYTES / 16 : 1];
};
template <int N, bool F32>
__device__ __forceinline__ GnRaw<N, F32> gn_load(const void* p, int64_t at) {
    using R = GnRaw<N, F32>;
    R r;
    const typename R::Word* q = reinterpret_cast<const typename R::Word*>(static_cast<const char*>(p) + at * (F32 ? 4 : 2));
#pragma unroll
    for (int i = 0; i < (int)(sizeof(r.w) / sizeof(r.w[0])); ++i) r.w[i] = q[i];
    return r;
}
template <int N, bool F32>
__device__ __forceinline__ void gn_values(const GnRaw<N, F32>& r, float x[N]) {
    if constexpr (N == 1) {
        x[0] = F32 ? __uint_as_float(r.w[0]) : __uint_as_float((uint32_t)r.w[0] << 16);
    } else if constexpr (N == 2 && !F32) {
        x[0] = __uint_as_float(r.w[0] << 16);
        x[1] = __uint_as_float(r.w[0] & 0xffff0000u);
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const uint32_t* u = &r.w[0].x;
            x[j] = F32 ? __uint_as_float(u[j]) : __uint_as_float(j % 2 ? u[j / 2] & 0xffff0000u : u[j / 2] << 16);
        }
    }
}
template <int N, bool F32>
__device__ __forceinline__ void gn_store(void* p, int64_t at, const float x[N], bool stream = false) {
    char* q = static_cast<char*>(p) + at * (F32 ? 4 : 2);
    if constexpr (N == 1) {
        if constexpr (F32) *reinterpret_cast<float*>(q) = x[0];
        else *reinterpret_cast<__bf16*>(q) = (__bf16)x[0];
    } else if constexpr (N == 2) {
        if constexpr (F32) *reinterpret_cast<gn_f32x2*>(q) = gn_f32x2{x[0], x[1]};
        else *reinterpret_cast<gn_bf16x2*>(q) = __builtin_convertvector(gn_f32x2{x[0], x[1]}, gn_bf16x2);
    } else if constexpr (F32) {
#pragma unroll
        for (int i = 0; i < N / 4; ++i)
            *reinterpret_cast<f32x4_t*>(q + 16 * i) = f32x4_t{x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]};
    } else {
#pragma unroll
        for (int i = 0; i < N / 8; ++i) {
            uint32_t u[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                u[j] = __builtin_bit_cast(uint32_t, __builtin_convertvector(gn_f32x2{x[8 * i + 2 * j], x[8 * i + 2 * j + 1]}, gn_bf16x2));
            gn_put(q + 16 * i, gn_u32x4{u[0], u[1], u[2], u[3]}, stream);
        }
    }
}

template <int CTRL>
__device__ __forceinline__ float dpp_take(float x) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xf, 0xf, true));
}
// The sum over each P adjacent lanes, in every one of them.
template <int P>
__device__ __forceinline__ float lanes_sum(float x) {
    x += dpp_take<0xb1>(x);              // the neighbour
    x += dpp_take<0x4e>(x);              // the other pair of four
    if constexpr (P >= 8) x += dpp_take<0x141>(x);   // the other four of eight
    if constexpr (P >= 16) x += dpp_take<0x140>(x);  // the other eight of sixteen
    if constexpr (P >= 32) x += __shfl_xor(x, 16);
    if constexpr (P >= 64) x += __shfl_xor(x, 32);
    return x;
}

// 1 / (1 + e^-u).  CLOSE: e^-u from the product's two halves, so that it keeps 32 bits' accuracy far from zero (the product alone is
// off by |u| 2^-24, which 16-bit outputs do not show; of a backward pass the weights' gradients are always of 32 bits).  Where e^-u
// is infinite already, the rest is of a finite factor, which leaves it so.  Beyond +-100 it is 0 or infinite in 32 bits anyway.  Of a
// NaN, some number.
template <bool CLOSE>
__device__ __forceinline__ float gn_sigmoid(float u) {
    constexpr float l2e = 1.44269502162933349609375f, l2e_rest = 1.925963033500011e-8f, ln2 = 0.693147182464599609375f;
    const float t = __builtin_amdgcn_fmed3f(-u, -100.f, 100.f), hi = t * l2e, e = __builtin_amdgcn_exp2f(hi);
    if constexpr (!CLOSE) return __builtin_amdgcn_rcpf(1.f + e);
    const float lo = fmaf(t, l2e_rest, fmaf(t, l2e, -hi));
    return __builtin_amdgcn_rcpf(1.f + fmaf(fminf(e, 3e38f), lo * ln2, e));
}

// act(u) and its slope; u times the sigmoid, or the sigmoid alone, by selection and not by branches between the values.
template <bool CLOSE, bool SLOPE>
__device__ __forceinline__ void gn_act(float u, bool alone, float& f, float& slope) {
    const float s = gn_sigmoid<CLOSE>(u);
    f = (alone ? (u == u ? 1.f : u) : u) * s;
    if constexpr (SLOPE) slope = fmaf(f, 1.f - s, alone ? 0.f : s);
}

template <bool XF, bool YF, int CPL, int P, int ITER, bool BWD, bool GATE>
__global__ __launch_bounds__(kGnThreads) void groupnorm_kernel(GroupNormArgs a, GnPlan plan) {
    constexpr int N = CPL * ITER;
    const int tid = threadIdx.x, p = tid % P, W = (int)a.width;
    const int gi = tid / P % plan.groups, ti = tid / (P * plan.groups);
    const int64_t group = (int64_t)blockIdx.x * plan.groups + gi, c0 = group * W, C = a.groups * W;
    const bool mine = group < a.groups && ti < plan.tokens, alone = a.act == 2;
    const float mean_of = 1.f / W;
    bool in[ITER];
    int at[ITER];
    float w[N], b[N], dw[N], db[N];
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
        at[i] = (i * P + p) * CPL;
        in[i] = mine && at[i] < W;
        if (!in[i]) at[i] = 0;
#pragma unroll
        for (int j = 0; j < CPL; ++j) {
            w[i * CPL + j] = 1.f;
            b[i * CPL + j] = dw[i * CPL + j] = db[i * CPL + j] = 0.f;
        }
        if (in[i] && a.weight) gn_values<CPL, true>(gn_load<CPL, true>(a.weight, c0 + at[i]), w + i * CPL);
        if (in[i] && a.bias) gn_values<CPL, true>(gn_load<CPL, true>(a.bias, c0 + at[i]), b + i * CPL);
    }
    const int64_t first = (int64_t)blockIdx.y * plan.block;
    const int64_t end = first + plan.block < a.tokens ? first + plan.block : a.tokens;

    // Lanes without a channel, and rows behind the last one, hold zeros: they add nothing to any sum.
    GnRaw<CPL, XF> rx[ITER];
    GnRaw<CPL, YF> rg[ITER], rd[ITER];
    auto fetch = [&](int64_t t) {
#pragma unroll
        for (int i = 0; i < ITER; ++i) {
            rx[i] = {}, rg[i] = {}, rd[i] = {};
            if (!in[i] || t >= end) continue;
            rx[i] = gn_load<CPL, XF>(a.x, t * a.x_stride + c0 + at[i]);
            if constexpr (GATE) rg[i] = gn_load<CPL, YF>(a.gate, t * a.gate_stride + c0 + at[i]);
            if constexpr (BWD) rd[i] = gn_load<CPL, YF>(a.dy, t * C + c0 + at[i]);
        }
    };
    int64_t t = first + ti;
    fetch(t);
    // the loop's count is the workgroup's: every lane takes part in its groups' sums
    for (int64_t t0 = first; t0 < end; t0 += plan.tokens, t += plan.tokens) {
        float x[N], u[N], dy[N];
#pragma unroll
        for (int i = 0; i < ITER; ++i) {
            gn_values<CPL, XF>(rx[i], x + i * CPL);
            if constexpr (GATE) gn_values<CPL, YF>(rg[i], u + i * CPL);
            if constexpr (BWD) gn_values<CPL, YF>(rd[i], dy + i * CPL);
        }
        const bool here = t < end;
        if (t0 + plan.tokens < end) fetch(t + plan.tokens);
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < N; ++k) sum += x[k];
        const float mean = lanes_sum<P>(sum) * mean_of;
        float squares = 0.f;
#pragma unroll
        for (int i = 0; i < ITER; ++i) {
            const float less = in[i] ? mean : 0.f;
#pragma unroll
            for (int j = 0; j < CPL; ++j) {
                float& v = x[i * CPL + j];
                v -= less;
                squares = fmaf(v, v, squares);
            }
        }
        // the square root and the division to the last bit: one each for a row
        float rstd = 1.f / sqrtf(fmaf(lanes_sum<P>(squares), mean_of, a.eps));
        if (!here) rstd = 0.f;  // of a row of zeros it may be infinite
        auto row = [&](auto with) {  // with an activation, or none
            constexpr bool ACT = decltype(with)::value;
            float s1 = 0.f, s2 = 0.f;
#pragma unroll
            for (int k = 0; k < N; ++k) {
                x[k] *= rstd;
                const float z = fmaf(x[k], w[k], b[k]), v = GATE ? u[k] : z;
                float f = v, slope = 1.f;
                if constexpr (ACT) gn_act<YF || BWD, BWD>(v, alone, f, slope);
                if constexpr (!BWD) {
                    x[k] = GATE ? z * f : f;
                } else {
                    if constexpr (GATE) u[k] = dy[k] * z * slope;  // the gate's gradient
                    const float dz = dy[k] * (GATE ? f : slope);
                    dw[k] = fmaf(dz, x[k], dw[k]);
                    db[k] += dz;
                    dy[k] = dz * w[k];
                    s1 += dy[k];
                    s2 = fmaf(dy[k], x[k], s2);
                }
            }
            if constexpr (BWD) {
                s1 = lanes_sum<P>(s1) * mean_of;
                s2 = lanes_sum<P>(s2) * mean_of;
#pragma unroll
                for (int k = 0; k < N; ++k) x[k] = rstd * (dy[k] - fmaf(x[k], s2, s1));
            }
        };
        a.act ? row(std::true_type()) : row(std::false_type());
#pragma unroll
        for (int i = 0; i < ITER; ++i) {
            if (!here || !in[i]) continue;
            if constexpr (BWD) {
                if constexpr (GATE) gn_store<CPL, YF>(a.dgate, t * C + c0 + at[i], u + i * CPL, plan.stream);
                gn_store<CPL, XF>(a.dx, t * C + c0 + at[i], x + i * CPL, plan.stream);
            } else {
                gn_store<CPL, YF>(a.y, t * C + c0 + at[i], x + i * CPL, plan.stream);
            }
        }
    }
    if constexpr (BWD) {
        if (!a.dweight) return;
        // the workgroup's tokens' sums, in the order of its rows
        __shared__ float part[2][kGnThreads * CPL];
        float* out = static_cast<float*>(a.ws) + (int64_t)blockIdx.y * 2 * C;
#pragma unroll
        for (int i = 0; i < ITER; ++i) {
            if (plan.tokens > 1) {
                __syncthreads();
#pragma unroll
                for (int j = 0; j < CPL; ++j) {
                    part[0][j * kGnThreads + tid] = dw[i * CPL + j];
                    part[1][j * kGnThreads + tid] = db[i * CPL + j];
                }
                __syncthreads();
            }
            if (ti || !in[i]) continue;
#pragma unroll
            for (int j = 0; j < CPL; ++j) {
                float sw = dw[i * CPL + j], sb = db[i * CPL + j];
                for (int r = 1; r < plan.tokens; ++r) {
                    sw += part[0][j * kGnThreads + tid + r * P * plan.groups];
                    sb += part[1][j * kGnThreads + tid + r * P * plan.groups];
                }
                out[c0 + at[i] + j] = sw;
                out[C + c0 + at[i] + j] = sb;
            }
        }
    }
}

// Channels that are read at a time: 8 or 2 where every row and its groups begin so, else one (forward and backward in fp32: 15000 x
// 12 x 128 29 and 57 us by eights, 34 and 81 by ones; 4099 x 12 x 90 9.7 and 19 by twos, 12 and 22 by ones).
inline int gn_piece(const GroupNormArgs& a) {
    if (groupnorm_wide(a)) return 8;
    auto odd = [](const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes; };
    const int xb = a.x_f32 ? 8 : 4, yb = a.y_f32 ? 8 : 4;
    return a.width % 2 || a.x_stride % 2 || a.gate_stride % 2 || odd(a.x, xb) || odd(a.dx, xb) || odd(a.gate, yb) || odd(a.y, yb) ||
                   odd(a.dy, yb) || odd(a.dgate, yb) || odd(a.weight, 8) || odd(a.bias, 8)
               ? 1
               : 2;
}

// Lanes and pieces of a row.  Pieces of 8: a lane for each.  Smaller ones: the fewest lanes, 16 at least, that hold the row in four
// pieces each, so that a lane has several loads under way and a row's sums few steps; beyond 64 lanes more pieces.  Against twice the
// lanes of half the pieces, forward and backward of 4.4 million fp32 values four times over: 12 x 42 channels 39 and 70 us for 48 and
// 107, 12 x 90 24 and 47 for 33 and 74, 12 x 126 24 and 43 for 26 and 54; three pieces for four: 12 x 130 31 and 62 for 36 and 70,
// 12 x 258 26 and 50 for 29 and 58; one channel at a time, 12 x 41: 32 and 66 for 47 and 114.
template <typename F>
void gn_shape(int piece, int64_t width, F&& f) {
    auto run = [&](auto cpl, auto p, auto iter) { f(cpl, p, iter); };
    auto i = [](auto v) { return v; };
#define KDA_GN(CPL, P, ITER) \
    run(i(std::integral_constant<int, CPL>()), i(std::integral_constant<int, P>()), i(std::integral_constant<int, ITER>()))
    if (piece == 8) {
        if (width <= 64) KDA_GN(8, 8, 1);
        else if (width <= 128) KDA_GN(8, 16, 1);
        else if (width <= 256) KDA_GN(8, 32, 1);
        else if (width <= 512) KDA_GN(8, 64, 1);
        else if (width <= 1024) KDA_GN(8, 64, 2);
        else KDA_GN(8, 64, 4);
    } else if (piece == 2) {
        if (width <= 32) KDA_GN(2, 16, 1);
        else if (width <= 64) KDA_GN(2, 16, 2);
        else if (width <= 96) KDA_GN(2, 16, 3);
        else if (width <= 128) KDA_GN(2, 16, 4);
        else if (width <= 192) KDA_GN(2, 32, 3);
        else if (width <= 256) KDA_GN(2, 32, 4);
        else if (width <= 384) KDA_GN(2, 64, 3);
        else if (width <= 512) KDA_GN(2, 64, 4);
        else KDA_GN(2, 64, 8);
    } else {
        if (width <= 16) KDA_GN(1, 16, 1);
        else if (width <= 32) KDA_GN(1, 16, 2);
        else if (width <= 48) KDA_GN(1, 16, 3);
        else if (width <= 64) KDA_GN(1, 16, 4);
        else if (width <= 96) KDA_GN(1, 32, 3);
        else if (width <= 128) KDA_GN(1, 32, 4);
        else if (width <= 192) KDA_GN(1, 64, 3);
        else if (width <= 256) KDA_GN(1, 64, 4);
        else if (width <= 512) KDA_GN(1, 64, 8);
        else KDA_GN(1, 64, 16);
    }
#undef KDA_GN
}

// Workgroups of all groups' columns; tokens in blocks, as many workgroups in all as `places`.  A block has kGnBlockTokens at least in a
// backward pass; in a forward one two where workgroups of one each would not fit on the chip at once anyway, so that the second
// one's loads are beside the first one's work (4099 x 12 x 90 fp32: 10.5 -> 9.4 us; 2048 x 16 x 128 fp32, which fit: 8.2 with two, 7.4).
template <bool BWD>
GnPlan gn_plan(const GroupNormArgs& a, int lanes, int64_t places, int64_t& columns) {
    GnPlan p;
    const int64_t fit = kGnThreads / lanes;
    p.groups = (int)(a.groups < fit ? a.groups : fit);
    p.tokens = (int)(fit / p.groups);
    columns = (a.groups + p.groups - 1) / p.groups;
    int64_t blocks = (places + columns - 1) / columns;
    const int64_t at_once = 8 * 256;  // workgroups of 256 threads on 256 CUs
    const int64_t least = BWD ? kGnBlockTokens : columns * ((a.tokens + p.tokens - 1) / p.tokens) > at_once ? 2 : 1;
    const int64_t most = (a.tokens + least - 1) / least;
    if (blocks > most) blocks = most;
    if (blocks < 1) blocks = 1;
    p.block = (a.tokens + blocks - 1) / blocks;
    p.block = (p.block + p.tokens - 1) / p.tokens * p.tokens;
    p.blocks = (a.tokens + p.block - 1) / p.block;
    // 16-bit rows that do not stay in the caches anyway: a store of a wave is whole lines (32768 x 16 x 128: forward from bf16 75 -> 61
    // us, from fp32 95 -> 92).  fp32 rows take two stores of 16 of every 32 bytes, which the caches have to make lines of (the same
    // in fp32, past them and through them: forward 183 and 142, backward 361 and 270).
    p.stream = a.tokens * a.groups * a.width * ((a.x_f32 ? 4 : 2) + (a.y_f32 ? 4 : 2)) >= kStreamBytes;
    return p;
}

}  // namespace

// Workgroups of a forward pass: rows of fp32 have twice the bytes (32768 x 16 x 128, to bf16: from fp32 92 us with 8192, 96 with 4096;
// from bf16 61 with 4096 and 59 with 8192, but 16384 x 12 x 90 22 and 24).
template <bool XF>
constexpr int64_t kGnForward = XF ? 8192 : 4096;

template <bool XF, bool YF, bool BWD>
void groupnorm_launch(const GroupNormArgs& a, hipStream_t st) {
    gn_shape(gn_piece(a), a.width, [&](auto cpl, auto p, auto iter) {
        constexpr int CPL = decltype(cpl)::value, P = decltype(p)::value, ITER = decltype(iter)::value;
        int64_t columns;
        const GnPlan plan = gn_plan<BWD>(a, P, BWD ? kGnBlocks : kGnForward<XF>, columns);
        const dim3 grid((unsigned)columns, (unsigned)plan.blocks);
        if (a.gate) hipLaunchKernelGGL((groupnorm_kernel<XF, YF, CPL, P, ITER, BWD, true>), grid, dim3(kGnThreads), 0, st, a, plan);
        else hipLaunchKernelGGL((groupnorm_kernel<XF, YF, CPL, P, ITER, BWD, false>), grid, dim3(kGnThreads), 0, st, a, plan);
        if (BWD && a.dweight) groupnorm_sums(a, plan.blocks, st);
    });
}

// Rows up to this wide are held in registers.
inline bool gn_in_registers(const GroupNormArgs& a) { return a.width <= (groupnorm_wide(a) ? 2048 : 1024); }
template <bool XF, bool YF>
void groupnorm_fwd_of(const GroupNormArgs& a, hipStream_t st);
template <bool XF, bool YF>
void groupnorm_bwd_of(const GroupNormArgs& a, hipStream_t st);

}  // namespace kda
