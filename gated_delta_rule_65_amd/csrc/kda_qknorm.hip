// Norm of queries and keys per head with the position rotation in the same pass, forward and backward
// (mathematics and layouts: include/kda_layer.h).
#include "kda_ckpt8.h"
#include "kda_layer_launch.h"

namespace kda {

namespace {

// The two chunks of eight channels that a lane of a row holds, such that both channels of every pair that is
// turned are in one lane: lane j of D/16 holds channels first(j) .. +7 and second(j) .. +7.  In halves,
// pair i is (i, i + rot/2); with adjacent pairs, and behind the turned channels, sixteen in a row.
struct Place {
    int first, second;
    bool turned;
    int pair;  // the first of the lane's eight pairs
};
__device__ __forceinline__ Place place_of(int j, int rot, bool interleaved) {
    const bool t = j < rot / 16;
    if (t && !interleaved) return {8 * j, rot / 2 + 8 * j, true, 8 * j};
    return {16 * j, 16 * j + 8, t, 8 * j};
}

template <bool F32>
__device__ __forceinline__ void load8(const void* p, int64_t i, float x[8]) {
    if constexpr (F32) {
        const float4* s = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
        const float4 u = s[0], v = s[1];
        x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
        x[4] = v.x; x[5] = v.y; x[6] = v.z; x[7] = v.w;
    } else {
        const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            x[2 * k] = __uint_as_float(u[k] << 16);
            x[2 * k + 1] = __uint_as_float(u[k] & 0xffff0000u);
        }
    }
}
template <bool F32>
__device__ __forceinline__ void store8(void* p, int64_t i, const float x[8]) {
    if constexpr (F32) {
        float4* d = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
        d[0] = make_float4(x[0], x[1], x[2], x[3]);
        d[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
        typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
        bf8 w;
#pragma unroll
        for (int k = 0; k < 8; ++k) w[k] = (__bf16)x[k];
        *reinterpret_cast<bf8*>(static_cast<uint16_t*>(p) + i) = w;
    }
}
// Eight packed values of one block.
__device__ __forceinline__ void load8_packed(const uint8_t* codes, int64_t i, int scale, float x[8]) {
    const uint2 w = *reinterpret_cast<const uint2*>(codes + i);
    x[0] = ckpt_value<0>(w.x, scale); x[1] = ckpt_value<1>(w.x, scale);
    x[2] = ckpt_value<2>(w.x, scale); x[3] = ckpt_value<3>(w.x, scale);
    x[4] = ckpt_value<0>(w.y, scale); x[5] = ckpt_value<1>(w.y, scale);
    x[6] = ckpt_value<2>(w.y, scale); x[7] = ckpt_value<3>(w.y, scale);
}

// Cosine and sine of pos * freq radians.  The product is taken in 64 bits and reduced to a fraction of a turn
// there, so that far positions keep float32's accuracy.
__device__ __forceinline__ void turn(double pos, double freq, float& c, float& s) {
    constexpr double inv_2pi = 0.15915494309189533577;
    const double t = pos * (freq * inv_2pi);
    sincospif(2.f * (float)(t - rint(t)), &s, &c);
}
// z = (x0 c - x1 s, x1 c + x0 s) on the lane's eight pairs; sign -1 turns back.
__device__ __forceinline__ void turn8(float a[8], float b[8], const float c[8], const float s[8], bool interleaved,
                                      float sign) {
    if (!interleaved) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float x = a[k], y = b[k], t = sign * s[k];
            a[k] = x * c[k] - y * t;
            b[k] = y * c[k] + x * t;
        }
        return;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        float x = a[2 * k], y = a[2 * k + 1], t = sign * s[k];
        a[2 * k] = x * c[k] - y * t;
        a[2 * k + 1] = y * c[k] + x * t;
        x = b[2 * k], y = b[2 * k + 1], t = sign * s[k + 4];
        b[2 * k] = x * c[k + 4] - y * t;
        b[2 * k + 1] = y * c[k + 4] + x * t;
    }
}

template <int LANES>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int off = LANES / 2; off > 0; off >>= 1) v += __shfl_xor(v, off);
    return v;
}

// (s |x|^2 + eps)^(-1/2) of a row, 0 where that is 0.  Rows whose sum of squares leaves float32's comfortable
// range are summed again at a power of two of their own size.
template <int LANES>
__device__ __forceinline__ float row_rsqrt(const float a[8], const float b[8], float s, float eps) {
    float ss = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) ss = fmaf(a[k], a[k], fmaf(b[k], b[k], ss));
    ss = row_sum<LANES>(ss);
    if (ss > 0x1p-100f && ss < 0x1p100f) return __builtin_amdgcn_rsqf(fmaf(ss, s, eps));
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        top = max(top, abs_bits(a[k]));
        top = max(top, abs_bits(b[k]));
    }
#pragma unroll
    for (int off = LANES / 2; off > 0; off >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, off));
    if (top >= kInfBits) return __uint_as_float(0x7fc00000u);  // a row that holds infinity or NaN has no norm
    if (top == 0) return eps > 0.f ? rsqrtf(eps) : 0.f;
    int e;
    frexpf(__uint_as_float(top), &e);
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const float u = ldexpf(a[k], -e), v = ldexpf(b[k], -e);
        sum = fmaf(u, u, fmaf(v, v, sum));
    }
    sum = row_sum<LANES>(sum);
    const double total = (double)sum * s * ldexp(1.0, 2 * e) + eps;
    return total < 0x1p-252 ? 0.f : (float)(1.0 / sqrt(total));
}

// A row (token, head) to D/16 lanes.
template <int D, bool F32, bool PACKED>
__global__ __launch_bounds__(256) void qknorm_fwd_kernel(QkArgs a) {
    constexpr int LANES = D / 16;
    const int H = a.Hq + a.Hk;
    const int64_t rows = a.tokens * H;
    const int j = threadIdx.x % LANES;
    const Place p = place_of(j, a.rot, a.interleaved);
    for (int64_t row = (int64_t)blockIdx.x * (256 / LANES) + threadIdx.x / LANES; row < rows;
         row += (int64_t)gridDim.x * (256 / LANES)) {
        const int64_t t = row / H;
        int h = (int)(row - t * H);
        const bool key = h >= a.Hq;
        if (key) h -= a.Hq;
        const void* src = key ? a.k : a.q;
        const int64_t in = t * (key ? a.k_stride : a.q_stride) + h * D;
        const int64_t out = (t * (key ? a.Hk : a.Hq) + h) * D;
        float x0[8], x1[8];
        if constexpr (PACKED) {
            const uint8_t* sc = (key ? a.ks : a.qs) + out / kCkptBlock;
            load8_packed(static_cast<const uint8_t*>(src), in + p.first, sc[p.first / kCkptBlock], x0);
            load8_packed(static_cast<const uint8_t*>(src), in + p.second, sc[p.second / kCkptBlock], x1);
        } else {
            load8<F32>(src, in + p.first, x0);
            load8<F32>(src, in + p.second, x1);
        }
        if constexpr (!PACKED) {
            if (a.q8) {
                // the lanes that share a block are not neighbours in halves; each takes its block's largest
                // magnitude over the whole row's exchange
                uint32_t m0 = 0, m1 = 0;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    m0 = max(m0, finite_abs_bits(x0[k]));
                    m1 = max(m1, finite_abs_bits(x1[k]));
                }
                uint32_t top[D / kCkptBlock] = {};
#pragma unroll
                for (int b = 0; b < D / kCkptBlock; ++b) {
                    if (p.first / kCkptBlock == b) top[b] = m0;
                    if (p.second / kCkptBlock == b) top[b] = max(top[b], m1);
#pragma unroll
                    for (int off = LANES / 2; off > 0; off >>= 1)
                        top[b] = max(top[b], (uint32_t)__shfl_xor((int)top[b], off));
                }
                uint8_t* codes = (key ? a.k8 : a.q8) + out;
                uint8_t* sc = (key ? a.k8s : a.q8s) + out / kCkptBlock;
#pragma unroll
                for (int b = 0; b < D / kCkptBlock; ++b) {
                    const int s = ckpt_scale(top[b]);
                    const float inv = ckpt_inverse(s);
                    if (j == b) sc[b] = (uint8_t)s;
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const int at = half ? p.second : p.first;
                        const float* x = half ? x1 : x0;
                        if (at / kCkptBlock == b) {
                            uint2 w;
                            w.x = ckpt_code2(x[0], x[1], inv) | ckpt_code2(x[2], x[3], inv) << 16;
                            w.y = ckpt_code2(x[4], x[5], inv) | ckpt_code2(x[6], x[7], inv) << 16;
                            *reinterpret_cast<uint2*>(codes + at) = w;
                        }
                    }
                }
            }
        }
        const float r = row_rsqrt<LANES>(x0, x1, a.rms ? 1.f / D : 1.f, a.eps);
        const float* w = key ? a.wk : a.wq;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            x0[k] *= r * (w ? w[p.first + k] : 1.f);
            x1[k] *= r * (w ? w[p.second + k] : 1.f);
        }
        if (p.turned) {
            const double pos = a.pos64 ? (double)static_cast<const int64_t*>(a.pos)[t]
                                       : (double)static_cast<const int32_t*>(a.pos)[t];
            float c[8], s[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) turn(pos, a.freqs[p.pair + k], c[k], s[k]);
            turn8(x0, x1, c, s, a.interleaved, 1.f);
        }
        void* dst = key ? a.k_out : a.q_out;
        store8<F32>(dst, out + p.first, x0);
        store8<F32>(dst, out + p.second, x1);
    }
}

// Gradients of the rows; a workgroup's sums for the weights go to its line of the workspace.
template <int D, bool F32, bool PACKED, bool GF32>
__global__ __launch_bounds__(256) void qknorm_bwd_kernel(QkArgs a) {
    constexpr int LANES = D / 16, ROWS = 256 / LANES;
    __shared__ float part[ROWS][D];
    const int H = a.Hq + a.Hk;
    const int j = threadIdx.x % LANES;
    const Place p = place_of(j, a.rot, a.interleaved);
    float* line = static_cast<float*>(a.ws) + (int64_t)blockIdx.x * 2 * D;
    for (int side = 0; side < 2; ++side) {
        const int Hs = side ? a.Hk : a.Hq;
        const int64_t rows = a.tokens * Hs;
        const void* src = side ? a.k : a.q;
        const void* grad = side ? a.d_k : a.d_q;
        const float* w = side ? a.wk : a.wq;
        float dw0[8] = {}, dw1[8] = {};
        for (int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / LANES; row < rows;
             row += (int64_t)gridDim.x * ROWS) {
            const int64_t t = row / Hs;
            const int h = (int)(row - t * Hs);
            const int64_t in = t * (side ? a.k_stride : a.q_stride) + h * D, out = row * D;
            float x0[8], x1[8], d0[8], d1[8];
            if constexpr (PACKED) {
                const uint8_t* sc = (side ? a.ks : a.qs) + out / kCkptBlock;
                load8_packed(static_cast<const uint8_t*>(src), in + p.first, sc[p.first / kCkptBlock], x0);
                load8_packed(static_cast<const uint8_t*>(src), in + p.second, sc[p.second / kCkptBlock], x1);
            } else {
                load8<F32>(src, in + p.first, x0);
                load8<F32>(src, in + p.second, x1);
            }
            load8<GF32>(grad, out + p.first, d0);
            load8<GF32>(grad, out + p.second, d1);
            const float sc = a.rms ? 1.f / D : 1.f;
            const float r = row_rsqrt<LANES>(x0, x1, sc, a.eps);
            if (p.turned) {
                const double pos = a.pos64 ? (double)static_cast<const int64_t*>(a.pos)[t]
                                           : (double)static_cast<const int32_t*>(a.pos)[t];
                float c[8], s[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) turn(pos, a.freqs[p.pair + k], c[k], s[k]);
                turn8(d0, d1, c, s, a.interleaved, -1.f);
            }
            float dot = 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                x0[k] *= r;
                x1[k] *= r;
                dw0[k] = fmaf(d0[k], x0[k], dw0[k]);
                dw1[k] = fmaf(d1[k], x1[k], dw1[k]);
                d0[k] *= w ? w[p.first + k] : 1.f;
                d1[k] *= w ? w[p.second + k] : 1.f;
                dot = fmaf(d0[k], x0[k], fmaf(d1[k], x1[k], dot));
            }
            dot = row_sum<LANES>(dot) * sc;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                x0[k] = r * fmaf(-dot, x0[k], d0[k]);
                x1[k] = r * fmaf(-dot, x1[k], d1[k]);
            }
            void* dst = side ? a.dk : a.dq;
            store8<F32>(dst, out + p.first, x0);
            store8<F32>(dst, out + p.second, x1);
        }
        if (a.dwq) {
            float* mine = part[threadIdx.x / LANES];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                mine[p.first + k] = dw0[k];
                mine[p.second + k] = dw1[k];
            }
            __syncthreads();
            if (threadIdx.x < D) {
                float sum = 0.f;
                for (int i = 0; i < ROWS; ++i) sum += part[i][threadIdx.x];
                line[side * D + threadIdx.x] = sum;
            }
            __syncthreads();
        }
    }
}

// The workgroups' lines added up in their order.
__global__ __launch_bounds__(256) void qknorm_dw_kernel(const float* __restrict__ lines, int count, int D,
                                                        float* __restrict__ dwq, float* __restrict__ dwk) {
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c >= 2 * D) return;
    float sum = 0.f;
    for (int i = 0; i < count; ++i) sum += lines[(int64_t)i * 2 * D + c];
    if (c < D) dwq[c] = sum;
    else dwk[c - D] = sum;
}

constexpr int kBwdGroups = 1024;
int bwd_groups(int64_t tokens, int Hq, int Hk, int D) {
    const int64_t need = (tokens * (Hq > Hk ? Hq : Hk) + 4095 / D) / (4096 / D);
    return (int)(need < kBwdGroups ? need : kBwdGroups);
}

}  // namespace

int64_t qknorm_bwd_workspace_bytes(int64_t tokens, int Hq, int Hk, int D) {
    return (int64_t)bwd_groups(tokens, Hq, Hk, D) * 2 * D * 4;
}

hipError_t launch_qknorm_fwd(const QkArgs& a, hipStream_t st) {
    const int64_t groups = (a.tokens * (a.Hq + a.Hk) + 4096 / a.D - 1) / (4096 / a.D);
    const dim3 grid((unsigned)(groups < 16384 ? groups : 16384)), block(256);
    const bool packed = a.qs != nullptr;
#define KDA_FWD(DIM)                                                                                          \
    if (a.f32 && packed) hipLaunchKernelGGL((qknorm_fwd_kernel<DIM, true, true>), grid, block, 0, st, a);     \
    else if (a.f32) hipLaunchKernelGGL((qknorm_fwd_kernel<DIM, true, false>), grid, block, 0, st, a);         \
    else if (packed) hipLaunchKernelGGL((qknorm_fwd_kernel<DIM, false, true>), grid, block, 0, st, a);        \
    else hipLaunchKernelGGL((qknorm_fwd_kernel<DIM, false, false>), grid, block, 0, st, a);
    if (a.D == 128) {
        KDA_FWD(128)
    } else {
        KDA_FWD(64)
    }
#undef KDA_FWD
    return hipGetLastError();
}

template <int D, bool GF32>
static void launch_bwd_types(const QkArgs& a, int groups, hipStream_t st) {
    const dim3 grid((unsigned)groups), block(256);
    const bool packed = a.qs != nullptr;
    if (a.f32 && packed) hipLaunchKernelGGL((qknorm_bwd_kernel<D, true, true, GF32>), grid, block, 0, st, a);
    else if (a.f32) hipLaunchKernelGGL((qknorm_bwd_kernel<D, true, false, GF32>), grid, block, 0, st, a);
    else if (packed) hipLaunchKernelGGL((qknorm_bwd_kernel<D, false, true, GF32>), grid, block, 0, st, a);
    else hipLaunchKernelGGL((qknorm_bwd_kernel<D, false, false, GF32>), grid, block, 0, st, a);
}

hipError_t launch_qknorm_bwd(const QkArgs& a, hipStream_t st) {
    const int groups = bwd_groups(a.tokens, a.Hq, a.Hk, a.D);
    if (groups == 0) {  // no tokens: only the weights' zero gradients are written
    } else if (a.D == 128) a.grad_f32 ? launch_bwd_types<128, true>(a, groups, st) : launch_bwd_types<128, false>(a, groups, st);
    else a.grad_f32 ? launch_bwd_types<64, true>(a, groups, st) : launch_bwd_types<64, false>(a, groups, st);
    if (a.dwq)
        hipLaunchKernelGGL(qknorm_dw_kernel, dim3((unsigned)((2 * a.D + 255) / 256)), dim3(256), 0, st,
                           static_cast<const float*>(a.ws), groups, a.D, a.dwq, a.dwk);
    return hipGetLastError();
}

}  // namespace kda
