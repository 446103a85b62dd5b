// Linear attention with a decay for each head (mathematics and layouts: include/kda_layer.h): a plain form of one token
// after another, for every size and type.
#include "kda_device.h"
#include "kda_layer_launch.h"

namespace kda {

namespace {

// a = e^(min(g, 0)); a NaN stays one.
__device__ __forceinline__ float decay_of(float g) { return expf(g > 0.f ? 0.f : g); }

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

// One of the four recurrences: rows out_t = out_scale * S_t^T a_t with S_t = decay S_(t-1) + in_scale b_t c_t^T, from the
// first token on; or back from the last one, where the state is decayed between its rows' output and the next one's.
struct LinOp {
    const void *a, *b, *c;
    void* out;
    const float* init;
    float* fin;
    bool turned;  // init is the transposed state
    bool back;
    float in_scale, out_scale;
};

template <int DA, bool F32>
__global__ void linattn_plain_kernel(LinOp op, const float* g, const int32_t* cu, int64_t T_fixed, int64_t total, int H, int DC) {
    const int64_t n = blockIdx.x / H;
    const int h = blockIdx.x % H, c = threadIdx.x;
    int64_t begin = n * T_fixed, end = begin + T_fixed;
    if (cu) {
        begin = cu[n] < 0 ? 0 : cu[n] > total ? total : cu[n];
        end = cu[n + 1] < begin ? begin : cu[n + 1] > total ? total : cu[n + 1];
    }
    __shared__ float sa[DA], sb[DA];
    const float decay = decay_of(g[h]);
    float S[DA];
    const int64_t at = (n * H + h) * (int64_t)DA * DC;
#pragma unroll
    for (int i = 0; i < DA; ++i) S[i] = !op.init ? 0.f : op.turned ? op.init[at + (int64_t)c * DA + i] : op.init[at + (int64_t)i * DC + c];
    for (int64_t s = begin; s < end; ++s) {
        const int64_t t = op.back ? end - 1 - (s - begin) : s, row = t * H + h;
        __syncthreads();
        for (int i = c; i < DA; i += DC) {
            sa[i] = load1<F32>(op.a, row * DA + i);
            sb[i] = load1<F32>(op.b, row * DA + i);
        }
        __syncthreads();
        const float x = op.in_scale * load1<F32>(op.c, row * DC + c);
        float o = 0.f;
#pragma unroll
        for (int i = 0; i < DA; ++i) {
            S[i] = op.back ? fmaf(sb[i], x, S[i]) : fmaf(decay, S[i], sb[i] * x);
            o = fmaf(sa[i], S[i], o);
            if (op.back) S[i] *= decay;
        }
        store1<F32>(op.out, row * DC + c, op.out_scale * o);
    }
    if (op.fin)
#pragma unroll
        for (int i = 0; i < DA; ++i) op.fin[at + (int64_t)i * DC + c] = S[i];
}

void plain(const LinArgs& a, const LinOp& op, int DA, int DC, hipStream_t st) {
    const dim3 grid((unsigned)(a.N * a.H)), block(DC);
    auto run = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, st, op, a.g, a.cu, a.T_fixed, a.total, a.H, DC); };
    if (a.f32) DA == 64 ? run(linattn_plain_kernel<64, true>) : run(linattn_plain_kernel<128, true>);
    else DA == 64 ? run(linattn_plain_kernel<64, false>) : run(linattn_plain_kernel<128, false>);
}

// One token.  A workgroup holds one head's state, four columns of RPT rows a thread, and reads and writes it once.
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
    const float decay = decay_of(g[bh % H]);
    const f32x4_t* S = reinterpret_cast<const f32x4_t*>(s_in + bh * (int64_t)DK * DV);
    f32x4_t* So = reinterpret_cast<f32x4_t*>(s_out + bh * (int64_t)DK * DV);
    f32x4_t s[RPT];
#pragma unroll
    for (int m = 0; m < RPT; ++m) s[m] = __builtin_nontemporal_load(&S[(rg + RG * m) * C4 + c4]);
    sq[ti] = qr;
    sk[ti] = kr;
    __syncthreads();
    f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int m = 0; m < RPT; ++m) {
        const int i = rg + RG * m;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            s[m][j] = fmaf(decay, s[m][j], sk[i] * x[j]);
            acc[j] = fmaf(sq[i], s[m][j], acc[j]);
        }
        __builtin_nontemporal_store(s[m], &So[i * C4 + c4]);
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

}  // namespace

int64_t linattn_workspace_bytes(const LinArgs&, bool) { return 0; }
int64_t linattn_groups(const LinArgs& a, bool) { return a.N * a.H; }

hipError_t launch_linattn_fwd(const LinArgs& a, hipStream_t st) {
    plain(a, LinOp{a.q, a.k, a.v, a.o, a.s0, a.s_final, false, false, 1.f, a.scale}, a.Dk, a.Dv, st);
    return hipGetLastError();
}

// dq = scale S d_o: the forward recurrence of the transposed state with d_o, v, k in the places of q, k, v.  dk = dS v
// and dv = dS^T k: the one from the last token back, of dS^T and of dS.
hipError_t launch_linattn_bwd(const LinArgs& a, hipStream_t st) {
    plain(a, LinOp{a.d_o, a.v, a.k, a.dq, a.s0, nullptr, true, false, 1.f, a.scale}, a.Dv, a.Dk, st);
    plain(a, LinOp{a.v, a.d_o, a.q, a.dk, a.d_sfinal, nullptr, true, true, a.scale, 1.f}, a.Dv, a.Dk, st);
    plain(a, LinOp{a.k, a.q, a.d_o, a.dv, a.d_sfinal, a.ds0, false, true, a.scale, 1.f}, a.Dk, a.Dv, st);
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
    using I64 = std::integral_constant<int, 64>;
    using I128 = std::integral_constant<int, 128>;
    if (a.Dk == 64) a.Dv == 64 ? types(I64(), I64()) : types(I64(), I128());
    else a.Dv == 64 ? types(I128(), I64()) : types(I128(), I128());
    return hipGetLastError();
}

}  // namespace kda
