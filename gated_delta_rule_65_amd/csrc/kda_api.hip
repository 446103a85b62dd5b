// C ABI of the library (declared in include/kda.h): host-side validation,
// error reporting and dispatch to the gfx950 kernels on the caller's stream.
#include <hip/hip_runtime.h>

#include <cstdarg>
#include <cstdio>
#include <mutex>
#include <string>

#include "kda.h"
#include "kda_layer.h"
#include "kda_layer_launch.h"
#include "kda_launch.h"

namespace {

thread_local std::string g_last_error;

kda_status fail(kda_status st, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    g_last_error = buf;
    return st;
}

kda_status ok() {
    g_last_error.clear();
    return KDA_OK;
}

kda_status check_head_dims(int H, int Dk, int Dv) {
    if (H < 1 || H > 65536) return fail(KDA_ERR_BAD_SHAPE, "H must be in [1, 65536] (got %d)", H);
    if (Dk != 64 && Dk != 128) return fail(KDA_ERR_BAD_SHAPE, "Dk must be 64 or 128 (got %d)", Dk);
    if (Dv != 64 && Dv != 128) return fail(KDA_ERR_BAD_SHAPE, "Dv must be 64 or 128 (got %d)", Dv);
    return KDA_OK;
}

kda_status check_dtype(kda_dtype dt) {
    if (dt != KDA_F32 && dt != KDA_BF16) return fail(KDA_ERR_BAD_DTYPE, "dtype must be KDA_F32 or KDA_BF16");
    return KDA_OK;
}

struct Ptr {
    const void* p;
    const char* name;
    bool required;
    int align = 16;
};

kda_status check_ptrs(std::initializer_list<Ptr> ptrs) {
    for (const Ptr& x : ptrs) {
        if (x.required && !x.p) return fail(KDA_ERR_NULL_ARG, "%s is NULL", x.name);
        if (reinterpret_cast<uintptr_t>(x.p) % x.align)
            return fail(KDA_ERR_MISALIGNED, "%s is not %d-byte aligned", x.name, x.align);
    }
    return KDA_OK;
}

kda_status read_prologue(const kda_prologue* p, kda::Prologue& out) {
    out = kda::Prologue{false, false, false, false, false};
    if (!p) return KDA_OK;
    if (p->g_dtype != KDA_F32 && p->g_dtype != KDA_BF16)
        return fail(KDA_ERR_BAD_DTYPE, "prologue g_dtype must be KDA_F32 or KDA_BF16");
    if (p->beta_dtype != KDA_F32 && p->beta_dtype != KDA_BF16)
        return fail(KDA_ERR_BAD_DTYPE, "prologue beta_dtype must be KDA_F32 or KDA_BF16");
    out.g_bf16 = p->g_dtype == KDA_BF16;
    out.g_logit = p->g_logit != 0;
    out.b_bf16 = p->beta_dtype == KDA_BF16;
    out.b_logit = p->beta_logit != 0;
    out.l2norm = p->qk_l2norm != 0;
    return KDA_OK;
}

kda_status launched(hipError_t e, const char* what) {
    if (e != hipSuccess) return fail(KDA_ERR_HIP, "%s launch failed: %s", what, hipGetErrorString(e));
    return ok();
}

kda_status run_chunked(const kda::ChunkArgs& a, void* workspace, size_t workspace_bytes, hipStream_t st,
                       const char* what) {
    const int64_t grid = kda::chunk_grid_size(a.N, a.H, a.Dv);
    if (grid > 0x7fffffff) return fail(KDA_ERR_BAD_SHAPE, "%s: %lld sequence-heads exceed the grid limit", what,
                                       (long long)(a.N * a.H));
    if (grid == 0) return ok();
    // without tokens there is nothing to prepare (the workspace size queries return 0 then): the
    // fused kernel passes s0 (or zeros) through to s_final
    if (!workspace || a.total == 0) return launched(kda::launch_chunk_fwd(a, st), what);
    if (kda::chunk_slots(a) * a.H > 0x7fffffffLL)
        return fail(KDA_ERR_BAD_SHAPE, "%s: %lld chunk-heads exceed the grid limit", what,
                    (long long)(kda::chunk_slots(a) * a.H));
    const int64_t need = kda::chunk_workspace_bytes(a);
    if ((uint64_t)need > (uint64_t)workspace_bytes)
        return fail(KDA_ERR_BAD_SHAPE, "%s: workspace holds %llu bytes, %lld needed", what,
                    (unsigned long long)workspace_bytes, (long long)need);
    return launched(kda::launch_chunk_fwd_two_pass(a, workspace, st), what);
}

// ---------------------------------------------------------------------------- fixed scratch
// Device memory of kda_chunk_fwd_noalloc, for callers that cannot allocate: the per-window records
// of the two-kernel path (and the carried state when s_final is NULL).  Every GPU that runs the
// library holds its own copy for the life of the process.  Its address on a device comes from
// hipGetSymbolAddress, looked up once per device with that device current; host code uses only that
// address, never the array's name (which on the host is a stand-in, not a device address).
constexpr int64_t kScratchBytes = int64_t(128) << 20;
static __device__ __align__(256) char scratch[kScratchBytes];

constexpr int kMaxDevices = 64;
std::mutex g_scratch_mu;
void* g_scratch_ptr[kMaxDevices] = {};

kda_status scratch_of_current_device(void** out, const char* what) {
    int dev = -1;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return fail(KDA_ERR_HIP, "%s: hipGetDevice failed: %s", what, hipGetErrorString(e));
    if (dev < 0 || dev >= kMaxDevices) return fail(KDA_ERR_HIP, "%s: device %d out of range", what, dev);
    std::lock_guard<std::mutex> lock(g_scratch_mu);
    if (!g_scratch_ptr[dev]) {
        void* p = nullptr;
        e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
        if (e != hipSuccess || !p)
            return fail(KDA_ERR_HIP, "%s: hipGetSymbolAddress(scratch) failed on device %d: %s", what, dev,
                        hipGetErrorString(e));
        g_scratch_ptr[dev] = p;
    }
    *out = g_scratch_ptr[dev];
    return KDA_OK;
}

// ---------------------------------------------------------------------------- kda_layer.h checks
bool overlap(const void* a, const void* b, int64_t a_bytes, int64_t b_bytes) {
    const char *p = static_cast<const char*>(a), *q = static_cast<const char*>(b);
    return p && q && p < q + b_bytes && q < p + a_bytes;
}

constexpr int64_t kMostElements = int64_t(1) << 40;  // of a tensor: byte offsets stay far inside 64 bits

kda_status check_ckpt8(int64_t rows, int64_t cols, kda_dtype dtype) {
    kda_status st;
    if ((st = check_dtype(dtype)) != KDA_OK) return st;
    if (rows < 0 || cols < 0) return fail(KDA_ERR_BAD_SHAPE, "rows and cols must be >= 0");
    if (cols > 0 && rows > kMostElements / cols) return fail(KDA_ERR_BAD_SHAPE, "rows*cols exceeds 2^40");
    if (cols > 0x7fffffff) return fail(KDA_ERR_BAD_SHAPE, "cols must be below 2^31");
    if (cols % 8 == 0 && rows * ((cols + 31) / 32) > kda::kMaxThreads - 256)  // a thread a block of 32 values
        return fail(KDA_ERR_BAD_SHAPE, "rows*ceil(cols/32) exceeds the grid limit");
    return KDA_OK;
}

// Rows that no wide load divides are read a value at a time and may begin at any.
kda_status ckpt8_ptrs(const void* x, const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, kda_dtype dtype) {
    const bool any = rows > 0 && cols > 0;
    const int value = cols % 8 == 0 ? 16 : dtype == KDA_F32 ? 4 : 2, byte = cols % 8 == 0 ? 16 : 1;
    return check_ptrs({{x, "x", any, value}, {codes, "codes", any, byte}, {scales, "scales", any, byte}});
}

bool scan_sizes(int64_t N, int64_t total, int64_t D) {
    return N >= 1 && N <= 0x7fffffff && total >= 0 && D >= 1 && D <= kda::kMaxChannels && total <= kMostElements / D &&
           N <= kMostElements / D;
}

kda_status scan_batch(kda::ScanArgs& a, int64_t B, int64_t T) {
    if (B < 0 || T < 0) return fail(KDA_ERR_BAD_SHAPE, "B and T must be >= 0");
    if (T > 0 && B > kMostElements / T) return fail(KDA_ERR_BAD_SHAPE, "B*T exceeds 2^40");
    a.N = B;
    a.T_fixed = T;
    a.total = B * T;
    return KDA_OK;
}

kda_status scan_packed(kda::ScanArgs& a, const int32_t* cu, int64_t N, int64_t total) {
    if (N < 0 || total < 0) return fail(KDA_ERR_BAD_SHAPE, "N and total must be >= 0");
    if (total > 0x7fffffffLL) return fail(KDA_ERR_BAD_SHAPE, "total exceeds the int32 range of cu_seqlens");
    if (N > 0 && !cu) return fail(KDA_ERR_NULL_ARG, "cu_seqlens is NULL");
    if (reinterpret_cast<uintptr_t>(cu) & 3u) return fail(KDA_ERR_MISALIGNED, "cu_seqlens is not 4-byte aligned");
    a.cu = cu;
    a.N = N;
    a.total = total;
    return KDA_OK;
}

kda_status scan_form(kda::ScanArgs& a, int64_t D, const kda_scan_form* f) {
    if (!f) return fail(KDA_ERR_NULL_ARG, "form is NULL");
    if ((f->x_dtype != KDA_F32 && f->x_dtype != KDA_BF16) || (f->g_dtype != KDA_F32 && f->g_dtype != KDA_BF16))
        return fail(KDA_ERR_BAD_DTYPE, "form x_dtype and g_dtype must be KDA_F32 or KDA_BF16");
    if (D < 1) return fail(KDA_ERR_BAD_SHAPE, "D must be >= 1 (got %lld)", (long long)D);
    if (a.N > 0 && !scan_sizes(a.N, a.total, D))
        return fail(KDA_ERR_BAD_SHAPE, "sizes out of range: %lld sequences, %lld tokens, D = %lld", (long long)a.N,
                    (long long)a.total, (long long)D);
    a.D = D;
    a.x_f32 = f->x_dtype == KDA_F32;
    a.g_f32 = f->g_dtype == KDA_F32;
    a.logit = f->g_logit != 0;
    a.complement = f->complement != 0;
    return KDA_OK;
}

kda_status scan_ws(kda::ScanArgs& a, void* ws, size_t bytes, const char* what) {
    if (kda::scan_places(a) > kda::kMaxThreads / kda::kScanThreads)
        return fail(KDA_ERR_BAD_SHAPE, "%s: %lld tokens of %lld channels exceed the grid limit", what,
                    (long long)a.total, (long long)a.D);
    const int64_t need = a.total ? kda::scan_workspace_bytes(a.N, a.total, a.D) : 0;
    if (need > 0 && !ws)
        return fail(KDA_ERR_NULL_ARG, "%s: workspace is NULL (%lld bytes needed)", what, (long long)need);
    if ((uint64_t)need > (uint64_t)bytes)
        return fail(KDA_ERR_BAD_SHAPE, "%s: workspace holds %llu bytes, %lld needed", what, (unsigned long long)bytes,
                    (long long)need);
    a.ws = ws;
    return KDA_OK;
}

// What a scan's rows are aligned to: 16 bytes, or an element where they are read one at a time.
struct ScanAlign {
    int x, g, state, code;
    ScanAlign(const kda::ScanArgs& a, int64_t together) {
        const bool wide = together % 4 == 0;
        x = wide ? 16 : a.x_f32 ? 4 : 2;
        g = wide ? 16 : a.g_f32 ? 4 : 2;
        state = wide ? 16 : 4;
        code = wide ? 16 : 1;
    }
};

kda_status scan_fwd(kda::ScanArgs& a, const void* x, const void* g, const float* h0, void* y, float* h_final,
                    float* carry, uint8_t* u, uint8_t* us, void* ws, size_t ws_bytes, void* stream, const char* what) {
    kda_status st;
    const bool tokens = a.N > 0 && a.total > 0, save = tokens && (u || us);
    const ScanAlign to(a, a.D);
    if ((st = check_ptrs({{x, "x", tokens, to.x}, {g, "g", tokens, to.g}, {y, "y", tokens, to.x},
                          {h0, "h0", false, to.state}, {h_final, "h_final", false, to.state},
                          {carry, "carry", false, to.state}, {u, "u_codes", save, to.code},
                          {us, "u_scales", save, to.code}, {ws, "workspace", false}})) != KDA_OK)
        return st;
    if (overlap(h0, h_final, a.N * a.D * 4, a.N * a.D * 4))
        return fail(KDA_ERR_BAD_SHAPE, "%s: h_final must not overlap h0", what);
    if (a.N == 0 || (!tokens && !h_final)) return ok();
    if ((st = scan_ws(a, ws, ws_bytes, what)) != KDA_OK) return st;
    a.x = x;
    a.g = g;
    a.h0 = h0;
    a.y = y;
    a.h_final = h_final;
    a.carry_out = carry;
    a.u_out = u;
    a.us_out = us;
    return launched(kda::launch_scan_fwd(a, static_cast<hipStream_t>(stream)), what);
}

kda_status scan_bwd(kda::ScanArgs& a, const void* x, const void* g, const float* h0, const float* carry,
                    const uint8_t* u, const uint8_t* us, const void* dy, const float* dh_final, void* dx, void* dg,
                    float* dh0, void* ws, size_t ws_bytes, void* stream, const char* what) {
    kda_status st;
    const bool tokens = a.N > 0 && a.total > 0, packed = u || us, need_u = tokens && packed;
    const bool need_x = tokens && !packed;
    if (need_x && !(x && carry))
        return fail(KDA_ERR_NULL_ARG, "%s: either x and carry or u_codes and u_scales must be given", what);
    const ScanAlign to(a, a.D);
    if ((st = check_ptrs({{x, "x", false, to.x}, {g, "g", tokens, to.g}, {dy, "dy", tokens, to.x},
                          {dx, "dx", tokens, to.x}, {dg, "dg", tokens, to.g}, {h0, "h0", false, to.state},
                          {carry, "carry", false, to.state}, {u, "u_codes", need_u, to.code},
                          {us, "u_scales", need_u, to.code}, {dh_final, "dh_final", false, to.state},
                          {dh0, "dh0", false, to.state}, {ws, "workspace", false}})) != KDA_OK)
        return st;
    if (overlap(dh0, dh_final, a.N * a.D * 4, a.N * a.D * 4) || overlap(dh0, h0, a.N * a.D * 4, a.N * a.D * 4))
        return fail(KDA_ERR_BAD_SHAPE, "%s: dh0 must not overlap dh_final or h0", what);
    if (a.N == 0 || (!tokens && !dh0)) return ok();
    if ((st = scan_ws(a, ws, ws_bytes, what)) != KDA_OK) return st;
    a.x = x;
    a.g = g;
    a.h0 = h0;
    a.carry = carry;
    a.u = u;
    a.us = us;
    a.dy = dy;
    a.dh_final = dh_final;
    a.dx = dx;
    a.dg = dg;
    a.dh0 = dh0;
    return launched(kda::launch_scan_bwd(a, static_cast<hipStream_t>(stream)), what);
}

kda_status qk_inputs(kda::QkArgs& a, const void* q, const void* k, const uint8_t* qs, const uint8_t* ks,
                     int64_t q_stride, int64_t k_stride, const float* wq, const float* wk, const void* pos,
                     const double* freqs, int64_t tokens, int Hq, int Hk, int D, kda_dtype dtype,
                     const kda_qknorm_form* f) {
    kda_status st;
    if ((st = check_dtype(dtype)) != KDA_OK) return st;
    if (!f) return fail(KDA_ERR_NULL_ARG, "form is NULL");
    if (Hq < 1 || Hq > 65536 || Hk < 1 || Hk > 65536)
        return fail(KDA_ERR_BAD_SHAPE, "Hq and Hk must be in [1, 65536] (got %d, %d)", Hq, Hk);
    if (D != 64 && D != 128) return fail(KDA_ERR_BAD_SHAPE, "D must be 64 or 128 (got %d)", D);
    if (tokens < 0) return fail(KDA_ERR_BAD_SHAPE, "tokens must be >= 0");
    if (f->norm != KDA_NORM_L2 && f->norm != KDA_NORM_RMS)
        return fail(KDA_ERR_BAD_SHAPE, "norm must be KDA_NORM_L2 or KDA_NORM_RMS");
    if (!(f->eps >= 0.f) || f->eps > 3.0e38f) return fail(KDA_ERR_BAD_SHAPE, "eps must be finite and >= 0");
    if (f->rot < 0 || f->rot > D || f->rot % 16)
        return fail(KDA_ERR_BAD_SHAPE, "rot must be a multiple of 16 in [0, D] (got %d)", f->rot);
    if (f->rot && f->pos_bytes != 4 && f->pos_bytes != 8)
        return fail(KDA_ERR_BAD_DTYPE, "pos_bytes must be 4 or 8 (got %d)", f->pos_bytes);
    const int64_t nq = (int64_t)Hq * D, nk = (int64_t)Hk * D, unit = dtype == KDA_F32 ? 4 : 8;
    if (qs || ks) {
        if (q_stride != nq || k_stride != nk)
            return fail(KDA_ERR_BAD_SHAPE, "packed q and k are contiguous: strides must be Hq*D and Hk*D");
    } else if (q_stride < nq || k_stride < nk || q_stride % unit || k_stride % unit) {
        return fail(KDA_ERR_BAD_SHAPE, "q_stride and k_stride must be at least Hq*D and Hk*D and multiples of 16 bytes");
    }
    const int64_t wide = q_stride > k_stride ? q_stride : k_stride;
    if (tokens > kMostElements / (wide > nq + nk ? wide : nq + nk))
        return fail(KDA_ERR_BAD_SHAPE, "q and k exceed 2^40 elements");
    const bool any = tokens > 0, packed = any && (qs || ks), turned = any && f->rot > 0;
    if ((st = check_ptrs({{q, "q", any}, {k, "k", any}, {qs, "q_scales", packed}, {ks, "k_scales", packed},
                          {wq, "wq", false}, {wk, "wk", false}, {pos, "pos", turned, f->rot ? f->pos_bytes : 1},
                          {freqs, "freqs", turned, f->rot ? 8 : 1}})) != KDA_OK)
        return st;
    a.q = q;
    a.k = k;
    a.qs = qs;
    a.ks = ks;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.wq = wq;
    a.wk = wk;
    a.pos = pos;
    a.freqs = freqs;
    a.tokens = tokens;
    a.Hq = Hq;
    a.Hk = Hk;
    a.D = D;
    a.rot = f->rot;
    a.f32 = dtype == KDA_F32;
    a.rms = f->norm == KDA_NORM_RMS;
    a.interleaved = f->interleaved != 0;
    a.pos64 = f->pos_bytes == 8;
    a.eps = f->eps;
    return KDA_OK;
}

// ---------------------------------------------------------------------------- linear attention
kda_status lin_sizes(kda::LinArgs& a, int64_t N, int64_t total, int H, int Dk, int Dv, float scale, kda_dtype dtype) {
    kda_status st;
    if ((st = check_dtype(dtype)) != KDA_OK) return st;
    if ((st = check_head_dims(H, Dk, Dv)) != KDA_OK) return st;
    const int64_t most = kMostElements / H / 128;
    if (N > most / 128 || total > most)
        return fail(KDA_ERR_BAD_SHAPE, "sizes out of range: %lld sequences, %lld tokens, H = %d", (long long)N,
                    (long long)total, H);
    a.N = N;
    a.total = total;
    a.H = H;
    a.Dk = Dk;
    a.Dv = Dv;
    a.scale = scale;
    a.f32 = dtype == KDA_F32;
    return KDA_OK;
}

kda_status lin_batch(kda::LinArgs& a, int64_t B, int64_t T, int H, int Dk, int Dv, float scale, kda_dtype dtype) {
    if (B < 0 || T < 0) return fail(KDA_ERR_BAD_SHAPE, "B and T must be >= 0");
    if (T > 0 && B > kMostElements / T) return fail(KDA_ERR_BAD_SHAPE, "B*T exceeds 2^40");
    a.T_fixed = T;
    return lin_sizes(a, B, B * T, H, Dk, Dv, scale, dtype);
}

kda_status lin_packed(kda::LinArgs& a, const int32_t* cu, int64_t N, int64_t total, int H, int Dk, int Dv, float scale,
                      kda_dtype dtype) {
    if (N < 0 || total < 0) return fail(KDA_ERR_BAD_SHAPE, "N and total must be >= 0");
    if (total > 0x7fffffffLL) return fail(KDA_ERR_BAD_SHAPE, "total exceeds the int32 range of cu_seqlens");
    if (N > 0 && !cu) return fail(KDA_ERR_NULL_ARG, "cu_seqlens is NULL");
    if (reinterpret_cast<uintptr_t>(cu) & 3u) return fail(KDA_ERR_MISALIGNED, "cu_seqlens is not 4-byte aligned");
    a.cu = cu;
    return lin_sizes(a, N, total, H, Dk, Dv, scale, dtype);
}

kda_status lin_ws(kda::LinArgs& a, bool backward, void* ws, size_t bytes, const char* what) {
    if (kda::linattn_threads(a, backward) > kda::kMaxThreads)
        return fail(KDA_ERR_BAD_SHAPE, "%s: %lld tokens of %lld sequences and %d heads exceed the grid limit", what,
                    (long long)a.total, (long long)a.N, a.H);
    const int64_t need = kda::linattn_workspace_bytes(a, backward);
    if (need > 0 && !ws)
        return fail(KDA_ERR_NULL_ARG, "%s: workspace is NULL (%lld bytes needed)", what, (long long)need);
    if ((uint64_t)need > (uint64_t)bytes)
        return fail(KDA_ERR_BAD_SHAPE, "%s: workspace holds %llu bytes, %lld needed", what, (unsigned long long)bytes,
                    (long long)need);
    a.ws = ws;
    return KDA_OK;
}

kda_status lin_fwd(kda::LinArgs& a, const void* q, const void* k, const void* v, const float* g, const float* s0, void* o,
                   float* s_final, void* ws, size_t ws_bytes, void* stream, const char* what) {
    kda_status st;
    const bool tokens = a.N > 0 && a.total > 0;
    const int64_t states = a.N * a.H * a.Dk * a.Dv * 4;
    if ((st = check_ptrs({{q, "q", tokens}, {k, "k", tokens}, {v, "v", tokens}, {g, "g", tokens, 4}, {o, "o", tokens},
                          {s0, "s0", false}, {s_final, "s_final", false}, {ws, "workspace", false}})) != KDA_OK)
        return st;
    if (overlap(s0, s_final, states, states)) return fail(KDA_ERR_BAD_SHAPE, "%s: s_final must not overlap s0", what);
    if (a.N == 0 || (!tokens && !s_final)) return ok();
    if ((st = lin_ws(a, false, ws, ws_bytes, what)) != KDA_OK) return st;
    a.q = q;
    a.k = k;
    a.v = v;
    a.g = g;
    a.s0 = s0;
    a.o = o;
    a.s_final = s_final;
    return launched(kda::launch_linattn_fwd(a, static_cast<hipStream_t>(stream)), what);
}

kda_status lin_bwd(kda::LinArgs& a, const void* q, const void* k, const void* v, const float* g, const float* s0,
                   const void* d_o, const float* d_sfinal, void* dq, void* dk, void* dv, float* ds0, void* ws,
                   size_t ws_bytes, void* stream, const char* what) {
    kda_status st;
    const bool tokens = a.N > 0 && a.total > 0;
    const int64_t states = a.N * a.H * a.Dk * a.Dv * 4;
    if ((st = check_ptrs({{q, "q", tokens}, {k, "k", tokens}, {v, "v", tokens}, {g, "g", tokens, 4},
                          {d_o, "d_o", tokens}, {dq, "dq", tokens}, {dk, "dk", tokens}, {dv, "dv", tokens},
                          {s0, "s0", false}, {d_sfinal, "d_sfinal", false}, {ds0, "ds0", false},
                          {ws, "workspace", false}})) != KDA_OK)
        return st;
    if (overlap(d_sfinal, ds0, states, states) || overlap(s0, ds0, states, states))
        return fail(KDA_ERR_BAD_SHAPE, "%s: ds0 must not overlap s0 or d_sfinal", what);
    if (a.N == 0 || (!tokens && !ds0)) return ok();
    if ((st = lin_ws(a, true, ws, ws_bytes, what)) != KDA_OK) return st;
    a.q = q;
    a.k = k;
    a.v = v;
    a.g = g;
    a.s0 = s0;
    a.d_o = d_o;
    a.d_sfinal = d_sfinal;
    a.dq = dq;
    a.dk = dk;
    a.dv = dv;
    a.ds0 = ds0;
    return launched(kda::launch_linattn_bwd(a, static_cast<hipStream_t>(stream)), what);
}

size_t lin_workspace_bytes(int64_t N, int64_t total, int H, int Dk, int Dv, kda_dtype dtype, bool backward) {
    kda::LinArgs a{};
    if (N < 1 || total < 1) return 0;
    if (H < 1 || H > 65536 || (Dk != 64 && Dk != 128) || (Dv != 64 && Dv != 128)) return 0;
    if ((dtype != KDA_F32 && dtype != KDA_BF16) || N > kMostElements / H / 128 / 128 || total > kMostElements / H / 128) return 0;
    a.N = N;
    a.total = total;
    a.H = H;
    a.Dk = Dk;
    a.Dv = Dv;
    a.f32 = dtype == KDA_F32;
    return (size_t)kda::linattn_workspace_bytes(a, backward);
}

// ---------------------------------------------------------------------------- group norm
kda_status gn_inputs(kda::GroupNormArgs& a, const void* x, int64_t x_stride, const float* weight, const float* bias,
                     const void* gate, int64_t gate_stride, int64_t tokens, int64_t groups, int64_t width,
                     const kda_groupnorm_form* f) {
    kda_status st;
    if (!f) return fail(KDA_ERR_NULL_ARG, "form is NULL");
    if ((f->x_dtype != KDA_F32 && f->x_dtype != KDA_BF16) || (f->y_dtype != KDA_F32 && f->y_dtype != KDA_BF16))
        return fail(KDA_ERR_BAD_DTYPE, "form x_dtype and y_dtype must be KDA_F32 or KDA_BF16");
    if (f->act != KDA_ACT_NONE && f->act != KDA_ACT_SILU && f->act != KDA_ACT_SIGMOID)
        return fail(KDA_ERR_BAD_SHAPE, "form act must be KDA_ACT_NONE, KDA_ACT_SILU or KDA_ACT_SIGMOID (got %d)", f->act);
    if (!(f->eps >= 0.f)) return fail(KDA_ERR_BAD_SHAPE, "form eps must be >= 0");
    if (tokens < 0) return fail(KDA_ERR_BAD_SHAPE, "tokens must be >= 0");
    if (groups < 1 || groups > kda::kMaxChannels) return fail(KDA_ERR_BAD_SHAPE, "groups must be in [1, 2^24]");
    if (width < 1 || width > kda::kMaxGroupWidth) return fail(KDA_ERR_BAD_SHAPE, "width must be in [1, 2^16]");
    const int64_t C = groups * width;
    if (C > kda::kMaxChannels) return fail(KDA_ERR_BAD_SHAPE, "groups*width exceeds 2^24");
    if (x_stride < C || (gate && gate_stride < C))
        return fail(KDA_ERR_BAD_SHAPE, "x_stride and gate_stride must be at least groups*width");
    if (x_stride > kMostElements || (gate && gate_stride > kMostElements) ||
        (tokens > 0 && tokens > kMostElements / (gate && gate_stride > x_stride ? gate_stride : x_stride)))
        return fail(KDA_ERR_BAD_SHAPE, "tokens times a stride exceeds 2^40");
    a.x = x;
    a.gate = gate;
    a.x_stride = x_stride;
    a.gate_stride = gate ? gate_stride : C;
    a.weight = weight;
    a.bias = bias;
    a.tokens = tokens;
    a.groups = groups;
    a.width = width;
    a.x_f32 = f->x_dtype == KDA_F32;
    a.y_f32 = f->y_dtype == KDA_F32;
    a.act = f->act;
    a.eps = f->eps;
    return check_ptrs({{x, "x", tokens > 0, a.x_f32 ? 4 : 2}, {gate, "gate", false, a.y_f32 ? 4 : 2}, {weight, "weight", false, 4},
                       {bias, "bias", false, 4}});
}

// With all of the call's pointers, which decide on its kernel.
kda_status gn_grid(const kda::GroupNormArgs& a) {
    if (kda::groupnorm_groups(a) > kda::kMaxThreads / 256)
        return fail(KDA_ERR_BAD_SHAPE, "%lld tokens of %lld groups exceed the grid limit", (long long)a.tokens, (long long)a.groups);
    return KDA_OK;
}

}  // namespace

extern "C" {

kda_status kda_chunk_fwd_noalloc(const void* q, const void* k, const void* v, const void* g, const void* beta,
                                 const float* s0, float* o, float* s_final, int64_t B, int64_t T, int H, int Dk,
                                 int Dv, int chunk, kda_dtype dtype, const kda_prologue* prologue, void* stream) {
    const char* what = "kda_chunk_fwd_noalloc";
    kda_status st;
    kda::Prologue pro;
    if ((st = check_dtype(dtype)) != KDA_OK) return st;
    if ((st = read_prologue(prologue, pro)) != KDA_OK) return st;
    if ((st = check_head_dims(H, Dk, Dv)) != KDA_OK) return st;
    if (chunk != 64) return fail(KDA_ERR_BAD_SHAPE, "chunk must be 64 (got %d)", chunk);
    if (B < 0 || T < 0) return fail(KDA_ERR_BAD_SHAPE, "B and T must be >= 0");
    if (T > 0 && B > INT64_MAX / T) return fail(KDA_ERR_BAD_SHAPE, "B*T overflows");
    const bool tokens = B > 0 && T > 0;
    if ((st = check_ptrs({{q, "q", tokens}, {k, "k", tokens}, {v, "v", tokens}, {g, "g", tokens},
                          {beta, "beta", tokens}, {o, "o", tokens}, {s0, "s0", false},
                          {s_final, "s_final", false}})) != KDA_OK)
        return st;
    if (B == 0 || (!tokens && !s_final)) return ok();
    kda::ChunkArgs a{q, k, v, g, beta, s0, o, s_final, nullptr, T, B * T, B, H, Dk, Dv, dtype == KDA_F32, pro};
    const int64_t grid = kda::chunk_grid_size(a.N, a.H, a.Dv);
    if (grid > 0x7fffffff) return fail(KDA_ERR_BAD_SHAPE, "%s: %lld sequence-heads exceed the grid limit", what,
                                       (long long)(a.N * a.H));
    hipStream_t hs = static_cast<hipStream_t>(stream);
    if (!tokens) return launched(kda::launch_chunk_fwd(a, hs), what);  // s0 (or zeros) to s_final, no scratch
    if (kda::chunk_window_chunks(a, kScratchBytes) < 1)
        return fail(KDA_ERR_BAD_SHAPE,
                    "%s: B*H = %lld sequence-heads need %lld bytes of scratch for one 64-token window; the fixed "
                    "scratch holds %lld",
                    what, (long long)(a.N * a.H),
                    (long long)(kda::chunk_window_state_bytes(a) + kda::chunk_workspace_bytes(
                        kda::ChunkArgs{q, k, v, g, beta, s0, o, s_final, nullptr, 64, B * 64, B, H, Dk, Dv,
                                       dtype == KDA_F32, pro})),
                    (long long)kScratchBytes);
    void* base = nullptr;
    if ((st = scratch_of_current_device(&base, what)) != KDA_OK) return st;
    return launched(kda::launch_chunk_fwd_windows(a, static_cast<char*>(base), kScratchBytes, hs), what);
}

kda_status kda_chunk_fwd(const void* q, const void* k, const void* v, const void* g, const void* beta,
                         const float* s0, float* o, float* s_final, int64_t B, int64_t T, int H, int Dk, int Dv,
                         int chunk, kda_dtype dtype, const kda_prologue* prologue, void* workspace,
                         size_t workspace_bytes, void* stream) {
    kda_status st;
    kda::Prologue pro;
    if ((st = check_dtype(dtype)) != KDA_OK) return st;
    if ((st = read_prologue(prologue, pro)) != KDA_OK) return st;
    if ((st = check_head_dims(H, Dk, Dv)) != KDA_OK) return st;
    if (chunk != 64) return fail(KDA_ERR_BAD_SHAPE, "chunk must be 64 (got %d)", chunk);
    if (B < 0 || T < 0) return fail(KDA_ERR_BAD_SHAPE, "B and T must be >= 0");
    if (T > 0 && B > INT64_MAX / T) return fail(KDA_ERR_BAD_SHAPE, "B*T overflows");
    const bool tokens = B > 0 && T > 0;
    if ((st = check_ptrs({{q, "q", tokens}, {k, "k", tokens}, {v, "v", tokens}, {g, "g", tokens},
                          {beta, "beta", tokens}, {o, "o", tokens}, {s0, "s0", false},
                          {s_final, "s_final", false}, {workspace, "workspace", false}})) != KDA_OK)
        return st;
    if (B == 0 || (!tokens && !s_final)) return ok();
    kda::ChunkArgs a{q, k, v, g, beta, s0, o, s_final, nullptr, T, B * T, B, H, Dk, Dv, dtype == KDA_F32, pro};
    return run_chunked(a, workspace, workspace_bytes, static_cast<hipStream_t>(stream), "kda_chunk_fwd");
}

kda_status kda_varlen_fwd(const void* q, const void* k, const void* v, const void* g, const void* beta,
                          const int32_t* cu_seqlens, int64_t N, int64_t total, const float* s0, float* o,
                          float* s_final, int H, int Dk, int Dv, int chunk, kda_dtype dtype,
                          const kda_prologue* prologue, void* workspace, size_t workspace_bytes, void* stream) {
    kda_status st;
    kda::Prologue pro;
    if ((st = check_dtype(dtype)) != KDA_OK) return st;
    if ((st = read_prologue(prologue, pro)) != KDA_OK) return st;
    if ((st = check_head_dims(H, Dk, Dv)) != KDA_OK) return st;
    if (chunk != 64) return fail(KDA_ERR_BAD_SHAPE, "chunk must be 64 (got %d)", chunk);
    if (N < 0 || total < 0) return fail(KDA_ERR_BAD_SHAPE, "N and total must be >= 0");
    if (total > 0x7fffffffLL) return fail(KDA_ERR_BAD_SHAPE, "total exceeds the int32 range of cu_seqlens");
    const bool tokens = total > 0;
    if (N > 0 && !cu_seqlens) return fail(KDA_ERR_NULL_ARG, "cu_seqlens is NULL");
    if ((st = check_ptrs({{q, "q", tokens}, {k, "k", tokens}, {v, "v", tokens}, {g, "g", tokens},
                          {beta, "beta", tokens}, {o, "o", tokens}, {s0, "s0", false},
                          {s_final, "s_final", false}, {workspace, "workspace", false}})) != KDA_OK)
        return st;
    if (N == 0 || (!tokens && !s_final)) return ok();
    kda::ChunkArgs a{q, k, v, g, beta, s0, o, s_final, cu_seqlens, 0, total, N, H, Dk, Dv, dtype == KDA_F32, pro};
    return run_chunked(a, workspace, workspace_bytes, static_cast<hipStream_t>(stream), "kda_varlen_fwd");
}

kda_status kda_decode_step(const void* q, const void* k, const void* v, const void* g, const void* beta,
                           const float* s_in, float* s_out, float* o, int64_t B, int H, int Dk, int Dv,
                           kda_dtype dtype, const kda_prologue* prologue, void* stream) {
    kda_status st;
    kda::Prologue pro;
    if ((st = check_dtype(dtype)) != KDA_OK) return st;
    if ((st = read_prologue(prologue, pro)) != KDA_OK) return st;
    if ((st = check_head_dims(H, Dk, Dv)) != KDA_OK) return st;
    if (B < 0) return fail(KDA_ERR_BAD_SHAPE, "B must be >= 0");
    if (B * H > 0x7fffffffLL) return fail(KDA_ERR_BAD_SHAPE, "B*H exceeds the grid limit");
    const bool any = B > 0;
    if ((st = check_ptrs({{q, "q", any}, {k, "k", any}, {v, "v", any}, {g, "g", any}, {beta, "beta", any},
                          {s_in, "s_in", any}, {s_out, "s_out", any}, {o, "o", any}})) != KDA_OK)
        return st;
    if (s_in != s_out && s_in && s_out) {
        const char* a0 = reinterpret_cast<const char*>(s_in);
        const char* b0 = reinterpret_cast<const char*>(s_out);
        const int64_t bytes = B * H * (int64_t)Dk * Dv * 4;
        if (a0 < b0 + bytes && b0 < a0 + bytes)
            return fail(KDA_ERR_BAD_SHAPE, "s_in and s_out overlap without being the same buffer");
    }
    if (!any) return ok();
    kda::DecodeArgs a{q, k, v, g, beta, s_in, s_out, o, B, H, Dk, Dv, dtype == KDA_F32, pro};
    return launched(kda::launch_decode(a, static_cast<hipStream_t>(stream)), "kda_decode_step");
}

static kda_status run_bwd(const kda::BwdArgs& a, void* workspace, size_t workspace_bytes, hipStream_t st,
                          const char* what) {
    if (a.N * (int64_t)a.H > 0x7fffffffLL / 4)
        return fail(KDA_ERR_BAD_SHAPE, "%s: %lld sequence-heads exceed the grid limit", what, (long long)(a.N * a.H));
    if (kda::bwd_slots(a) * a.H > 0x7fffffffLL)
        return fail(KDA_ERR_BAD_SHAPE, "%s: %lld chunk-heads exceed the grid limit", what,
                    (long long)(kda::bwd_slots(a) * a.H));
    const int64_t need = kda::bwd_workspace_bytes(a);
    if (need > 0 && !workspace) return fail(KDA_ERR_NULL_ARG, "%s: workspace is NULL (%lld bytes needed)", what,
                                            (long long)need);
    if ((uint64_t)need > (uint64_t)workspace_bytes)
        return fail(KDA_ERR_BAD_SHAPE, "%s: workspace holds %llu bytes, %lld needed", what,
                    (unsigned long long)workspace_bytes, (long long)need);
    return launched(kda::launch_bwd(a, workspace, st), what);
}

kda_status kda_chunk_bwd(const void* q, const void* k, const void* v, const float* g, const float* beta,
                         const float* s0, const float* d_o, const float* d_sfinal, float* dq, float* dk, float* dv,
                         float* dg, float* dbeta, float* ds0, int64_t B, int64_t T, int H, int Dk, int Dv, int chunk,
                         kda_dtype dtype, void* workspace, size_t workspace_bytes, void* stream) {
    kda_status st;
    if ((st = check_dtype(dtype)) != KDA_OK) return st;
    if ((st = check_head_dims(H, Dk, Dv)) != KDA_OK) return st;
    if (chunk != 64) return fail(KDA_ERR_BAD_SHAPE, "chunk must be 64 (got %d)", chunk);
    if (B < 0 || T < 0) return fail(KDA_ERR_BAD_SHAPE, "B and T must be >= 0");
    if (T > 0 && B > INT64_MAX / T) return fail(KDA_ERR_BAD_SHAPE, "B*T overflows");
    const bool tokens = B > 0 && T > 0;
    if ((st = check_ptrs({{q, "q", tokens}, {k, "k", tokens}, {v, "v", tokens}, {g, "g", tokens},
                          {beta, "beta", tokens}, {d_o, "d_o", tokens}, {dq, "dq", tokens}, {dk, "dk", tokens},
                          {dv, "dv", tokens}, {dg, "dg", tokens}, {dbeta, "dbeta", tokens}, {s0, "s0", false},
                          {d_sfinal, "d_sfinal", false}, {ds0, "ds0", false}, {workspace, "workspace", false}})) !=
        KDA_OK)
        return st;
    if (B == 0 || (!tokens && !ds0)) return ok();
    kda::BwdArgs a{q, k, v, g, beta, s0, d_o, d_sfinal, dq, dk, dv, dg, dbeta, ds0, nullptr, T, B * T, B, H, Dk, Dv,
                   dtype == KDA_F32};
    return run_bwd(a, workspace, workspace_bytes, static_cast<hipStream_t>(stream), "kda_chunk_bwd");
}

kda_status kda_varlen_bwd(const void* q, const void* k, const void* v, const float* g, const float* beta,
                          const int32_t* cu_seqlens, int64_t N, int64_t total, const float* s0, const float* d_o,
                          const float* d_sfinal, float* dq, float* dk, float* dv, float* dg, float* dbeta, float* ds0,
                          int H, int Dk, int Dv, int chunk, kda_dtype dtype, void* workspace, size_t workspace_bytes,
                          void* stream) {
    kda_status st;
    if ((st = check_dtype(dtype)) != KDA_OK) return st;
    if ((st = check_head_dims(H, Dk, Dv)) != KDA_OK) return st;
    if (chunk != 64) return fail(KDA_ERR_BAD_SHAPE, "chunk must be 64 (got %d)", chunk);
    if (N < 0 || total < 0) return fail(KDA_ERR_BAD_SHAPE, "N and total must be >= 0");
    if (total > 0x7fffffffLL) return fail(KDA_ERR_BAD_SHAPE, "total exceeds the int32 range of cu_seqlens");
    const bool tokens = total > 0;
    if (N > 0 && !cu_seqlens) return fail(KDA_ERR_NULL_ARG, "cu_seqlens is NULL");
    if ((st = check_ptrs({{q, "q", tokens}, {k, "k", tokens}, {v, "v", tokens}, {g, "g", tokens},
                          {beta, "beta", tokens}, {d_o, "d_o", tokens}, {dq, "dq", tokens}, {dk, "dk", tokens},
                          {dv, "dv", tokens}, {dg, "dg", tokens}, {dbeta, "dbeta", tokens}, {s0, "s0", false},
                          {d_sfinal, "d_sfinal", false}, {ds0, "ds0", false}, {workspace, "workspace", false}})) !=
        KDA_OK)
        return st;
    if (N == 0 || (!tokens && !ds0)) return ok();
    kda::BwdArgs a{q, k, v, g, beta, s0, d_o, d_sfinal, dq, dk, dv, dg, dbeta, ds0, cu_seqlens, 0, total, N, H, Dk,
                   Dv, dtype == KDA_F32};
    return run_bwd(a, workspace, workspace_bytes, static_cast<hipStream_t>(stream), "kda_varlen_bwd");
}

size_t kda_chunk_bwd_workspace_bytes(int64_t B, int64_t T, int H, int Dk, int Dv, kda_dtype dtype) {
    if (B <= 0 || T < 0 || H < 1 || (Dk != 64 && Dk != 128) || (Dv != 64 && Dv != 128)) return 0;
    if (dtype != KDA_F32 && dtype != KDA_BF16) return 0;
    kda::BwdArgs a{};
    a.f32 = dtype == KDA_F32;
    a.T_fixed = T;
    a.N = B;
    a.total = B * T;
    a.H = H;
    a.Dk = Dk;
    a.Dv = Dv;
    return (size_t)kda::bwd_workspace_bytes(a);
}

size_t kda_varlen_bwd_workspace_bytes(int64_t N, int64_t total, int H, int Dk, int Dv, kda_dtype dtype) {
    if (N <= 0 || total < 0 || H < 1 || (Dk != 64 && Dk != 128) || (Dv != 64 && Dv != 128)) return 0;
    if (dtype != KDA_F32 && dtype != KDA_BF16) return 0;
    kda::BwdArgs a{};
    a.f32 = dtype == KDA_F32;
    static const int32_t dummy = 0;
    a.cu_seqlens = &dummy;  // only its presence matters for the size
    a.N = N;
    a.total = total;
    a.H = H;
    a.Dk = Dk;
    a.Dv = Dv;
    return (size_t)kda::bwd_workspace_bytes(a);
}

size_t kda_chunk_workspace_bytes(int64_t B, int64_t T, int H, int Dk, int Dv, kda_dtype dtype) {
    if (B <= 0 || T <= 0 || H < 1 || (Dk != 64 && Dk != 128) || (Dv != 64 && Dv != 128)) return 0;
    if (dtype != KDA_F32 && dtype != KDA_BF16) return 0;
    kda::ChunkArgs a{};
    a.f32 = dtype == KDA_F32;
    a.T_fixed = T;
    a.N = B;
    a.total = B * T;
    a.H = H;
    a.Dk = Dk;
    a.Dv = Dv;
    return (size_t)kda::chunk_workspace_bytes(a);
}

size_t kda_varlen_workspace_bytes(int64_t N, int64_t total, int H, int Dk, int Dv, kda_dtype dtype) {
    if (N <= 0 || total <= 0 || H < 1 || (Dk != 64 && Dk != 128) || (Dv != 64 && Dv != 128)) return 0;
    if (dtype != KDA_F32 && dtype != KDA_BF16) return 0;
    kda::ChunkArgs a{};
    a.f32 = dtype == KDA_F32;
    static const int32_t dummy = 0;
    a.cu_seqlens = &dummy;  // only its presence matters for the size
    a.N = N;
    a.total = total;
    a.H = H;
    a.Dk = Dk;
    a.Dv = Dv;
    return (size_t)kda::chunk_workspace_bytes(a);
}

// ---------------------------------------------------------------------------- kda_layer.h

kda_status kda_ckpt8_pack(const void* x, uint8_t* codes, uint8_t* scales, int64_t rows, int64_t cols,
                          kda_dtype dtype, void* stream) {
    kda_status st;
    if ((st = check_ckpt8(rows, cols, dtype)) != KDA_OK) return st;
    const bool any = rows > 0 && cols > 0;
    if ((st = ckpt8_ptrs(x, codes, scales, rows, cols, dtype)) != KDA_OK) return st;
    if (!any) return ok();
    return launched(kda::launch_ckpt8_pack(x, codes, scales, rows, cols, dtype == KDA_F32,
                                           static_cast<hipStream_t>(stream)), "kda_ckpt8_pack");
}

kda_status kda_ckpt8_unpack(const uint8_t* codes, const uint8_t* scales, void* x, int64_t rows, int64_t cols,
                            kda_dtype dtype, void* stream) {
    kda_status st;
    if ((st = check_ckpt8(rows, cols, dtype)) != KDA_OK) return st;
    const bool any = rows > 0 && cols > 0;
    if ((st = ckpt8_ptrs(x, codes, scales, rows, cols, dtype)) != KDA_OK) return st;
    if (!any) return ok();
    return launched(kda::launch_ckpt8_unpack(codes, scales, x, rows, cols, dtype == KDA_F32,
                                             static_cast<hipStream_t>(stream)), "kda_ckpt8_unpack");
}

kda_status kda_scan_fwd(const void* x, const void* g, const float* h0, void* y, float* h_final, float* carry,
                        uint8_t* u_codes, uint8_t* u_scales, int64_t B, int64_t T, int64_t D,
                        const kda_scan_form* form, void* workspace, size_t workspace_bytes, void* stream) {
    kda_status st;
    kda::ScanArgs a{};
    if ((st = scan_batch(a, B, T)) != KDA_OK || (st = scan_form(a, D, form)) != KDA_OK) return st;
    return scan_fwd(a, x, g, h0, y, h_final, carry, u_codes, u_scales, workspace, workspace_bytes, stream,
                    "kda_scan_fwd");
}

kda_status kda_scan_varlen_fwd(const void* x, const void* g, const int32_t* cu_seqlens, int64_t N, int64_t total,
                               const float* h0, void* y, float* h_final, float* carry, uint8_t* u_codes,
                               uint8_t* u_scales, int64_t D, const kda_scan_form* form, void* workspace,
                               size_t workspace_bytes, void* stream) {
    kda_status st;
    kda::ScanArgs a{};
    if ((st = scan_packed(a, cu_seqlens, N, total)) != KDA_OK || (st = scan_form(a, D, form)) != KDA_OK) return st;
    return scan_fwd(a, x, g, h0, y, h_final, carry, u_codes, u_scales, workspace, workspace_bytes, stream,
                    "kda_scan_varlen_fwd");
}

kda_status kda_scan_bwd(const void* x, const void* g, const float* h0, const float* carry, const uint8_t* u_codes,
                        const uint8_t* u_scales, const void* dy, const float* dh_final, void* dx, void* dg,
                        float* dh0, int64_t B, int64_t T, int64_t D, const kda_scan_form* form, void* workspace,
                        size_t workspace_bytes, void* stream) {
    kda_status st;
    kda::ScanArgs a{};
    if ((st = scan_batch(a, B, T)) != KDA_OK || (st = scan_form(a, D, form)) != KDA_OK) return st;
    return scan_bwd(a, x, g, h0, carry, u_codes, u_scales, dy, dh_final, dx, dg, dh0, workspace, workspace_bytes,
                    stream, "kda_scan_bwd");
}

kda_status kda_scan_varlen_bwd(const void* x, const void* g, const int32_t* cu_seqlens, int64_t N, int64_t total,
                               const float* h0, const float* carry, const uint8_t* u_codes, const uint8_t* u_scales,
                               const void* dy, const float* dh_final, void* dx, void* dg, float* dh0, int64_t D,
                               const kda_scan_form* form, void* workspace, size_t workspace_bytes, void* stream) {
    kda_status st;
    kda::ScanArgs a{};
    if ((st = scan_packed(a, cu_seqlens, N, total)) != KDA_OK || (st = scan_form(a, D, form)) != KDA_OK) return st;
    return scan_bwd(a, x, g, h0, carry, u_codes, u_scales, dy, dh_final, dx, dg, dh0, workspace, workspace_bytes,
                    stream, "kda_scan_varlen_bwd");
}

kda_status kda_scan_zero_behind(const int32_t* cu_seqlens, int64_t N, int64_t total, void* a, int64_t a_row_bytes,
                                void* b, int64_t b_row_bytes, void* stream) {
    kda_status st;
    if (N < 0 || total < 0) return fail(KDA_ERR_BAD_SHAPE, "N and total must be >= 0");
    if (N > 0x7fffffffLL || total > 0x7fffffffLL)
        return fail(KDA_ERR_BAD_SHAPE, "N or total exceeds the int32 range of cu_seqlens");
    if (!b) b_row_bytes = 0;
    for (const int64_t row : {a_row_bytes, b_row_bytes})
        if (row < 0 || row % 2 || row > kda::kMaxChannels * 4)
            return fail(KDA_ERR_BAD_SHAPE, "row bytes must be even and in [0, 4 * 2^24] (got %lld)", (long long)row);
    const bool any = total > 0 && (a_row_bytes > 0 || b_row_bytes > 0);
    if (any && !cu_seqlens) return fail(KDA_ERR_NULL_ARG, "cu_seqlens is NULL");
    if (reinterpret_cast<uintptr_t>(cu_seqlens) & 3u) return fail(KDA_ERR_MISALIGNED, "cu_seqlens is not 4-byte aligned");
    if ((st = check_ptrs({{a, "a", any}, {b, "b", false}})) != KDA_OK) return st;
    if (!any) return ok();
    return launched(kda::launch_scan_zero_behind(cu_seqlens, N, total, a, a_row_bytes, b, b_row_bytes,
                                                 static_cast<hipStream_t>(stream)), "kda_scan_zero_behind");
}

kda_status kda_scan_step(const void* x, const void* g, const float* h_in, float* h_out, void* y, int64_t B,
                         int64_t D, const kda_scan_form* form, void* stream) {
    kda_status st;
    kda::ScanArgs a{};
    if ((st = scan_batch(a, B, 1)) != KDA_OK || (st = scan_form(a, D, form)) != KDA_OK) return st;
    if (B * D / (B * D % 4 ? 1 : 4) > kda::kMaxThreads - 256) return fail(KDA_ERR_BAD_SHAPE, "B*D exceeds the grid limit");
    const bool any = B > 0;
    const ScanAlign to(a, B * D);
    if ((st = check_ptrs({{x, "x", any, to.x}, {g, "g", any, to.g}, {h_in, "h_in", any, to.state},
                          {h_out, "h_out", any, to.state}, {y, "y", any, to.x}})) != KDA_OK)
        return st;
    if (h_in != h_out && overlap(h_in, h_out, B * D * 4, B * D * 4))
        return fail(KDA_ERR_BAD_SHAPE, "h_in and h_out overlap without being the same buffer");
    if (!any) return ok();
    a.x = x;
    a.g = g;
    a.y = y;
    return launched(kda::launch_scan_step(a, h_in, h_out, static_cast<hipStream_t>(stream)), "kda_scan_step");
}

size_t kda_scan_workspace_bytes(int64_t N, int64_t total, int64_t D) {
    if (!scan_sizes(N, total, D) || total == 0) return 0;
    return (size_t)kda::scan_workspace_bytes(N, total, D);
}

size_t kda_scan_carry_bytes(int64_t N, int64_t total, int64_t D) {
    if (!scan_sizes(N, total, D) || total == 0) return 0;
    return (size_t)(kda::scan_most_segments(N, total) * D * 4);
}

kda_status kda_qknorm_fwd(const void* q, const void* k, const uint8_t* q_scales, const uint8_t* k_scales,
                          int64_t q_stride, int64_t k_stride, const float* wq, const float* wk, const void* pos,
                          const double* freqs, void* q_out, void* k_out, uint8_t* q8, uint8_t* q8_scales,
                          uint8_t* k8, uint8_t* k8_scales, int64_t tokens, int Hq, int Hk, int D, kda_dtype dtype,
                          const kda_qknorm_form* form, void* stream) {
    kda_status st;
    kda::QkArgs a{};
    if ((st = qk_inputs(a, q, k, q_scales, k_scales, q_stride, k_stride, wq, wk, pos, freqs, tokens, Hq, Hk, D, dtype,
                        form)) != KDA_OK)
        return st;
    const bool any = tokens > 0, save = q8 || k8 || q8_scales || k8_scales;
    if ((st = check_ptrs({{q_out, "q_out", any}, {k_out, "k_out", any}, {q8, "q8", save}, {k8, "k8", save},
                          {q8_scales, "q8_scales", save}, {k8_scales, "k8_scales", save}})) != KDA_OK)
        return st;
    if (save && q_scales) return fail(KDA_ERR_BAD_SHAPE, "q and k are packed already: q8 and k8 must be NULL");
    if (!any) return ok();
    a.q_out = q_out;
    a.k_out = k_out;
    a.q8 = q8;
    a.q8s = q8_scales;
    a.k8 = k8;
    a.k8s = k8_scales;
    return launched(kda::launch_qknorm_fwd(a, static_cast<hipStream_t>(stream)), "kda_qknorm_fwd");
}

kda_status kda_qknorm_bwd(const void* q, const void* k, const uint8_t* q_scales, const uint8_t* k_scales,
                          int64_t q_stride, int64_t k_stride, const float* wq, const float* wk, const void* pos,
                          const double* freqs, const void* d_q, const void* d_k, void* dq, void* dk, float* dwq,
                          float* dwk, int64_t tokens, int Hq, int Hk, int D, kda_dtype dtype, kda_dtype grad_dtype,
                          const kda_qknorm_form* form, void* workspace, size_t workspace_bytes, void* stream) {
    kda_status st;
    kda::QkArgs a{};
    if ((st = qk_inputs(a, q, k, q_scales, k_scales, q_stride, k_stride, wq, wk, pos, freqs, tokens, Hq, Hk, D, dtype,
                        form)) != KDA_OK)
        return st;
    if (grad_dtype != KDA_F32 && grad_dtype != KDA_BF16)
        return fail(KDA_ERR_BAD_DTYPE, "grad_dtype must be KDA_F32 or KDA_BF16");
    const bool any = tokens > 0, sums = dwq || dwk;
    if ((st = check_ptrs({{d_q, "d_q", any}, {d_k, "d_k", any}, {dq, "dq", any}, {dk, "dk", any},
                          {dwq, "dwq", sums}, {dwk, "dwk", sums}, {workspace, "workspace", false}})) != KDA_OK)
        return st;
    if (!any && !sums) return ok();
    const int64_t need = sums ? kda::qknorm_bwd_workspace_bytes(tokens, Hq, Hk, D) : 0;
    if (need > 0 && !workspace)
        return fail(KDA_ERR_NULL_ARG, "kda_qknorm_bwd: workspace is NULL (%lld bytes needed)", (long long)need);
    if ((uint64_t)need > (uint64_t)workspace_bytes)
        return fail(KDA_ERR_BAD_SHAPE, "kda_qknorm_bwd: workspace holds %llu bytes, %lld needed",
                    (unsigned long long)workspace_bytes, (long long)need);
    a.d_q = d_q;
    a.d_k = d_k;
    a.grad_f32 = grad_dtype == KDA_F32;
    a.dq = dq;
    a.dk = dk;
    a.dwq = dwq;
    a.dwk = dwk;
    a.ws = workspace;
    return launched(kda::launch_qknorm_bwd(a, static_cast<hipStream_t>(stream)), "kda_qknorm_bwd");
}

size_t kda_qknorm_bwd_workspace_bytes(int64_t tokens, int Hq, int Hk, int D) {
    if (tokens <= 0 || Hq < 1 || Hk < 1 || Hq > 65536 || Hk > 65536 || (D != 64 && D != 128)) return 0;
    return (size_t)kda::qknorm_bwd_workspace_bytes(tokens, Hq, Hk, D);
}

kda_status kda_linattn_fwd(const void* q, const void* k, const void* v, const float* g, const float* s0, void* o,
                           float* s_final, int64_t B, int64_t T, int H, int Dk, int Dv, float scale, kda_dtype dtype,
                           void* workspace, size_t workspace_bytes, void* stream) {
    kda_status st;
    kda::LinArgs a{};
    if ((st = lin_batch(a, B, T, H, Dk, Dv, scale, dtype)) != KDA_OK) return st;
    return lin_fwd(a, q, k, v, g, s0, o, s_final, workspace, workspace_bytes, stream, "kda_linattn_fwd");
}

kda_status kda_linattn_varlen_fwd(const void* q, const void* k, const void* v, const float* g, const int32_t* cu_seqlens,
                                  int64_t N, int64_t total, const float* s0, void* o, float* s_final, int H, int Dk,
                                  int Dv, float scale, kda_dtype dtype, void* workspace, size_t workspace_bytes,
                                  void* stream) {
    kda_status st;
    kda::LinArgs a{};
    if ((st = lin_packed(a, cu_seqlens, N, total, H, Dk, Dv, scale, dtype)) != KDA_OK) return st;
    return lin_fwd(a, q, k, v, g, s0, o, s_final, workspace, workspace_bytes, stream, "kda_linattn_varlen_fwd");
}

kda_status kda_linattn_bwd(const void* q, const void* k, const void* v, const float* g, const float* s0, const void* d_o,
                           const float* d_sfinal, void* dq, void* dk, void* dv, float* ds0, int64_t B, int64_t T, int H,
                           int Dk, int Dv, float scale, kda_dtype dtype, void* workspace, size_t workspace_bytes,
                           void* stream) {
    kda_status st;
    kda::LinArgs a{};
    if ((st = lin_batch(a, B, T, H, Dk, Dv, scale, dtype)) != KDA_OK) return st;
    return lin_bwd(a, q, k, v, g, s0, d_o, d_sfinal, dq, dk, dv, ds0, workspace, workspace_bytes, stream,
                   "kda_linattn_bwd");
}

kda_status kda_linattn_varlen_bwd(const void* q, const void* k, const void* v, const float* g, const int32_t* cu_seqlens,
                                  int64_t N, int64_t total, const float* s0, const void* d_o, const float* d_sfinal,
                                  void* dq, void* dk, void* dv, float* ds0, int H, int Dk, int Dv, float scale,
                                  kda_dtype dtype, void* workspace, size_t workspace_bytes, void* stream) {
    kda_status st;
    kda::LinArgs a{};
    if ((st = lin_packed(a, cu_seqlens, N, total, H, Dk, Dv, scale, dtype)) != KDA_OK) return st;
    return lin_bwd(a, q, k, v, g, s0, d_o, d_sfinal, dq, dk, dv, ds0, workspace, workspace_bytes, stream,
                   "kda_linattn_varlen_bwd");
}

kda_status kda_linattn_step(const void* q, const void* k, const void* v, const float* g, const float* s_in, float* s_out,
                            void* o, int64_t B, int H, int Dk, int Dv, float scale, kda_dtype dtype, void* stream) {
    kda_status st;
    kda::LinArgs a{};
    if ((st = lin_batch(a, B, 1, H, Dk, Dv, scale, dtype)) != KDA_OK) return st;
    if (B * H > kda::kMaxThreads / 256)
        return fail(KDA_ERR_BAD_SHAPE, "%lld sequence-heads exceed the grid limit", (long long)(B * H));
    const bool any = B > 0;
    if ((st = check_ptrs({{q, "q", any}, {k, "k", any}, {v, "v", any}, {g, "g", any, 4}, {s_in, "s_in", any},
                          {s_out, "s_out", any}, {o, "o", any}})) != KDA_OK)
        return st;
    const int64_t states = B * H * Dk * Dv * 4;
    if (s_in != s_out && overlap(s_in, s_out, states, states))
        return fail(KDA_ERR_BAD_SHAPE, "s_in and s_out overlap without being the same buffer");
    if (!any) return ok();
    a.q = q;
    a.k = k;
    a.v = v;
    a.g = g;
    a.o = o;
    return launched(kda::launch_linattn_step(a, s_in, s_out, static_cast<hipStream_t>(stream)), "kda_linattn_step");
}

size_t kda_linattn_workspace_bytes(int64_t N, int64_t total, int H, int Dk, int Dv, kda_dtype dtype) {
    return lin_workspace_bytes(N, total, H, Dk, Dv, dtype, false);
}

size_t kda_linattn_bwd_workspace_bytes(int64_t N, int64_t total, int H, int Dk, int Dv, kda_dtype dtype) {
    return lin_workspace_bytes(N, total, H, Dk, Dv, dtype, true);
}

kda_status kda_groupnorm_fwd(const void* x, int64_t x_stride, const float* weight, const float* bias, const void* gate,
                             int64_t gate_stride, void* y, int64_t tokens, int64_t groups, int64_t width,
                             const kda_groupnorm_form* form, void* stream) {
    kda_status st;
    kda::GroupNormArgs a{};
    if ((st = gn_inputs(a, x, x_stride, weight, bias, gate, gate_stride, tokens, groups, width, form)) != KDA_OK) return st;
    if ((st = check_ptrs({{y, "y", tokens > 0, a.y_f32 ? 4 : 2}})) != KDA_OK) return st;
    if (tokens == 0) return ok();
    a.y = y;
    if ((st = gn_grid(a)) != KDA_OK) return st;
    return launched(kda::launch_groupnorm_fwd(a, static_cast<hipStream_t>(stream)), "kda_groupnorm_fwd");
}

kda_status kda_groupnorm_bwd(const void* x, int64_t x_stride, const float* weight, const float* bias, const void* gate,
                             int64_t gate_stride, const void* dy, void* dx, void* dgate, float* dweight, float* dbias,
                             int64_t tokens, int64_t groups, int64_t width, const kda_groupnorm_form* form,
                             void* workspace, size_t workspace_bytes, void* stream) {
    kda_status st;
    kda::GroupNormArgs a{};
    if ((st = gn_inputs(a, x, x_stride, weight, bias, gate, gate_stride, tokens, groups, width, form)) != KDA_OK) return st;
    const bool any = tokens > 0, sums = dweight || dbias;
    const int xa = a.x_f32 ? 4 : 2, ya = a.y_f32 ? 4 : 2;
    if ((st = check_ptrs({{dy, "dy", any, ya}, {dx, "dx", any, xa}, {dgate, "dgate", any && gate, ya},
                          {dweight, "dweight", sums}, {dbias, "dbias", sums}, {workspace, "workspace", false}})) != KDA_OK)
        return st;
    if (dgate && !gate) return fail(KDA_ERR_BAD_SHAPE, "dgate without a gate");
    if (!any && !sums) return ok();
    const int64_t need = sums ? kda::groupnorm_bwd_workspace_bytes(tokens, groups, width) : 0;
    if (need > 0 && !workspace)
        return fail(KDA_ERR_NULL_ARG, "kda_groupnorm_bwd: workspace is NULL (%lld bytes needed)", (long long)need);
    if ((uint64_t)need > (uint64_t)workspace_bytes)
        return fail(KDA_ERR_BAD_SHAPE, "kda_groupnorm_bwd: workspace holds %llu bytes, %lld needed",
                    (unsigned long long)workspace_bytes, (long long)need);
    a.dy = dy;
    a.dx = dx;
    a.dgate = dgate;
    a.dweight = dweight;
    a.dbias = dbias;
    a.ws = workspace;
    if ((st = gn_grid(a)) != KDA_OK) return st;
    return launched(kda::launch_groupnorm_bwd(a, static_cast<hipStream_t>(stream)), "kda_groupnorm_bwd");
}

size_t kda_groupnorm_bwd_workspace_bytes(int64_t tokens, int64_t groups, int64_t width) {
    if (tokens < 1 || groups < 1 || groups > kda::kMaxChannels || width < 1 || width > kda::kMaxGroupWidth ||
        groups * width > kda::kMaxChannels)
        return 0;
    return (size_t)kda::groupnorm_bwd_workspace_bytes(tokens, groups, width);
}

const char* kda_last_error(void) { return g_last_error.c_str(); }

const char* kda_version(void) { return "kda-gfx950 0.4"; }

}  // extern "C"
