// Internal launch interface of the operators around the recurrence (C ABI in kda_layer.h).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace kda {

// Rows that a call reads and writes once go past the caches where there are so many bytes of them that they would not stay in
// the 256 MB behind the L2s anyway; smaller calls find their inputs there and leave their outputs there (head norm of
// 4099 x 14 x 64 fp32, backward: 13.9 us through the caches, 15.9 past them; of 32768 x 32 x 128 bf16 from 8 bits: 137 and 125).
constexpr int64_t kStreamBytes = int64_t(128) << 20;

// Threads of a launch: its size is a 32-bit number of them.
constexpr int64_t kMaxThreads = 0xffffffffLL;

// ---- checkpoints in 8 bits (kda_ckpt8.hip)
hipError_t launch_ckpt8_pack(const void* x, uint8_t* codes, uint8_t* scales, int64_t rows, int64_t cols, bool f32,
                             hipStream_t st);
hipError_t launch_ckpt8_unpack(const uint8_t* codes, const uint8_t* scales, void* x, int64_t rows, int64_t cols,
                               bool f32, hipStream_t st);

// ---- gated scan (kda_scan.hip)
constexpr int kScanSeg = 64;  // tokens of a segment
constexpr int kScanThreads = 512;
constexpr int64_t kMaxChannels = 1 << 24;

struct ScanArgs {
    const void *x, *g;
    const float* h0;
    int64_t T_fixed, N, total, D;   // cu == nullptr: N sequences of T_fixed tokens
    const int32_t* cu;
    bool x_f32, g_f32, logit, complement;
    void* ws;
    // forward
    void* y;
    float *h_final, *carry_out;
    uint8_t *u_out, *us_out;
    // backward
    const float* carry;
    const uint8_t *u, *us;
    const void* dy;
    const float* dh_final;
    void *dx, *dg;
    float* dh0;
};

// Segments of 64 tokens: of the packed rows, or of each sequence where all are equally long (the last one of each may be
// shorter).  Sequences of less than half a segment are taken as packed rows: a segment each would leave most of a
// workgroup without rows.
inline bool scan_flat(const ScanArgs& a) { return a.cu || a.T_fixed < kScanSeg / 2; }
inline int64_t scan_segments(const ScanArgs& a) {
    return scan_flat(a) ? (a.total + kScanSeg - 1) / kScanSeg : a.N * ((a.T_fixed + kScanSeg - 1) / kScanSeg);
}
int64_t scan_places(const ScanArgs& a);  // workgroups of a call
int64_t scan_most_segments(int64_t N, int64_t total);
int64_t scan_workspace_bytes(int64_t N, int64_t total, int64_t D);
hipError_t launch_scan_fwd(const ScanArgs& a, hipStream_t st);
hipError_t launch_scan_bwd(const ScanArgs& a, hipStream_t st);
// rows cu[N] .. total - 1 of both buffers (b may be nullptr) to zero
hipError_t launch_scan_zero_behind(const int32_t* cu, int64_t N, int64_t total, void* a, int64_t a_row, void* b,
                                   int64_t b_row, hipStream_t st);
hipError_t launch_scan_step(const ScanArgs& a, const float* h_in, float* h_out, hipStream_t st);

// ---- head norm with rotation (kda_qknorm.hip)
struct QkArgs {
    const void *q, *k;
    const uint8_t *qs, *ks;  // scales of packed q, k; nullptr: plain
    int64_t q_stride, k_stride;
    const float *wq, *wk;
    const void* pos;
    const double* freqs;
    int64_t tokens;
    int Hq, Hk, D, rot;
    bool f32, rms, interleaved, pos64;
    float eps;
    // forward
    void *q_out, *k_out;
    uint8_t *q8, *q8s, *k8, *k8s;
    // backward
    const void *d_q, *d_k;
    bool grad_f32;
    void *dq, *dk;
    float *dwq, *dwk;
    void* ws;
};
int64_t qknorm_bwd_workspace_bytes(int64_t tokens, int Hq, int Hk, int D);
hipError_t launch_qknorm_fwd(const QkArgs& a, hipStream_t st);
hipError_t launch_qknorm_bwd(const QkArgs& a, hipStream_t st);

// ---- linear attention with a decay for each head (kda_linattn.hip)
struct LinArgs {
    const void *q, *k, *v;
    const float *g, *s0;
    int64_t T_fixed, N, total;  // cu == nullptr: N sequences of T_fixed tokens
    const int32_t* cu;
    int H, Dk, Dv;
    float scale;
    bool f32;
    void* ws;
    // forward
    void* o;
    float* s_final;
    // backward
    const void* d_o;
    const float* d_sfinal;
    void *dq, *dk, *dv;
    float* ds0;
};
int64_t linattn_workspace_bytes(const LinArgs& a, bool backward);
int64_t linattn_threads(const LinArgs& a, bool backward);  // of a call's largest launch
hipError_t launch_linattn_fwd(const LinArgs& a, hipStream_t st);
hipError_t launch_linattn_bwd(const LinArgs& a, hipStream_t st);
hipError_t launch_linattn_step(const LinArgs& a, const float* s_in, float* s_out, hipStream_t st);

// ---- group norm with an activation (kda_groupnorm.hip)
constexpr int64_t kMaxGroupWidth = 1 << 16;

struct GroupNormArgs {
    const void *x, *gate;
    int64_t x_stride, gate_stride;
    const float *weight, *bias;
    int64_t tokens, groups, width;
    bool x_f32, y_f32;
    int act;
    float eps;
    // forward
    void* y;
    // backward
    const void* dy;
    void *dx, *dgate;
    float *dweight, *dbias;
    void* ws;
};
bool groupnorm_wide(const GroupNormArgs& a);  // rows are read 16 bytes at a time
int64_t groupnorm_groups(const GroupNormArgs& a);  // of a call's largest launch
int64_t groupnorm_bwd_workspace_bytes(int64_t tokens, int64_t groups, int64_t width);
hipError_t launch_groupnorm_fwd(const GroupNormArgs& a, hipStream_t st);
hipError_t launch_groupnorm_bwd(const GroupNormArgs& a, hipStream_t st);

}  // namespace kda
