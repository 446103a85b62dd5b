/*
 * kda_layer.h -- the operators around the gated delta rule in a layer: the gated scan over
 * channels (the recurrence's sibling with a vector state), the head norm of queries and keys with
 * the position rotation, activation checkpoints in 8 bits, linear attention with a decay for each head
 * (the recurrence's sibling without the delta rule) and the group norm with an activation that the heads'
 * outputs pass.  Same library, conventions, status
 * codes and kda_last_error() as kda.h: DEVICE pointers, row-major and contiguous unless a stride
 * is named, 16-byte aligned unless said otherwise; the caller owns every buffer, the library allocates nothing; calls
 * are asynchronous on `stream`, validated on the host before any launch, and never abort or
 * throw.  Outputs must not overlap inputs or one another except where an argument says so.
 */
#ifndef KDA_LAYER_H
#define KDA_LAYER_H

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------ checkpoints in 8 bits
 *
 * A packed activation is one code byte per value and one scale byte for each 32 values of a row
 * (the last block of a row may be shorter; blocks do not cross rows).  A code is an e4m3 float
 * (sign, 4 exponent bits, 3 fraction bits, largest 448, no infinities); a scale byte s stands for
 * 2^(s - 127).  Packing a block with largest finite magnitude amax takes the smallest
 * e >= -120 with amax <= 448 * 2^e, stores s = e + 127 and rounds x * 2^-e to the nearest code,
 * ties to even: a value that is not far below its block's largest is kept to half a step of 3
 * fraction bits (2^-4 of it), values below 2^-6 * 2^e to 2^-10 * 2^e.  Powers of two cost no
 * rounding, and every packed value is exact in bf16 and in fp32.  Infinities and NaN become the
 * NaN code and leave the block's other values as they would be without them; magnitudes above
 * 1.875 * 2^127 are packed as that, so that they do not unpack to infinity.
 */

/* x [rows, cols] dtype -> codes [rows, cols], scales [rows, ceil(cols / 32)]; cols below 2^31.  Where cols
 * is not a multiple of 8, rows are read a value at a time and the buffers may begin at any value. */
kda_status kda_ckpt8_pack(const void* x, uint8_t* codes, uint8_t* scales, int64_t rows, int64_t cols,
                          kda_dtype dtype, void* stream);

/* codes, scales -> the values they stand for, x [rows, cols] dtype (exact in either type). */
kda_status kda_ckpt8_unpack(const uint8_t* codes, const uint8_t* scales, void* x, int64_t rows, int64_t cols,
                            kda_dtype dtype, void* stream);

/* ------------------------------------------------------------------ gated scan over channels
 *
 * Per channel c of a sequence, with the recurrence's gates (kda.h: clamped log gates, or logits):
 *     l_t = clamp(g_t, -5, 0), or clamp(-softplus(g_t), -5, 0) with g_logit;   a_t = e^(l_t)
 *     h_t = a_t h_{t-1} + w_t x_t,    w_t = 1, or 1 - a_t with complement;     y_t = h_t
 * x, g, y: [B, T, D] (or [total, D] packed); h0, h_final: [B, D] (or [N, D]) float32.  y has x's
 * type and is rounded once; the state is float32 throughout.  D is any number of channels up
 * to 2^24, heads and their sizes flattened.  D % 4 == 0 takes wide loads; others are read an element
 * at a time, and their buffers may begin at any element (not the workspace).  A non-finite x or g makes the
 * rest of its own sequence and channel non-finite and touches nothing else.
 */
typedef struct {
    kda_dtype x_dtype;  /* x, y, dy, dx */
    kda_dtype g_dtype;  /* g, dg */
    int g_logit;        /* nonzero: g holds gate logits */
    int complement;     /* nonzero: w_t = 1 - a_t, else 1 */
} kda_scan_form;

/*
 * What the backward pass needs beside g is written by the forward pass, in one of two forms:
 *   carry                 float32, kda_scan_carry_bytes(): the state at every 64th token; with x
 *                         the backward pass recomputes the states between, to full precision
 *   u_codes, u_scales     packed 8-bit [tokens, D]: u_t = h_{t-1}, less x_t with complement, the
 *                         factor of the gate's gradient; x is not needed then.  dx and dh0 do not
 *                         depend on it; dg takes the rounding of its 3 fraction bits.
 * Each may be NULL (u_codes and u_scales together).
 */
kda_status kda_scan_fwd(const void* x, const void* g, const float* h0, void* y, float* h_final, float* carry,
                        uint8_t* u_codes, uint8_t* u_scales, int64_t B, int64_t T, int64_t D,
                        const kda_scan_form* form, void* workspace, size_t workspace_bytes, void* stream);

/* Packed sequences; cu_seqlens as for kda_varlen_fwd (DEVICE int32 [N+1]; sequences may be empty: their
 * h_final is h0).  Tokens from cu_seqlens[N] on, if total is larger, are neither read into any
 * sequence nor written. */
kda_status kda_scan_varlen_fwd(const void* x, const void* g, const int32_t* cu_seqlens, int64_t N, int64_t total,
                               const float* h0, void* y, float* h_final, float* carry, uint8_t* u_codes,
                               uint8_t* u_scales, int64_t D, const kda_scan_form* form, void* workspace,
                               size_t workspace_bytes, void* stream);

/*
 * Gradients for dL/dy = dy (x's type) and dL/dh_T = dh_final (float32, or NULL for zero):
 *   dx (x's type), dg (g's type; with respect to g before the clamp, which passes on [-5, 0]),
 *   dh0 float32 or NULL.  Either x and carry, or u_codes and u_scales, as the forward pass wrote
 * them; h0 as given to it.  Rows of dx and dg behind the last packed sequence are left as they were.
 */
kda_status kda_scan_bwd(const void* x, const void* g, const float* h0, const float* carry, const uint8_t* u_codes,
                        const uint8_t* u_scales, const void* dy, const float* dh_final, void* dx, void* dg,
                        float* dh0, int64_t B, int64_t T, int64_t D, const kda_scan_form* form, void* workspace,
                        size_t workspace_bytes, void* stream);
kda_status kda_scan_varlen_bwd(const void* x, const void* g, const int32_t* cu_seqlens, int64_t N, int64_t total,
                               const float* h0, const float* carry, const uint8_t* u_codes, const uint8_t* u_scales,
                               const void* dy, const float* dh_final, void* dx, void* dg, float* dh0, int64_t D,
                               const kda_scan_form* form, void* workspace, size_t workspace_bytes, void* stream);

/* Sets rows cu_seqlens[N] .. total - 1 of a and of b (or NULL) to zero: rows of a packed buffer behind its last
 * sequence, which the calls above leave as they were.  Row sizes in bytes, even. */
kda_status kda_scan_zero_behind(const int32_t* cu_seqlens, int64_t N, int64_t total, void* a, int64_t a_row_bytes,
                                void* b, int64_t b_row_bytes, void* stream);

/* One token per sequence: x, g, y [B, D], h_in, h_out [B, D] float32 (h_out == h_in allowed).  Where B * D is
 * not a multiple of 4 they may begin at any element. */
kda_status kda_scan_step(const void* x, const void* g, const float* h_in, float* h_out, void* y, int64_t B,
                         int64_t D, const kda_scan_form* form, void* stream);

/* Bytes of the workspace of the four scan calls (N sequences, total tokens in all; needs no initial
 * contents and must not be shared by calls that may run at once), and of carry.  0: none needed, or
 * unsupported sizes. */
size_t kda_scan_workspace_bytes(int64_t N, int64_t total, int64_t D);
size_t kda_scan_carry_bytes(int64_t N, int64_t total, int64_t D);

/* ------------------------------------------------------------------ head norm with rotation
 *
 * Per token and head, for queries (weight wq) and keys (weight wk) in one pass:
 *     r = (s |x|^2 + eps)^(-1/2),  s = 1 (KDA_NORM_L2) or 1/D (KDA_NORM_RMS); r = 0 where that sum is
 *         below 2^-252, so a zero vector stays zero; a row that holds an infinity or NaN becomes NaN
 *     z = w * r x   (w per channel of a head, shared by the heads; NULL: ones)
 *     y = z with the pairs of its first `rot` channels turned by pos * freqs[i], i < rot / 2:
 *         pair i is (i, i + rot/2), or (2i, 2i + 1) with interleaved
 * Angles are reduced to a fraction of a turn in twice float64's precision before the sine and cosine:
 * positions of any size keep float32's accuracy, as long as |pos * freq| is below 2^80 radians.
 */
enum { KDA_NORM_L2 = 0, KDA_NORM_RMS = 1 };

typedef struct {
    int norm;         /* KDA_NORM_L2 or KDA_NORM_RMS */
    float eps;        /* >= 0 */
    int rot;          /* channels turned: 0, or a multiple of 16 up to D */
    int interleaved;
    int pos_bytes;    /* 4 or 8: pos holds int32 or int64 (any value, negative too) */
} kda_qknorm_form;

/*
 *   q [tokens, Hq, D], k [tokens, Hk, D] dtype; D in {64, 128}.  q_stride, k_stride: elements from one
 *     token to the next (at least Hq*D, Hk*D, and a multiple of 16 bytes): q and k may be columns of
 *     a wider projection.  With q_scales and k_scales given (both or neither), q and k are packed
 *     codes instead, contiguous, and `dtype` is the type of the outputs.
 *   wq, wk [D] float32 or NULL; pos [tokens]; freqs [rot/2] float64, radians per position (both
 *     may be NULL when rot = 0; they may begin at any element).
 *   q_out, k_out: contiguous, dtype.
 *   q8, q8_scales, k8, k8_scales: q and k packed in 8 bits as by kda_ckpt8_pack with rows of D, for the
 *     backward pass; NULL (all four) not to, and refused where q and k are packed already.
 */
kda_status kda_qknorm_fwd(const void* q, const void* k, const uint8_t* q_scales, const uint8_t* k_scales,
                          int64_t q_stride, int64_t k_stride, const float* wq, const float* wk, const void* pos,
                          const double* freqs, void* q_out, void* k_out, uint8_t* q8, uint8_t* q8_scales,
                          uint8_t* k8, uint8_t* k8_scales, int64_t tokens, int Hq, int Hk, int D, kda_dtype dtype,
                          const kda_qknorm_form* form, void* stream);

/*
 * Gradients: d_q, d_k (contiguous, grad_dtype) with respect to q_out and k_out -> dq, dk (contiguous,
 * dtype) with respect to q and k; dwq, dwk [D] float32 (both or neither; a NULL weight's gradient is that of
 * ones).  q, k and the rest as for the forward pass; packed q and k are taken for the values they stand for.
 * The sums over tokens and heads are in a fixed order: the same call gives the same bits.
 * The workspace (kda_qknorm_bwd_workspace_bytes, no initial contents needed) is read only if
 * dwq and dwk are given.
 */
kda_status kda_qknorm_bwd(const void* q, const void* k, const uint8_t* q_scales, const uint8_t* k_scales,
                          int64_t q_stride, int64_t k_stride, const float* wq, const float* wk, const void* pos,
                          const double* freqs, const void* d_q, const void* d_k, void* dq, void* dk, float* dwq,
                          float* dwk, int64_t tokens, int Hq, int Hk, int D, kda_dtype dtype, kda_dtype grad_dtype,
                          const kda_qknorm_form* form, void* workspace, size_t workspace_bytes, void* stream);

size_t kda_qknorm_bwd_workspace_bytes(int64_t tokens, int Hq, int Hk, int D);

/* ------------------------------------------------------------------ linear attention with a decay for each head
 *
 * Per sequence and head h, with a state S (Dk x Dv, float32) and one decay a = e^(min(g_h, 0)) for all tokens:
 *     S_t = a S_(t-1) + k_t v_t^T,    o_t = scale * S_t^T q_t
 * q, k: [B, T, H, Dk], v, o: [B, T, H, Dv] (or [total, H, D] packed), all of `dtype`; g [H] float32, the log of the decay
 * (any value; -infinity keeps nothing; may begin at any element); s0, s_final [B, H, Dk, Dv] (or [N, ...]) float32.
 * Dk, Dv in {64, 128}.  The state and all sums are float32, o is rounded once.  What is not finite in q reaches its own row
 * of o; what is not finite in k or v makes that sequence's rows of that head non-finite from that token on, and touches no
 * row before it nor another head or sequence.  s_final may be NULL, s0 NULL is zero.
 */
kda_status kda_linattn_fwd(const void* q, const void* k, const void* v, const float* g, const float* s0, void* o,
                           float* s_final, int64_t B, int64_t T, int H, int Dk, int Dv, float scale, kda_dtype dtype,
                           void* workspace, size_t workspace_bytes, void* stream);

/* Packed sequences; cu_seqlens as for kda_varlen_fwd (sequences may be empty: their s_final is s0).  Tokens from
 * cu_seqlens[N] on, if total is larger, are neither read into any sequence nor written. */
kda_status kda_linattn_varlen_fwd(const void* q, const void* k, const void* v, const float* g, const int32_t* cu_seqlens,
                                  int64_t N, int64_t total, const float* s0, void* o, float* s_final, int H, int Dk,
                                  int Dv, float scale, kda_dtype dtype, void* workspace, size_t workspace_bytes,
                                  void* stream);

/*
 * Gradients for dL/do = d_o (dtype) and dL/dS_T = d_sfinal (float32, or NULL for zero): dq, dk, dv (dtype) and ds0
 * (float32, or NULL):
 *     dS_t = scale q_t d_o_t^T + a dS_(t+1)  (from dS_T = scale q_T d_o_T^T + d_sfinal),   ds0 = a dS_1
 *     dq_t = scale S_t d_o_t,  dk_t = dS_t v_t,  dv_t = dS_t^T k_t
 * The decays are constants.  Rows of dq, dk, dv behind the last packed sequence are left as they were.
 */
kda_status kda_linattn_bwd(const void* q, const void* k, const void* v, const float* g, const float* s0, const void* d_o,
                           const float* d_sfinal, void* dq, void* dk, void* dv, float* ds0, int64_t B, int64_t T, int H,
                           int Dk, int Dv, float scale, kda_dtype dtype, void* workspace, size_t workspace_bytes,
                           void* stream);
kda_status kda_linattn_varlen_bwd(const void* q, const void* k, const void* v, const float* g, const int32_t* cu_seqlens,
                                  int64_t N, int64_t total, const float* s0, const void* d_o, const float* d_sfinal,
                                  void* dq, void* dk, void* dv, float* ds0, int H, int Dk, int Dv, float scale,
                                  kda_dtype dtype, void* workspace, size_t workspace_bytes, void* stream);

/* One token per sequence: q, k [B, H, Dk], v, o [B, H, Dv], s_in, s_out [B, H, Dk, Dv] (s_out == s_in allowed). */
kda_status kda_linattn_step(const void* q, const void* k, const void* v, const float* g, const float* s_in, float* s_out,
                            void* o, int64_t B, int H, int Dk, int Dv, float scale, kda_dtype dtype, void* stream);

/* Bytes of the workspace of the forward calls and of the backward calls for N sequences of total tokens in all, equally
 * long or packed (no initial contents needed; not to be shared by calls that may run at once).  0: none needed, or
 * unsupported sizes. */
size_t kda_linattn_workspace_bytes(int64_t N, int64_t total, int H, int Dk, int Dv, kda_dtype dtype);
size_t kda_linattn_bwd_workspace_bytes(int64_t N, int64_t total, int H, int Dk, int Dv, kda_dtype dtype);

/* ------------------------------------------------------------------ group norm with an activation, channels last
 *
 * Per token and group of `width` adjacent channels (a head's outputs, say):
 *     n = (x - mean x) / sqrt(mean (x - mean x)^2 + eps),    z = n * weight + bias
 *     y = act(z),  or with a gate  y = z * act(gate)
 * act: the value itself, x / (1 + e^-x) or 1 / (1 + e^-x).  x [tokens, groups * width] x_dtype, gate and y as many of
 * y_dtype; x_stride, gate_stride: elements from one token to the next (at least groups * width), so that they may be columns
 * of wider rows; y is contiguous.  weight, bias [groups * width] float32, each may be NULL (ones, zeros).  All of it is
 * computed in float32 and rounded once.  x, gate and y, their gradients, weight and bias may begin at any element; where all of
 * them begin at 16 bytes and width and the strides are multiples of 8, rows are read 16 bytes at a time, else an element or two.
 * width up to 2^16.
 */
enum { KDA_ACT_NONE = 0, KDA_ACT_SILU = 1, KDA_ACT_SIGMOID = 2 };

typedef struct {
    kda_dtype x_dtype;  /* x, dx */
    kda_dtype y_dtype;  /* y, gate, dy, dgate */
    int act;
    float eps;          /* >= 0 */
} kda_groupnorm_form;

kda_status kda_groupnorm_fwd(const void* x, int64_t x_stride, const float* weight, const float* bias, const void* gate,
                             int64_t gate_stride, void* y, int64_t tokens, int64_t groups, int64_t width,
                             const kda_groupnorm_form* form, void* stream);

/* Gradients for dL/dy = dy (contiguous, y_dtype): dx (contiguous, x_dtype), dgate (contiguous, y_dtype; NULL exactly where
 * gate is), dweight and dbias [groups * width] float32 (both or neither: NULL where no sums are wanted; a NULL weight's is
 * that of ones).  The sums over tokens are in a fixed order: the same call gives the same bits.  The workspace
 * (kda_groupnorm_bwd_workspace_bytes, no initial contents needed) is read only if dweight and dbias are given. */
kda_status kda_groupnorm_bwd(const void* x, int64_t x_stride, const float* weight, const float* bias, const void* gate,
                             int64_t gate_stride, const void* dy, void* dx, void* dgate, float* dweight, float* dbias,
                             int64_t tokens, int64_t groups, int64_t width, const kda_groupnorm_form* form,
                             void* workspace, size_t workspace_bytes, void* stream);

size_t kda_groupnorm_bwd_workspace_bytes(int64_t tokens, int64_t groups, int64_t width);

#ifdef __cplusplus
}
#endif

#endif /* KDA_LAYER_H */
