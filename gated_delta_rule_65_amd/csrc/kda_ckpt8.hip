// Packing activations to 8 bits for the backward pass, and unpacking them (format: kda_ckpt8.h).
//
// Both move their bytes once and are bound by HBM.  Rows of a multiple of 8 values go by pieces of 8: a lane reads 16 (bf16) or
// 32 bytes, four lanes share a block and find its largest magnitude by two exchanges inside a quad, and write 8 bytes
// of codes each.  A workgroup takes four pieces a lane, all loaded before the first is used (one piece a
// lane leaves too few bytes in flight, more keep too few workgroups on a CU).  Where rows are whole
// blocks (a multiple of 32), pieces follow one another over the whole tensor and no index is divided.
// Other row lengths take a value a lane.
//
// Measured: 67M bf16 values packed in 34 us and unpacked in 29 us (204 MB each: 6.0 and 6.9 TB/s, as fast as they copy);
// 333 x 1000 fp32 values in 4 and 3 us, launches alone.
#include "kda_ckpt8.h"
#include "kda_layer_launch.h"

namespace kda {

namespace {

constexpr int kPieces = 4;  // of a lane

template <bool F32>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
    if constexpr (F32) return static_cast<const float*>(p)[i];
    else return __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
}

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// Piece i: four to a block, `blocks` blocks in all, per_row of them to a row; where it begins, and whether it holds values.
template <bool WHOLE>
__device__ __forceinline__ bool piece_at(int64_t i, int64_t blocks, uint32_t per_row, int64_t cols, int64_t& at) {
    const int64_t b = i >> 2;
    if constexpr (WHOLE) {
        at = i * 8;
        return b < blocks;
    } else {
        const int64_t row = blocks <= 0xffffffffLL ? (int64_t)((uint32_t)b / per_row) : b / per_row;
        const int64_t c = (b - row * per_row) * kCkptBlock + (i & 3) * 8;
        at = row * cols + c;
        return b < blocks && c < cols;
    }
}

template <bool F32, bool WHOLE>
__global__ __launch_bounds__(256) void pack8_kernel(const void* __restrict__ x, uint8_t* __restrict__ codes,
                                                    uint8_t* __restrict__ scales, int64_t blocks, uint32_t per_row,
                                                    int64_t cols) {
    const int64_t i0 = (int64_t)blockIdx.x * (256 * kPieces) + threadIdx.x;
    u32x4 raw[kPieces][F32 ? 2 : 1];
    int64_t at[kPieces];
    bool in[kPieces];
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
        in[j] = piece_at<WHOLE>(i0 + 256 * j, blocks, per_row, cols, at[j]);
        const u32x4* p = reinterpret_cast<const u32x4*>(static_cast<const char*>(x) + (in[j] ? at[j] : 0) * (F32 ? 4 : 2));
        raw[j][0] = __builtin_nontemporal_load(p);
        if constexpr (F32) raw[j][1] = __builtin_nontemporal_load(p + 1);
    }
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if constexpr (F32) v[k] = __uint_as_float(raw[j][k / 4][k % 4]);
            else v[k] = __uint_as_float(k % 2 ? raw[j][0][k / 2] & 0xffff0000u : raw[j][0][k / 2] << 16);
        }
        bool any;
        const int s = ckpt_block<4, 8>(v, in[j], any);
        const float inv = ckpt_inverse(s);
        if (!in[j]) continue;
        *reinterpret_cast<u32x2*>(codes + at[j]) = u32x2{ckpt_code4(v, inv, any), ckpt_code4(v + 4, inv, any)};
        if ((threadIdx.x & 3) == 0) scales[(i0 + 256 * j) >> 2] = (uint8_t)s;
    }
}

template <bool F32, bool WHOLE>
__global__ __launch_bounds__(256) void unpack8_kernel(const uint8_t* __restrict__ codes,
                                                      const uint8_t* __restrict__ scales, void* __restrict__ x,
                                                      int64_t blocks, uint32_t per_row, int64_t cols) {
    const int64_t i0 = (int64_t)blockIdx.x * (256 * kPieces) + threadIdx.x;
    u32x2 raw[kPieces];
    uint8_t s[kPieces];
    int64_t at[kPieces];
    bool in[kPieces];
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
        in[j] = piece_at<WHOLE>(i0 + 256 * j, blocks, per_row, cols, at[j]);
        raw[j] = *reinterpret_cast<const u32x2*>(codes + (in[j] ? at[j] : 0));
        s[j] = scales[in[j] ? (i0 + 256 * j) >> 2 : 0];
    }
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
        if (!in[j]) continue;
        float v[8];
        const float unit = ckpt_unit(s[j]);
        ckpt_value4(raw[j][0], unit, v);
        ckpt_value4(raw[j][1], unit, v + 4);
        uint32_t w[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) w[k] = __float_as_uint(v[k]);
        if constexpr (F32) {
            u32x4* p = reinterpret_cast<u32x4*>(static_cast<float*>(x) + at[j]);
            __builtin_nontemporal_store(u32x4{w[0], w[1], w[2], w[3]}, p);
            __builtin_nontemporal_store(u32x4{w[4], w[5], w[6], w[7]}, p + 1);
        } else {  // exact: the upper halves
            u32x4 o;
#pragma unroll
            for (int k = 0; k < 4; ++k) o[k] = w[2 * k] >> 16 | (w[2 * k + 1] & 0xffff0000u);
            __builtin_nontemporal_store(o, reinterpret_cast<u32x4*>(static_cast<uint16_t*>(x) + at[j]));
        }
    }
}

// Rows of any length: a block of 32 values to 32 lanes.
template <bool F32>
__global__ __launch_bounds__(256) void pack1_kernel(const void* __restrict__ x, uint8_t* __restrict__ codes,
                                                    uint8_t* __restrict__ scales, int64_t blocks, int64_t per_row,
                                                    int64_t cols) {
    const int lane = threadIdx.x & 31;
    const int64_t step = (int64_t)gridDim.x * 8;
    for (int64_t b = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); b < blocks; b += step) {
        const int64_t row = b / per_row, c = (b - row * per_row) * kCkptBlock + lane;
        const bool in = c < cols;
        const float v = in ? load1<F32>(x, row * cols + c) : 0.f;
        bool any;
        const int s = ckpt_block<32, 1>(&v, in, any);
        if (in) codes[row * cols + c] = (uint8_t)ckpt_code_any(v, ckpt_inverse(s));
        if (lane == 0) scales[b] = (uint8_t)s;
    }
}

template <bool F32>
__global__ __launch_bounds__(256) void unpack1_kernel(const uint8_t* __restrict__ codes,
                                                      const uint8_t* __restrict__ scales, void* __restrict__ x,
                                                      int64_t blocks, int64_t per_row, int64_t cols) {
    const int lane = threadIdx.x & 31;
    const int64_t step = (int64_t)gridDim.x * 8;
    for (int64_t b = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); b < blocks; b += step) {
        const int64_t row = b / per_row, c = (b - row * per_row) * kCkptBlock + lane;
        if (c >= cols) continue;
        float v[4];
        ckpt_value4(codes[row * cols + c], ckpt_unit(scales[b]), v);
        if constexpr (F32) static_cast<float*>(x)[row * cols + c] = v[0];
        else static_cast<uint16_t*>(x)[row * cols + c] = (uint16_t)(__float_as_uint(v[0]) >> 16);  // exact
    }
}

// The kernel for rows of `cols` values and its grid.
template <class By8, class By1>
hipError_t by_rows(int64_t rows, int64_t cols, By8 by8, By1 by1) {
    const int64_t per_row = (cols + kCkptBlock - 1) / kCkptBlock, blocks = rows * per_row;
    if (cols % 8 == 0) {
        const int64_t groups = (blocks + 64 * kPieces - 1) / (64 * kPieces);
        by8(dim3((unsigned)groups), blocks, per_row);
    } else {
        const int64_t groups = (blocks + 7) / 8;
        by1(dim3((unsigned)(groups < 16384 ? groups : 16384)), blocks, per_row);
    }
    return hipGetLastError();
}

}  // namespace

#define KDA_CKPT(KERNEL, GRID, ...)                                                              \
    do {                                                                                         \
        if (f32) hipLaunchKernelGGL((KERNEL(true)), GRID, dim3(256), 0, st, __VA_ARGS__);        \
        else hipLaunchKernelGGL((KERNEL(false)), GRID, dim3(256), 0, st, __VA_ARGS__);           \
    } while (0)

hipError_t launch_ckpt8_pack(const void* x, uint8_t* codes, uint8_t* scales, int64_t rows, int64_t cols, bool f32,
                             hipStream_t st) {
#define KDA_WHOLE(F) pack8_kernel<F, true>
#define KDA_PART(F) pack8_kernel<F, false>
#define KDA_ONE(F) pack1_kernel<F>
    return by_rows(
        rows, cols,
        [&](dim3 grid, int64_t blocks, int64_t per_row) {
            if (cols % kCkptBlock == 0) KDA_CKPT(KDA_WHOLE, grid, x, codes, scales, blocks, (uint32_t)per_row, cols);
            else KDA_CKPT(KDA_PART, grid, x, codes, scales, blocks, (uint32_t)per_row, cols);
        },
        [&](dim3 grid, int64_t blocks, int64_t per_row) {
            KDA_CKPT(KDA_ONE, grid, x, codes, scales, blocks, per_row, cols);
        });
#undef KDA_WHOLE
#undef KDA_PART
#undef KDA_ONE
}

hipError_t launch_ckpt8_unpack(const uint8_t* codes, const uint8_t* scales, void* x, int64_t rows, int64_t cols,
                               bool f32, hipStream_t st) {
#define KDA_WHOLE(F) unpack8_kernel<F, true>
#define KDA_PART(F) unpack8_kernel<F, false>
#define KDA_ONE(F) unpack1_kernel<F>
    return by_rows(
        rows, cols,
        [&](dim3 grid, int64_t blocks, int64_t per_row) {
            if (cols % kCkptBlock == 0) KDA_CKPT(KDA_WHOLE, grid, codes, scales, x, blocks, (uint32_t)per_row, cols);
            else KDA_CKPT(KDA_PART, grid, codes, scales, x, blocks, (uint32_t)per_row, cols);
        },
        [&](dim3 grid, int64_t blocks, int64_t per_row) {
            KDA_CKPT(KDA_ONE, grid, codes, scales, x, blocks, per_row, cols);
        });
#undef KDA_WHOLE
#undef KDA_PART
#undef KDA_ONE
}

}  // namespace kda
