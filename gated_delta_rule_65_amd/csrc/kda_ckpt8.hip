// Packing activations to 8 bits for the backward pass, and unpacking them (format: kda_ckpt8.h).
#include "kda_ckpt8.h"
#include "kda_layer_launch.h"

namespace kda {

template <bool F32>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
    if constexpr (F32) return static_cast<const float*>(p)[i];
    else return __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
}

// A block of 32 values to 32 lanes; the largest magnitude by five lane exchanges.
template <bool F32>
__global__ __launch_bounds__(256) void pack_kernel(const void* __restrict__ x, uint8_t* __restrict__ codes,
                                                   uint8_t* __restrict__ scales, int64_t blocks, int64_t per_row,
                                                   int64_t cols) {
    const int lane = threadIdx.x & 31;
    const int64_t step = (int64_t)gridDim.x * 8;
    for (int64_t b = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); b < blocks; b += step) {
        const int64_t row = b / per_row, c = (b - row * per_row) * kCkptBlock + lane;
        const bool in = c < cols;
        const float v = in ? load1<F32>(x, row * cols + c) : 0.f;
        uint32_t top = finite_abs_bits(v);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
            const uint32_t o = (uint32_t)__shfl_xor((int)top, off);
            top = top > o ? top : o;
        }
        const int s = ckpt_scale(top);
        if (in) codes[row * cols + c] = (uint8_t)ckpt_code2(v, 0.f, ckpt_inverse(s));
        if (lane == 0) scales[b] = (uint8_t)s;
    }
}

template <bool F32>
__global__ __launch_bounds__(256) void unpack_kernel(const uint8_t* __restrict__ codes,
                                                     const uint8_t* __restrict__ scales, void* __restrict__ x,
                                                     int64_t blocks, int64_t per_row, int64_t cols) {
    const int lane = threadIdx.x & 31;
    const int64_t step = (int64_t)gridDim.x * 8;
    for (int64_t b = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); b < blocks; b += step) {
        const int64_t row = b / per_row, c = (b - row * per_row) * kCkptBlock + lane;
        if (c >= cols) continue;
        const float v = ckpt_value<0>(codes[row * cols + c], scales[b]);
        if constexpr (F32) static_cast<float*>(x)[row * cols + c] = v;
        else static_cast<uint16_t*>(x)[row * cols + c] = (uint16_t)(__float_as_uint(v) >> 16);  // exact
    }
}

static unsigned ckpt_grid(int64_t blocks) {
    const int64_t wg = (blocks + 7) / 8;
    return (unsigned)(wg < 8192 ? wg : 8192);
}

hipError_t launch_ckpt8_pack(const void* x, uint8_t* codes, uint8_t* scales, int64_t rows, int64_t cols, bool f32,
                             hipStream_t st) {
    const int64_t per_row = (cols + kCkptBlock - 1) / kCkptBlock, blocks = rows * per_row;
    const dim3 grid(ckpt_grid(blocks));
    if (f32) hipLaunchKernelGGL((pack_kernel<true>), grid, dim3(256), 0, st, x, codes, scales, blocks, per_row, cols);
    else hipLaunchKernelGGL((pack_kernel<false>), grid, dim3(256), 0, st, x, codes, scales, blocks, per_row, cols);
    return hipGetLastError();
}

hipError_t launch_ckpt8_unpack(const uint8_t* codes, const uint8_t* scales, void* x, int64_t rows, int64_t cols,
                               bool f32, hipStream_t st) {
    const int64_t per_row = (cols + kCkptBlock - 1) / kCkptBlock, blocks = rows * per_row;
    const dim3 grid(ckpt_grid(blocks));
    if (f32) hipLaunchKernelGGL((unpack_kernel<true>), grid, dim3(256), 0, st, codes, scales, x, blocks, per_row, cols);
    else hipLaunchKernelGGL((unpack_kernel<false>), grid, dim3(256), 0, st, codes, scales, x, blocks, per_row, cols);
    return hipGetLastError();
}

}  // namespace kda
