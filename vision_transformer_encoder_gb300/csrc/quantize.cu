// quantize.cu -- rows and weights to e4m3 with a scale for each block of 128 (fp8.cuh).
//
// Rows: x (rows, K) -> q (rows, K), scales (rows, ceil(K / 128)): one block is 128 columns of
// one row. Weights: w (K, N), stored (in, out) as everywhere in the library -> q (N, K), the
// transpose, so that the product reads both operands along K, and scales
// (ceil(N / 128), ceil(K / 128)), one for each 128 x 128 block.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "fp8.cuh"
#include "kernels.h"
#include "launch.cuh"

namespace vit {
namespace {

constexpr int QT_THREADS = 256;

// Generic rows kernel: one warp per block of 128 columns, any width and alignment.
template <typename T>
__global__ void __launch_bounds__(QT_THREADS)
quantize_rows_generic_kernel(const T* __restrict__ x, int64_t rows, int64_t K, uint8_t* __restrict__ q,
                             float* __restrict__ scales) {
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t nblk = (K + kFp8Block - 1) / kFp8Block, total = rows * nblk;
    const int64_t step = (int64_t)gridDim.x * (QT_THREADS / 32);
    for (int64_t g = (int64_t)blockIdx.x * (QT_THREADS / 32) + (threadIdx.x >> 5); g < total; g += step) {
        const int64_t row = g / nblk, b = g - row * nblk;
        float y[4], amax = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t c = b * kFp8Block + i * 32 + lane;
            y[i] = c < K ? to_f32(x[row * K + c]) : 0.f;
            amax = fmaxf(amax, fabsf(y[i]));
        }
        const float sc = fp8_block_scale(warp_max(amax));
        if (lane == 0) scales[g] = sc;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t c = b * kFp8Block + i * 32 + lane;
            if (c < K) q[row * K + c] = fp8_pack1(__fdiv_rn(y[i], sc));
        }
    }
}

// Generic weight kernel: one CTA per 128 x 128 block; the block's values are read twice (the
// second time from L1/L2), its codes are transposed through shared memory.
template <typename T>
__global__ void __launch_bounds__(QT_THREADS)
quantize_weight_generic_kernel(const T* __restrict__ w, int64_t K, int64_t N, uint8_t* __restrict__ q,
                               float* __restrict__ scales) {
    __shared__ uint8_t tile[kFp8Block][kFp8Block + 4];   // [n][k]
    __shared__ float part[QT_THREADS / 32];
    griddep_wait();
    griddep_launch_dependents();
    const int64_t kblk = (K + kFp8Block - 1) / kFp8Block, nblk = (N + kFp8Block - 1) / kFp8Block;
    const int n = threadIdx.x % kFp8Block, kk = threadIdx.x / kFp8Block;
    for (int64_t t = blockIdx.x; t < kblk * nblk; t += gridDim.x) {
        const int64_t nb = t / kblk, kb = t - nb * kblk, n0 = nb * kFp8Block, k0 = kb * kFp8Block;
        float amax = 0.f;
        for (int k = kk; k < kFp8Block; k += QT_THREADS / kFp8Block)
            if (k0 + k < K && n0 + n < N) amax = fmaxf(amax, fabsf(to_f32(w[(k0 + k) * N + n0 + n])));
        amax = warp_max(amax);
        __syncthreads();   // the previous block's tile and part have been read
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = amax;
        __syncthreads();
        for (int i = 0; i < QT_THREADS / 32; ++i) amax = fmaxf(amax, part[i]);
        const float sc = fp8_block_scale(amax);
        if (threadIdx.x == 0) scales[t] = sc;
        for (int k = kk; k < kFp8Block; k += QT_THREADS / kFp8Block)
            if (k0 + k < K && n0 + n < N) tile[n][k] = fp8_pack1(__fdiv_rn(to_f32(w[(k0 + k) * N + n0 + n]), sc));
        __syncthreads();
        for (int i = threadIdx.x; i < kFp8Block * kFp8Block; i += QT_THREADS) {
            const int r = i / kFp8Block, c = i % kFp8Block;
            if (n0 + r < N && k0 + c < K) q[(n0 + r) * K + k0 + c] = tile[r][c];
        }
    }
}

}  // namespace

cudaError_t launch_quantize_rows(const void* x, int dt, int64_t rows, int64_t K, void* q, float* scales,
                                 const DeviceInfo& dev, cudaStream_t s) {
    const int64_t warps = rows * ((K + kFp8Block - 1) / kFp8Block);
    int64_t grid = (warps + QT_THREADS / 32 - 1) / (QT_THREADS / 32);
    if (grid > 16 * (int64_t)dev.num_sms) grid = 16 * (int64_t)dev.num_sms;
    if (dt == DT_BF16)
        return launch_dependent(quantize_rows_generic_kernel<__nv_bfloat16>, dim3((unsigned)grid), dim3(QT_THREADS), 0,
                                s, static_cast<const __nv_bfloat16*>(x), rows, K, static_cast<uint8_t*>(q), scales);
    return launch_dependent(quantize_rows_generic_kernel<float>, dim3((unsigned)grid), dim3(QT_THREADS), 0, s,
                            static_cast<const float*>(x), rows, K, static_cast<uint8_t*>(q), scales);
}

cudaError_t launch_quantize_weight(const void* w, int dt, int64_t K, int64_t N, void* q, float* scales,
                                   const DeviceInfo& dev, cudaStream_t s) {
    int64_t grid = ((K + kFp8Block - 1) / kFp8Block) * ((N + kFp8Block - 1) / kFp8Block);
    if (grid > 16 * (int64_t)dev.num_sms) grid = 16 * (int64_t)dev.num_sms;
    if (dt == DT_BF16)
        return launch_dependent(quantize_weight_generic_kernel<__nv_bfloat16>, dim3((unsigned)grid), dim3(QT_THREADS),
                                0, s, static_cast<const __nv_bfloat16*>(w), K, N, static_cast<uint8_t*>(q), scales);
    return launch_dependent(quantize_weight_generic_kernel<float>, dim3((unsigned)grid), dim3(QT_THREADS), 0, s,
                            static_cast<const float*>(w), K, N, static_cast<uint8_t*>(q), scales);
}

}  // namespace vit
