// gemm_fp8.cu -- the 8-bit matrix product with a scale for each block of 128:
//   z[m, n] = sum_b sa[m, b] sw[n / 128, b] sum_{k in block b} a[m, k] w[n, k]   (+ bias[n])
//   out     = z,  GELU_tanh(z)  or  residual + z
// a (M, K) and w (N, K) are e4m3, sa (M, ceil(K / 128)) and sw (ceil(N / 128), ceil(K / 128))
// fp32. Products of e4m3 values are exact in fp32; a block's sum and the sum over blocks are
// fp32. An e4m3 output takes one scale for each 128 columns of a row (fp8.cuh).
//
// Generic kernel: CUDA cores, any size and alignment; a CTA makes 16 rows x 128 columns (one
// output block per row), a thread eight columns of one row.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "fp8.cuh"
#include "kernels.h"
#include "launch.cuh"

namespace vit {
namespace {

constexpr int GG_ROWS = 16, GG_COLS = 128, GG_THREADS = 256;

__device__ __forceinline__ float load_f32(const void* p, bool f32, int64_t i) {
    return f32 ? static_cast<const float*>(p)[i] : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}

__global__ void __launch_bounds__(GG_THREADS)
gemm_fp8_generic_kernel(const Fp8GemmDesc d) {
    __shared__ float sa[GG_ROWS][kFp8Block];
    __shared__ uint8_t sw[GG_COLS][kFp8Block + 4];
    griddep_wait();
    griddep_launch_dependents();
    const int64_t kblk = (d.K + kFp8Block - 1) / kFp8Block, nblk = (d.N + GG_COLS - 1) / GG_COLS;
    const int64_t tiles = ((d.M + GG_ROWS - 1) / GG_ROWS) * nblk;
    const int r = threadIdx.x >> 4, c = threadIdx.x & 15;   // a row's 16 threads are half a warp
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        const int64_t mt = t / nblk, nt = t - mt * nblk, m = mt * GG_ROWS + r, n0 = nt * GG_COLS;
        float acc[8] = {};
        for (int64_t kb = 0; kb < kblk; ++kb) {
            const int64_t k0 = kb * kFp8Block;
            __syncthreads();
            for (int i = threadIdx.x; i < GG_ROWS * kFp8Block; i += GG_THREADS) {
                const int64_t mm = mt * GG_ROWS + i / kFp8Block, k = k0 + i % kFp8Block;
                sa[i / kFp8Block][i % kFp8Block] = mm < d.M && k < d.K ? fp8_value(d.a[mm * d.K + k]) : 0.f;
            }
            for (int i = threadIdx.x; i < GG_COLS * kFp8Block; i += GG_THREADS) {
                const int64_t n = n0 + i / kFp8Block, k = k0 + i % kFp8Block;
                sw[i / kFp8Block][i % kFp8Block] = n < d.N && k < d.K ? d.w[n * d.K + k] : 0;
            }
            __syncthreads();
            float p[8] = {};
            for (int k = 0; k < kFp8Block; ++k) {
                const float av = sa[r][k];
#pragma unroll
                for (int j = 0; j < 8; ++j) p[j] = fmaf(av, fp8_value(sw[c + 16 * j][k]), p[j]);
            }
            if (m < d.M) {
                const float sc = d.a_scales[m * kblk + kb] * d.w_scales[nt * kblk + kb];
#pragma unroll
                for (int j = 0; j < 8; ++j) acc[j] = fmaf(sc, p[j], acc[j]);
            }
        }
        float amax = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int64_t n = n0 + c + 16 * j;
            if (m < d.M && n < d.N) {
                if (d.bias) acc[j] += load_f32(d.bias, d.bias_f32, n);
                if (d.epi == TC_EPI_GELU) acc[j] = gelu_tanh_acc(acc[j]);
                if (d.epi == TC_EPI_RESID) acc[j] += load_f32(d.residual, d.residual_f32, m * d.N + n);
                amax = fmaxf(amax, fabsf(acc[j]));
            }
        }
        float sc = 1.f;
        if (d.out_dt == DT_E4M3) {
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            sc = fp8_block_scale(amax);
            if (c == 0 && m < d.M) d.out_scales[m * nblk + nt] = sc;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int64_t n = n0 + c + 16 * j;
            if (m >= d.M || n >= d.N) continue;
            const int64_t at = m * d.N + n;
            if (d.out_dt == DT_E4M3) static_cast<uint8_t*>(d.out)[at] = fp8_pack1(__fdiv_rn(acc[j], sc));
            else if (d.out_dt == DT_F32) static_cast<float*>(d.out)[at] = acc[j];
            else static_cast<__nv_bfloat16*>(d.out)[at] = __float2bfloat16_rn(acc[j]);
        }
    }
}

}  // namespace

cudaError_t launch_gemm_fp8(const Fp8GemmDesc& d, const DeviceInfo& dev, cudaStream_t s) {
    int64_t grid = ((d.M + GG_ROWS - 1) / GG_ROWS) * ((d.N + GG_COLS - 1) / GG_COLS);
    if (grid > 8 * (int64_t)dev.num_sms) grid = 8 * (int64_t)dev.num_sms;
    return launch_dependent(gemm_fp8_generic_kernel, dim3((unsigned)grid), dim3(GG_THREADS), 0, s, d);
}

}  // namespace vit
