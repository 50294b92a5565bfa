// rmsnorm.cu -- root-mean-square norm of rows with the residual's addition, its output in the
// stream's type or in e4m3 with one scale for each 128 columns:
//   s = x + residual,  y = s / sqrt(mean(s^2) + eps) * gamma
// s is formed and normalised in fp32 (fp64 for fp64) and rounded only where it is stored as the
// new residual stream; sums of squares are fp32 over at most a few hundred terms per thread and
// then a tree, so their relative error stays far below one bf16 step.
//
// Generic kernel: one CTA per row, any width, alignment and type. Two passes over x and the
// residual; an element is read and then overwritten by the same thread, so the sum may be
// stored in place of either.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "common.cuh"
#include "fp8.cuh"
#include "kernels.h"
#include "launch.cuh"

namespace vit {
namespace {

constexpr int RN_THREADS = 256;

// A row whose squares sum past kSquaresLimit (values of about 1e19 and more) is summed again from
// values scaled by 2^-80, whose squares stay in the fp32 range for every finite row.
constexpr float kSquaresLimit = 3.4028234e38f;
constexpr float kPreScale = 8.271806125530277e-25f;

template <typename T> __device__ __forceinline__ T block_sum(T v, T* part) {
    v = warp_sum(v);
    __syncthreads();   // part is free again
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    T t = 0;
    for (int i = 0; i < (int)(blockDim.x >> 5); ++i) t += part[i];
    return t;
}

// TX, TR: element types of x and of the residual stream (residual and sum may be null);
// TO: the output's, or uint8_t for e4m3. A: arithmetic.
template <typename TX, typename TR, typename TO, typename A>
__global__ void __launch_bounds__(RN_THREADS)
rmsnorm_generic_kernel(const TX* x, const TR* residual, int64_t rows, int64_t D, A eps, const void* gamma,
                       int gamma_dt, TR* sum, TO* out, float* scales) {
    __shared__ A part[RN_THREADS / 32];
    griddep_wait();
    griddep_launch_dependents();
    constexpr bool Q = std::is_same<TO, uint8_t>::value;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t nblk = (D + kFp8Block - 1) / kFp8Block;
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
        const TX* xr = x + row * D;
        const TR* rr = residual ? residual + row * D : nullptr;
        auto value = [&](int64_t c) {
            A v = to_acc<A>(xr[c]);
            if (rr) v += to_acc<A>(rr[c]);
            return v;
        };
        auto gain = [&](int64_t c) -> A {
            if (!gamma) return (A)1;
            if (gamma_dt == DT_BF16) return to_acc<A>(static_cast<const __nv_bfloat16*>(gamma)[c]);
            if (gamma_dt == DT_F32) return (A) static_cast<const float*>(gamma)[c];
            return (A) static_cast<const double*>(gamma)[c];
        };
        A ss = 0, eps_row = eps;
        for (int64_t c = threadIdx.x; c < D; c += blockDim.x) {
            const A v = value(c);
            ss += v * v;
        }
        ss = block_sum(ss, part);
        A pre = 1;
        if (ss > (A)kSquaresLimit) {   // squares past the fp32 range: again from scaled values
            pre = (A)kPreScale;
            ss = 0;
            for (int64_t c = threadIdx.x; c < D; c += blockDim.x) {
                const A v = value(c) * pre;
                ss += v * v;
            }
            ss = block_sum(ss, part);
            eps_row = 0;   // far below half a unit of the scaled mean square
        }
        A r;
        if constexpr (std::is_same<A, double>::value) r = 1.0 / sqrt(ss / (A)D + eps_row);
        else r = 1.f / sqrtf(ss / (A)D + eps_row);
        // a warp takes one block of 128 columns at a time, so its scale is a warp reduction
        for (int64_t b = warp; b < nblk; b += RN_THREADS / 32) {
            A y[4];
            float amax = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t c = b * kFp8Block + i * 32 + lane;
                y[i] = 0;
                if (c < D) {
                    const A v = value(c);
                    if (sum) sum[row * D + c] = from_acc<TR>(v);
                    y[i] = v * pre * r * gain(c);
                }
                amax = fmaxf(amax, fabsf((float)y[i]));
            }
            if constexpr (Q) {
                const float sc = fp8_block_scale(warp_max(amax));
                if (lane == 0) scales[row * nblk + b] = sc;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int64_t c = b * kFp8Block + i * 32 + lane;
                    if (c < D) out[row * D + c] = fp8_pack1(__fdiv_rn((float)y[i], sc));
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int64_t c = b * kFp8Block + i * 32 + lane;
                    if (c < D) out[row * D + c] = from_acc<TO>(y[i]);
                }
            }
        }
    }
}

template <typename TX, typename TR, typename TO, typename A>
cudaError_t generic(const RmsNormDesc& d, cudaStream_t s) {
    const unsigned grid = (unsigned)(d.rows < (1 << 20) ? d.rows : (1 << 20));
    return launch_dependent(rmsnorm_generic_kernel<TX, TR, TO, A>, dim3(grid), dim3(RN_THREADS), 0, s,
                            static_cast<const TX*>(d.x), static_cast<const TR*>(d.residual), d.rows, d.D, (A)d.eps,
                            d.gamma, d.gamma_dt, static_cast<TR*>(d.sum), static_cast<TO*>(d.out), d.scales);
}

template <typename TX, typename TR>
cudaError_t by_out(const RmsNormDesc& d, cudaStream_t s) {
    switch (d.out_dt) {
        case DT_BF16: return generic<TX, TR, __nv_bfloat16, float>(d, s);
        case DT_F32: return generic<TX, TR, float, float>(d, s);
        case DT_E4M3: return generic<TX, TR, uint8_t, float>(d, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_rmsnorm(const RmsNormDesc& d, const DeviceInfo& dev, cudaStream_t s) {
    if (d.x_dt == DT_F64) return generic<double, double, double, double>(d, s);
    if (d.x_dt == DT_F32) return by_out<float, float>(d, s);
    return d.residual_dt == DT_F32 ? by_out<__nv_bfloat16, float>(d, s) : by_out<__nv_bfloat16, __nv_bfloat16>(d, s);
}

}  // namespace vit
