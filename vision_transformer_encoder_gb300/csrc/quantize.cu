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

// 8 consecutive elements, 16-byte aligned.
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
    const float2 a = unpack_bf16x2(u.x), b = unpack_bf16x2(u.y), c = unpack_bf16x2(u.z), d = unpack_bf16x2(u.w);
    v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
    v[4] = c.x; v[5] = c.y; v[6] = d.x; v[7] = d.y;
}
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ float amax8(const float (&v)[8]) {
    return fmaxf(fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3]))),
                 fmaxf(fmaxf(fabsf(v[4]), fabsf(v[5])), fmaxf(fabsf(v[6]), fabsf(v[7]))));
}

// 8 elements as they are loaded: their largest magnitude, and their codes at 1 / scale = inv.
struct Raw8B {
    uint4 u;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = __ldg(reinterpret_cast<const uint4*>(p)); }
    __device__ __forceinline__ void zero() { u = make_uint4(0, 0, 0, 0); }
    // magnitudes of bf16 numbers compare like their bits; a NaN's are above infinity's and do not count
    __device__ __forceinline__ float amax() const {
        const __nv_bfloat162 m = __hmax2(__hmax2(mag(u.x), mag(u.y)), __hmax2(mag(u.z), mag(u.w)));
        const float2 f = __bfloat1622float2(m);
        return fmaxf(f.x, f.y);
    }
    __device__ __forceinline__ uint2 codes(float inv) const {
        const float2 a = unpack_bf16x2(u.x), b = unpack_bf16x2(u.y), c = unpack_bf16x2(u.z), d = unpack_bf16x2(u.w);
        return make_uint2(fp8_pack4(a.x * inv, a.y * inv, b.x * inv, b.y * inv),
                          fp8_pack4(c.x * inv, c.y * inv, d.x * inv, d.y * inv));
    }
    __device__ static __forceinline__ __nv_bfloat162 mag(uint32_t w) {
        w &= 0x7FFF7FFFu;
        return *reinterpret_cast<const __nv_bfloat162*>(&w);
    }
};
struct Raw8F {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = __ldg(reinterpret_cast<const float4*>(p));
        b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ float amax() const {
        return fmaxf(fmaxf(fmaxf(fabsf(a.x), fabsf(a.y)), fmaxf(fabsf(a.z), fabsf(a.w))),
                     fmaxf(fmaxf(fabsf(b.x), fabsf(b.y)), fmaxf(fabsf(b.z), fabsf(b.w))));
    }
    __device__ __forceinline__ uint2 codes(float inv) const {
        return make_uint2(fp8_pack4(a.x * inv, a.y * inv, a.z * inv, a.w * inv),
                          fp8_pack4(b.x * inv, b.y * inv, b.z * inv, b.w * inv));
    }
};
template <typename T> struct Raw8Of;
template <> struct Raw8Of<__nv_bfloat16> { typedef Raw8B type; };
template <> struct Raw8Of<float> { typedef Raw8F type; };

// Rows, K % 8 == 0 and aligned: half a warp takes a block of 128 columns, 8 per thread; each thread
// has QR_STEPS blocks in flight, a grid's width apart, as they were loaded. HBM-bound: one read,
// one write. 12608 x 1024: 7.7 us (5.1 TB/s), of which some 2 are the launch; the generic kernel took 21.5.
constexpr int QR_STEPS = 4;
template <typename T>
__global__ void __launch_bounds__(QT_THREADS)
quantize_rows_kernel(const T* __restrict__ x, int64_t blocks, int K, int nblk, uint8_t* __restrict__ q,
                     float* __restrict__ scales) {
    griddep_wait();
    griddep_launch_dependents();
    const int64_t half = (int64_t)gridDim.x * (QT_THREADS / 16);
    const int64_t g0 = (int64_t)blockIdx.x * (QT_THREADS / 16) + (threadIdx.x >> 4);
    const int l16 = threadIdx.x & 15;
    typename Raw8Of<T>::type v[QR_STEPS];
    int64_t at[QR_STEPS];   // -1: nothing to do
#pragma unroll
    for (int i = 0; i < QR_STEPS; ++i) {
        const int64_t g = g0 + i * half;
        const int64_t row = blocks <= 0x7fffffff ? (int64_t)((uint32_t)g / (uint32_t)nblk) : g / nblk;
        const int c = (int)(g - row * nblk) * kFp8Block + l16 * 8;
        at[i] = g < blocks && c < K ? row * K + c : -1;
        if (at[i] >= 0) v[i].load(x + at[i]);
        else v[i].zero();
    }
#pragma unroll
    for (int i = 0; i < QR_STEPS; ++i) {
        float amax = v[i].amax();
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        const float sc = fp8_block_scale(amax);
        if (at[i] >= 0) {
            if (l16 == 0) scales[g0 + i * half] = sc;
            *reinterpret_cast<uint2*>(q + at[i]) = v[i].codes(fp8_inverse(sc));
        }
    }
}

// Weights, K and N multiples of 8 and aligned: one CTA per 128 x 128 block, read once into registers
// (thread: 8 columns of 8 rows), its codes transposed through shared memory four rows to a word. Word
// rows are 33 words apart: a half warp's writes (one column each, 8 columns apart) and a warp's
// reads fall in different banks. 1024 x 4096: 4.0 us (the generic kernel 17.0), a load's and a store's latency.
template <typename T>
__global__ void __launch_bounds__(QT_THREADS)
quantize_weight_kernel(const T* __restrict__ w, int K, int N, int kblk, uint8_t* __restrict__ q,
                       float* __restrict__ scales) {
    __shared__ uint32_t tile[kFp8Block][33];   // [n][k / 4]
    __shared__ float part[QT_THREADS / 32];
    griddep_wait();
    griddep_launch_dependents();
    const int nb = blockIdx.x / kblk, kb = blockIdx.x - nb * kblk, n0 = nb * kFp8Block, k0 = kb * kFp8Block;
    const int cv = threadIdx.x & 15, rv = threadIdx.x >> 4;   // columns 8 cv.., rows 4 rv.. and 64 + 4 rv..
    float v[8][8], amax = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int k = k0 + (i >> 2) * 64 + rv * 4 + (i & 3), n = n0 + cv * 8;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
        if (k < K && n < N) load8(w + (int64_t)k * N + n, v[i]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = fmaxf(amax, amax8(v[i]));
    amax = warp_max(amax);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = amax;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < QT_THREADS / 32; ++i) amax = fmaxf(amax, part[i]);
    const float sc = fp8_block_scale(amax), inv = fp8_inverse(sc);
    if (threadIdx.x == 0) scales[blockIdx.x] = sc;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < 8; ++j)
            tile[cv * 8 + j][h * 16 + rv] =
                fp8_pack4(v[h * 4][j] * inv, v[h * 4 + 1][j] * inv, v[h * 4 + 2][j] * inv, v[h * 4 + 3][j] * inv);
    __syncthreads();
    for (int i = threadIdx.x; i < kFp8Block * 16; i += QT_THREADS) {
        const int r = i >> 4, c = i & 15;   // 8 codes
        if (n0 + r < N && k0 + c * 8 < K)
            *reinterpret_cast<uint2*>(q + (int64_t)(n0 + r) * K + k0 + c * 8) = make_uint2(tile[r][2 * c], tile[r][2 * c + 1]);
    }
}

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
            if (c < K) q[row * K + c] = fp8_pack1(y[i] * fp8_inverse(sc));
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
            if (k0 + k < K && n0 + n < N) tile[n][k] = fp8_pack1(to_f32(w[(k0 + k) * N + n0 + n]) * fp8_inverse(sc));
        __syncthreads();
        for (int i = threadIdx.x; i < kFp8Block * kFp8Block; i += QT_THREADS) {
            const int r = i / kFp8Block, c = i % kFp8Block;
            if (n0 + r < N && k0 + c < K) q[(n0 + r) * K + k0 + c] = tile[r][c];
        }
    }
}

}  // namespace

namespace {

template <typename T>
cudaError_t rows_of(const T* x, int64_t rows, int64_t K, uint8_t* q, float* scales, const DeviceInfo& dev, cudaStream_t s) {
    const int64_t nblk = (K + kFp8Block - 1) / kFp8Block, blocks = rows * nblk;
    constexpr int per = QT_THREADS / 16 * QR_STEPS;
    if (K % 8 == 0 && !(reinterpret_cast<uintptr_t>(x) & 15) && !(reinterpret_cast<uintptr_t>(q) & 7) &&
        K <= 0x7fffffff - 256 && blocks / per < 0x7ffffff0)
        return launch_dependent(quantize_rows_kernel<T>, dim3((unsigned)((blocks + per - 1) / per)), dim3(QT_THREADS), 0,
                                s, x, blocks, (int)K, (int)nblk, q, scales);
    int64_t grid = (blocks + QT_THREADS / 32 - 1) / (QT_THREADS / 32);
    if (grid > 16 * (int64_t)dev.num_sms) grid = 16 * (int64_t)dev.num_sms;
    return launch_dependent(quantize_rows_generic_kernel<T>, dim3((unsigned)grid), dim3(QT_THREADS), 0, s, x, rows, K, q,
                            scales);
}

template <typename T>
cudaError_t weight_of(const T* w, int64_t K, int64_t N, uint8_t* q, float* scales, const DeviceInfo& dev, cudaStream_t s) {
    const int64_t kblk = (K + kFp8Block - 1) / kFp8Block, grid = kblk * ((N + kFp8Block - 1) / kFp8Block);
    if (K % 8 == 0 && N % 8 == 0 && !(reinterpret_cast<uintptr_t>(w) & 15) && !(reinterpret_cast<uintptr_t>(q) & 7) &&
        K <= 0x7fffffff - 256 && N <= 0x7fffffff - 256 && grid <= 0x7fffffff)
        return launch_dependent(quantize_weight_kernel<T>, dim3((unsigned)grid), dim3(QT_THREADS), 0, s, w, (int)K, (int)N,
                                (int)kblk, q, scales);
    const int64_t most = 16 * (int64_t)dev.num_sms;
    return launch_dependent(quantize_weight_generic_kernel<T>, dim3((unsigned)(grid < most ? grid : most)),
                            dim3(QT_THREADS), 0, s, w, K, N, q, scales);
}

}  // namespace

cudaError_t launch_quantize_rows(const void* x, int dt, int64_t rows, int64_t K, void* q, float* scales,
                                 const DeviceInfo& dev, cudaStream_t s) {
    uint8_t* o = static_cast<uint8_t*>(q);
    return dt == DT_BF16 ? rows_of(static_cast<const __nv_bfloat16*>(x), rows, K, o, scales, dev, s)
                         : rows_of(static_cast<const float*>(x), rows, K, o, scales, dev, s);
}

cudaError_t launch_quantize_weight(const void* w, int dt, int64_t K, int64_t N, void* q, float* scales,
                                   const DeviceInfo& dev, cudaStream_t s) {
    uint8_t* o = static_cast<uint8_t*>(q);
    return dt == DT_BF16 ? weight_of(static_cast<const __nv_bfloat16*>(w), K, N, o, scales, dev, s)
                         : weight_of(static_cast<const float*>(w), K, N, o, scales, dev, s);
}

}  // namespace vit
