// rmsnorm.cu -- root-mean-square norm of rows with the residual's addition, its output in the
// stream's type or in e4m3 with one scale for each 128 columns:
//   s = x + residual,  y = s / sqrt(mean(s^2) + eps) * gamma
// s is formed and normalised in fp32 (fp64 for fp64) and rounded only where it is stored as the
// new residual stream. Sums of squares stay in that type: at most 32 terms in turn per thread, and in the
// generic kernel ceil(D / 256), then a tree, so that their relative error is below 2^-24 (max(32, D / 256) + 10).
//
// Fast kernel (D % 8 == 0, 16-byte aligned, D up to 16384): a row is read once, by the threads of a
// group of 1 to 16 warps, 8 elements per thread and step, and stays in registers as fp32 sums until
// its mean square is known. Sixteen neighbouring threads hold 128 columns, so an e4m3 block's
// scale is a maximum over half a warp. Bound by HBM. With few rows more warps share a row, because
// latency counts.
//
// Rows kernel (many rows): groups of 1 to 16 warps that stay, a row at a time; a group's next row
// travels, as it was stored, while this one is worked on. Without that all warps of a wave load and
// then compute together: 16400 x 1280, bf16 with residual to e4m3, 31.6 us; with it 24.9 us
// (5.9 TB/s).
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

// A row whose squares sum past the arithmetic's range (values of about 1e19 and more, fp64 1e154) is summed again
// from values scaled by 2^-80 (fp64 2^-600), whose squares stay in the range for every finite row.
constexpr float kSquaresLimit = 3.4028234e38f;
constexpr float kPreScale = 8.271806125530277e-25f;
template <typename A> struct LargeRows {
    static constexpr A limit = kSquaresLimit, pre = kPreScale;
};
template <> struct LargeRows<double> {
    static constexpr double limit = 1.7976931348623157e308, pre = 0x1p-600;
};

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
        if (ss > LargeRows<A>::limit) {   // squares past the range: again from scaled values
            pre = LargeRows<A>::pre;
            ss = 0;
            for (int64_t c = threadIdx.x; c < D; c += blockDim.x) {
                const A v = value(c) * pre;
                ss += v * v;
            }
            ss = block_sum(ss, part);
            eps_row = eps * pre * pre;
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
                    if (c < D) out[row * D + c] = fp8_pack1((float)y[i] * fp8_inverse(sc));
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

// 8 consecutive elements, 16-byte aligned. x may be overwritten by the same thread later, so
// these are plain loads.
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const float2 a = unpack_bf16x2(u.x), b = unpack_bf16x2(u.y), c = unpack_bf16x2(u.z), d = unpack_bf16x2(u.w);
    v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
    v[4] = c.x; v[5] = c.y; v[6] = d.x; v[7] = d.y;
}
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                                              pack_bf16x2(v[6], v[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}

// G warps per row, NV steps of 8 columns per thread; blockDim.x = 32 G times the rows of a CTA
// (one row when G > 1).
template <typename TX, typename TR, typename TO, int NV>
__global__ void __launch_bounds__(512, 2)   // 64 registers: 32 warps per SM
rmsnorm_fast_kernel(const TX* x, const TR* residual, int64_t rows, int D, float eps, const void* __restrict__ gamma,
                    int gamma_dt, TR* sum, TO* out, float* __restrict__ scales, int G) {
    constexpr bool Q = std::is_same<TO, uint8_t>::value;
    __shared__ float part[2][16];
    griddep_wait();
    griddep_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, threads = 32 * G;
    const int t = G == 1 ? lane : (int)threadIdx.x;
    const int64_t row = G == 1 ? (int64_t)blockIdx.x * (blockDim.x >> 5) + warp : (int64_t)blockIdx.x;
    if (row >= rows) return;   // whole warps, and whole CTAs when warps share a row
    const int64_t at = row * D;
    float v[NV][8];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * threads + t) * 8;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
        if (c < D) {
            load8(x + at + c, v[i]);
            if (residual) {
                float r[8];
                load8(residual + at + c, r);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] += r[j];
            }
        }
    }
    auto total = [&](float w, int round) {
        w = warp_sum(w);
        if (G > 1) {
            if (lane == 0) part[round][warp] = w;
            __syncthreads();
            w = lane < G ? part[round][lane] : 0.f;
            w = warp_sum(w);
        }
        return w;
    };
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(v[i][j], v[i][j], ss);
    if (sum) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * threads + t) * 8;
            if (c < D) store8(sum + at + c, v[i]);
        }
    }
    ss = total(ss, 0);
    float e = eps;
    if (ss > kSquaresLimit) {   // squares past the fp32 range: again from scaled values
        float s2 = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[i][j] *= kPreScale;
                s2 = fmaf(v[i][j], v[i][j], s2);
            }
        ss = total(s2, 1);
        e = eps * kPreScale * kPreScale;
    }
    const float r = 1.f / sqrtf(ss / (float)D + e);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * threads + t) * 8;
        float y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = v[i][j] * r;
        if (gamma && c < D) {
            float g[8];
            if (gamma_dt == DT_BF16) load8(static_cast<const __nv_bfloat16*>(gamma) + c, g);
            else load8(static_cast<const float*>(gamma) + c, g);
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] *= g[j];
        }
        if constexpr (Q) {
            // NaN must not hide: fmaxf drops it, but its code below is NaN whatever the scale
            float amax = fmaxf(fmaxf(fmaxf(fabsf(y[0]), fabsf(y[1])), fmaxf(fabsf(y[2]), fabsf(y[3]))),
                               fmaxf(fmaxf(fabsf(y[4]), fabsf(y[5])), fmaxf(fabsf(y[6]), fabsf(y[7]))));
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            const float sc = fp8_block_scale(amax), inv = fp8_inverse(sc);
            if (c < D) {
                if ((lane & 15) == 0) scales[row * ((D + kFp8Block - 1) / kFp8Block) + c / kFp8Block] = sc;
                *reinterpret_cast<uint2*>(out + at + c) =
                    make_uint2(fp8_pack4(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv),
                               fp8_pack4(y[4] * inv, y[5] * inv, y[6] * inv, y[7] * inv));
            }
        } else {
            if (c < D) store8(out + at + c, y);
        }
    }
}

// 8 elements as they are stored.
template <typename T> struct Raw8;
template <> struct Raw8<__nv_bfloat16> {
    uint4 u;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void zero() { u = make_uint4(0, 0, 0, 0); }
    // elements 2 i and 2 i + 1 as a packed pair of floats
    __device__ __forceinline__ unsigned long long pair(int i) const {
        const uint32_t w = i == 0 ? u.x : i == 1 ? u.y : i == 2 ? u.z : u.w;
        return f2_pack(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    }
};
template <> struct Raw8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = *reinterpret_cast<const float4*>(p);
        b = *reinterpret_cast<const float4*>(p + 4);
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ unsigned long long pair(int i) const {
        return i == 0 ? f2_pack(a.x, a.y) : i == 1 ? f2_pack(a.z, a.w) : i == 2 ? f2_pack(b.x, b.y) : f2_pack(b.z, b.w);
    }
};

__device__ __forceinline__ void unpack4(const unsigned long long (&p)[4], float (&v)[8]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) f2_unpack(p[j], v[2 * j], v[2 * j + 1]);
}

constexpr int RR_THREADS = 128;

// WIDE: a CTA of up to 16 warps shares each row; otherwise each of its four warps has its own.
template <typename TX, typename TR, typename TO, int NV, bool RES, bool WIDE>
__global__ void __launch_bounds__(WIDE ? 512 : RR_THREADS, WIDE ? 1 : NV * (sizeof(TX) + (RES ? sizeof(TR) : 0)) <= 12 ? 5 : 4)
rmsnorm_rows_kernel(const TX* x, const TR* residual, int64_t rows, int D, float eps, const void* __restrict__ gamma,
                    int gamma_dt, TR* sum, TO* out, float* __restrict__ scales) {
    constexpr bool Q = std::is_same<TO, uint8_t>::value;
    __shared__ float part[2][16];
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, nblk = (D + kFp8Block - 1) / kFp8Block;
    const int t = WIDE ? (int)threadIdx.x : lane, threads = WIDE ? (int)blockDim.x : 32;
    const int64_t stride = WIDE ? (int64_t)gridDim.x : (int64_t)gridDim.x * (RR_THREADS / 32);
    int64_t row = WIDE ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * (RR_THREADS / 32) + (threadIdx.x >> 5);
    int round = 0;
    auto total = [&](float w) {   // over the row's threads
        w = warp_sum(w);
        if constexpr (WIDE) {
            // two sets of partial sums in turn: nobody writes a set that another warp still reads
            if (lane == 0) part[round & 1][threadIdx.x >> 5] = w;
            __syncthreads();
            w = warp_sum(lane < (threads >> 5) ? part[round & 1][lane] : 0.f);
            ++round;
        }
        return w;
    };
    const float inv_d = 1.f / (float)D;
    Raw8<TX> xr[NV];
    Raw8<TR> rr[RES ? NV : 1];
    auto fetch = [&](int64_t r) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * threads + t) * 8;
            if (c < D) {
                xr[i].load(x + r * D + c);
                if (RES) rr[RES ? i : 0].load(residual + r * D + c);
            } else {
                xr[i].zero();
                if (RES) rr[RES ? i : 0].zero();
            }
        }
    };
    if (row < rows) fetch(row);
    for (; row < rows; row += stride) {
        unsigned long long v[NV][4], s2 = 0ull;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[i][j] = xr[i].pair(j);
                if (RES) v[i][j] = f2_add(v[i][j], rr[RES ? i : 0].pair(j));
                s2 = f2_fma(v[i][j], v[i][j], s2);
            }
        const int64_t at = row * D;
        // each element is read before it is overwritten, by the same thread
        if (row + stride < rows) fetch(row + stride);
        if (RES && sum) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (i * threads + t) * 8;
                float f[8];
                unpack4(v[i], f);
                if (c < D) store8(sum + at + c, f);
            }
        }
        float a, b;
        f2_unpack(s2, a, b);
        float ss = total(a + b), e = eps;
        if (ss > kSquaresLimit) {   // squares past the fp32 range: again from scaled values
            const unsigned long long pre = f2_pack(kPreScale, kPreScale);
            s2 = 0ull;
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    v[i][j] = f2_mul(v[i][j], pre);
                    s2 = f2_fma(v[i][j], v[i][j], s2);
                }
            f2_unpack(s2, a, b);
            ss = total(a + b);
            e = eps * kPreScale * kPreScale;
        }
        const float r = 1.f / sqrtf(ss * inv_d + e);
        const unsigned long long r2 = f2_pack(r, r);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * threads + t) * 8;
#pragma unroll
            for (int j = 0; j < 4; ++j) v[i][j] = f2_mul(v[i][j], r2);
            if (gamma && c < D) {
                if (gamma_dt == DT_BF16) {
                    Raw8<__nv_bfloat16> g;
                    g.load(static_cast<const __nv_bfloat16*>(gamma) + c);
#pragma unroll
                    for (int j = 0; j < 4; ++j) v[i][j] = f2_mul(v[i][j], g.pair(j));
                } else {
                    Raw8<float> g;
                    g.load(static_cast<const float*>(gamma) + c);
#pragma unroll
                    for (int j = 0; j < 4; ++j) v[i][j] = f2_mul(v[i][j], g.pair(j));
                }
            }
            float y[8];
            unpack4(v[i], y);
            if constexpr (Q) {
                float amax = fmaxf(fmaxf(fmaxf(fabsf(y[0]), fabsf(y[1])), fmaxf(fabsf(y[2]), fabsf(y[3]))),
                                   fmaxf(fmaxf(fabsf(y[4]), fabsf(y[5])), fmaxf(fabsf(y[6]), fabsf(y[7]))));
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
                const float sc = fp8_block_scale(amax), inv = fp8_inverse(sc);
                const unsigned long long i2 = f2_pack(inv, inv);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[i][j] = f2_mul(v[i][j], i2);
                unpack4(v[i], y);
                if (c < D) {
                    if ((lane & 15) == 0) scales[row * nblk + c / kFp8Block] = sc;
                    *reinterpret_cast<uint2*>(out + at + c) =
                        make_uint2(fp8_pack4(y[0], y[1], y[2], y[3]), fp8_pack4(y[4], y[5], y[6], y[7]));
                }
            } else {
                if (c < D) store8(out + at + c, y);
            }
        }
    }
}

template <typename TX, typename TR, typename TO, int NV, bool RES, bool WIDE>
cudaError_t rows_inst(const RmsNormDesc& d, const DeviceInfo& dev, int threads, cudaStream_t s) {
    auto k = rmsnorm_rows_kernel<TX, TR, TO, NV, RES, WIDE>;
    int resident = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&resident, k, threads, 0) != cudaSuccess || resident < 1) resident = 1;
    const int per = WIDE ? 1 : threads / 32;
    const int64_t need = (d.rows + per - 1) / per, most = (int64_t)resident * dev.num_sms;
    // the same number of rows for every group, as nearly as they divide
    const int64_t turns = (need + most - 1) / most, grid = (need + turns - 1) / turns;
    return launch_dependent(k, dim3((unsigned)grid), dim3(threads), 0, s, static_cast<const TX*>(d.x),
                            static_cast<const TR*>(d.residual), d.rows, (int)d.D, (float)d.eps, d.gamma, d.gamma_dt,
                            static_cast<TR*>(d.sum), static_cast<TO*>(d.out), d.scales);
}

template <typename TX, typename TR, typename TO, bool RES>
cudaError_t rows_nv(const RmsNormDesc& d, const DeviceInfo& dev, int nv, int G, cudaStream_t s) {
    // steps whose two rows (one as stored, one in fp32) fit in registers
    constexpr int MAXNV = 20 / (sizeof(TX) + (RES ? sizeof(TR) : 0)) < 5 ? 20 / (sizeof(TX) + (RES ? sizeof(TR) : 0)) : 5;
    constexpr int N3 = MAXNV < 3 ? MAXNV : 3, N4 = MAXNV < 4 ? MAXNV : 4;
    // a row that more warps than one share fills more than half of the steps of each
    constexpr int W2 = MAXNV == 5 ? 3 : 2;
    if (G > 1) switch (nv) {
        case 2: return rows_inst<TX, TR, TO, W2, RES, true>(d, dev, 32 * G, s);
        case 3: return rows_inst<TX, TR, TO, N3, RES, true>(d, dev, 32 * G, s);
        case 4: return rows_inst<TX, TR, TO, N4, RES, true>(d, dev, 32 * G, s);
        case 5: return rows_inst<TX, TR, TO, MAXNV, RES, true>(d, dev, 32 * G, s);
    }
    switch (nv) {
        case 1: return rows_inst<TX, TR, TO, 1, RES, false>(d, dev, RR_THREADS, s);
        case 2: return rows_inst<TX, TR, TO, 2, RES, false>(d, dev, RR_THREADS, s);
        case 3: return rows_inst<TX, TR, TO, N3, RES, false>(d, dev, RR_THREADS, s);
        case 4: return rows_inst<TX, TR, TO, N4, RES, false>(d, dev, RR_THREADS, s);
        case 5: return rows_inst<TX, TR, TO, MAXNV, RES, false>(d, dev, RR_THREADS, s);
    }
    return cudaErrorInvalidValue;
}

template <typename TX, typename TR, typename TO, int NV>
cudaError_t fast_inst(const RmsNormDesc& d, int G, cudaStream_t s) {
    const int per = G == 1 ? 8 : 1;   // rows per CTA
    return launch_dependent(rmsnorm_fast_kernel<TX, TR, TO, NV>, dim3((unsigned)((d.rows + per - 1) / per)),
                            dim3(32 * G * per), 0, s, static_cast<const TX*>(d.x), static_cast<const TR*>(d.residual),
                            d.rows, (int)d.D, (float)d.eps, d.gamma, d.gamma_dt, static_cast<TR*>(d.sum),
                            static_cast<TO*>(d.out), d.scales, G);
}

template <typename TX, typename TR, typename TO>
cudaError_t fast(const RmsNormDesc& d, const DeviceInfo& dev, cudaStream_t s) {
    const int steps = (int)((d.D + 255) / 256);   // of one warp
    // many rows: as few warps per row as hold it and the next one in registers; worth it from two
    // rows for each group on
    const int raw = (int)(sizeof(TX) + (d.residual ? sizeof(TR) : 0)), most = 20 / raw < 5 ? 20 / raw : 5;
    int G = 1;
    while (G < 16 && steps > most * G) G *= 2;
    if (steps <= most * G && d.rows * G >= 32 * (int64_t)dev.num_sms) {
        const int nv = (steps + G - 1) / G;
        // (without a residual its type is x's)
        if constexpr (std::is_same<TX, TR>::value)
            if (!d.residual) return rows_nv<TX, TR, TO, false>(d, dev, nv, G, s);
        return rows_nv<TX, TR, TO, true>(d, dev, nv, G, s);
    }
    // fewer: as many warps as leave every thread one step, up to 16
    G = 1;
    while (G < 16 && steps > G) G *= 2;
    const int nv = (steps + G - 1) / G;
    switch (nv) {
        case 1: return fast_inst<TX, TR, TO, 1>(d, G, s);
        case 2: return fast_inst<TX, TR, TO, 2>(d, G, s);
        case 3: return fast_inst<TX, TR, TO, 3>(d, G, s);
        case 4: return fast_inst<TX, TR, TO, 4>(d, G, s);
    }
    return cudaErrorInvalidValue;
}

bool fast_ok(const RmsNormDesc& d) {
    const void* ps[] = {d.x, d.residual, d.gamma, d.sum, d.out};
    for (const void* p : ps)
        if (reinterpret_cast<uintptr_t>(p) & 15) return false;
    return d.D % 8 == 0 && d.D <= 16384 && d.rows <= 0x7fffffff;
}

template <typename TX, typename TR, typename TO, typename A>
cudaError_t generic(const RmsNormDesc& d, cudaStream_t s) {
    const unsigned grid = (unsigned)(d.rows < (1 << 20) ? d.rows : (1 << 20));
    return launch_dependent(rmsnorm_generic_kernel<TX, TR, TO, A>, dim3(grid), dim3(RN_THREADS), 0, s,
                            static_cast<const TX*>(d.x), static_cast<const TR*>(d.residual), d.rows, d.D, (A)d.eps,
                            d.gamma, d.gamma_dt, static_cast<TR*>(d.sum), static_cast<TO*>(d.out), d.scales);
}

template <typename TX, typename TR>
cudaError_t by_out(const RmsNormDesc& d, const DeviceInfo& dev, cudaStream_t s) {
    if (fast_ok(d)) switch (d.out_dt) {
        case DT_BF16: return fast<TX, TR, __nv_bfloat16>(d, dev, s);
        case DT_F32: return fast<TX, TR, float>(d, dev, s);
        case DT_E4M3: return fast<TX, TR, uint8_t>(d, dev, s);
    }
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
    if (d.x_dt == DT_F32) return by_out<float, float>(d, dev, s);
    return d.residual_dt == DT_F32 ? by_out<__nv_bfloat16, float>(d, dev, s)
                                     : by_out<__nv_bfloat16, __nv_bfloat16>(d, dev, s);
}

}  // namespace vit
