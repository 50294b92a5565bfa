// attention_cross.cu -- attention of queries to the states of another sequence:
//   o[b, t, h] = sum_{u < len_b} softmax_u(scale q[b, t, h] . k[b, u, h / G]) v[b, u, h / G]
// G = H / Hkv query heads share a key head; len_b = kv_lens[b] (clamped to [0, Tk]) or Tk; a
// sequence with no keys gives zeros. Keys at and past len_b are never read into a product, so
// whatever they hold (NaN included) does not matter. q, k and v are strided in sequence, token
// and head; o is contiguous.
//
// Generic kernel: any type, head width up to 512, stride and alignment; one warp per query row
// with the running maximum and sum of the softmax. 32 keys at a time: each lane scores one key,
// then the lanes share out the columns of the output row.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "launch.cuh"

namespace vit {
namespace {

constexpr int CG_WARPS = 4;

template <typename T, typename A>
__global__ void __launch_bounds__(CG_WARPS * 32)
cross_generic_kernel(const CrossDesc d) {
    extern __shared__ __align__(16) uint8_t smem[];
    griddep_wait();
    griddep_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, dh = (int)d.dh;
    A* sq = reinterpret_cast<A*>(smem) + (size_t)warp * 2 * dh;
    A* so = sq + dh;
    const A scale = (A)d.scale;
    const int64_t rows = d.B * d.Tq * d.H;
    for (int64_t row = (int64_t)blockIdx.x * CG_WARPS + warp; row < rows; row += (int64_t)gridDim.x * CG_WARPS) {
        const int64_t h = row % d.H, t = (row / d.H) % d.Tq, b = row / (d.H * d.Tq);
        const int64_t hk = h / (d.H / d.Hkv);
        const T* q = static_cast<const T*>(d.q) + b * d.qs[0] + t * d.qs[1] + h * d.qs[2];
        const T* k = static_cast<const T*>(d.k) + b * d.ks[0] + hk * d.ks[2];
        const T* v = static_cast<const T*>(d.v) + b * d.vs[0] + hk * d.vs[2];
        T* o = static_cast<T*>(d.o) + row * dh;
        int64_t len = d.Tk;
        if (d.kv_lens) len = min((int64_t)max(d.kv_lens[b], 0), d.Tk);
        __syncwarp();
        for (int c = lane; c < dh; c += 32) {
            sq[c] = to_acc<A>(q[c]);
            so[c] = 0;
        }
        __syncwarp();
        A m = -INFINITY, l = 0;
        for (int64_t u0 = 0; u0 < len; u0 += 32) {
            const int n = (int)min((int64_t)32, len - u0);
            A x = -INFINITY;
            if (lane < n) {
                const T* kr = k + (u0 + lane) * d.ks[1];
                x = 0;
                for (int c = 0; c < dh; ++c) x = sq[c] * to_acc<A>(kr[c]) + x;
                // rounded here: the maximum and what it is taken off are the same numbers
                if constexpr (std::is_same<A, double>::value) x = __dmul_rn(x, scale);
                else x = __fmul_rn(x, scale);
            }
            A mn = x;
#pragma unroll
            for (int i = 16; i > 0; i >>= 1) {
                const A other = __shfl_xor_sync(0xffffffffu, mn, i);
                mn = mn > other ? mn : other;   // a NaN score is not kept here, but its exp below is NaN
            }
            mn = mn > m ? mn : m;
            const A base = mn == -INFINITY ? (A)0 : mn;   // only infinite scores so far: their weights are zero
            A p, alpha;
            if constexpr (std::is_same<A, double>::value) {
                p = lane < n ? exp(x - base) : 0.0;
                alpha = exp(m - base);
            } else {
                p = lane < n ? expf(x - base) : 0.f;
                alpha = expf(m - base);
            }
            l = l * alpha + warp_sum(p);
            m = mn;
            for (int c = lane; c < ((dh + 31) & ~31); c += 32) {
                A acc = c < dh ? so[c] * alpha : (A)0;
                for (int i = 0; i < n; ++i) {
                    const A pi = __shfl_sync(0xffffffffu, p, i);
                    if (c < dh) acc += pi * to_acc<A>(v[(u0 + i) * d.vs[1] + c]);
                }
                if (c < dh) so[c] = acc;
            }
        }
        for (int c = lane; c < dh; c += 32) o[c] = from_acc<T>(len > 0 ? so[c] / l : (A)0);
    }
}

template <typename T, typename A>
cudaError_t generic(const CrossDesc& d, const DeviceInfo& dev, cudaStream_t s) {
    int64_t grid = (d.B * d.Tq * d.H + CG_WARPS - 1) / CG_WARPS;
    if (grid > 64 * (int64_t)dev.num_sms) grid = 64 * (int64_t)dev.num_sms;
    return launch_dependent(cross_generic_kernel<T, A>, dim3((unsigned)grid), dim3(CG_WARPS * 32),
                            (size_t)CG_WARPS * 2 * d.dh * sizeof(A), s, d);
}

}  // namespace

cudaError_t launch_cross_attention(const CrossDesc& d, const DeviceInfo& dev, cudaStream_t s) {
    if (cross_f32_supported(d)) return launch_cross_f32(d, dev, s);
    if (cross_rows_supported(d)) return launch_cross_rows(d, dev, s);
    if (cross_tc_supported(d)) return launch_cross_tc(d, dev, s);
    if (d.dt == DT_F64) return generic<double, double>(d, dev, s);
    if (d.dt == DT_F32) return generic<float, float>(d, dev, s);
    return generic<__nv_bfloat16, float>(d, dev, s);
}

}  // namespace vit
