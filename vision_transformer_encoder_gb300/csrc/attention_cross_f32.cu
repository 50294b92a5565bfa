// attention_cross_f32.cu -- cross attention in fp32 on the CUDA cores: the mathematics of
// attention_cross.cu for head widths 32, 48, 64, 80, 96, 112 and 128.
//
// A CTA of four warps takes 64 packed query rows (row = token * G + head of the group) of one key
// head and walks the keys 64 at a time, K and V tiles arriving by cp.async a tile ahead. A thread
// makes an 8 x 4 piece of S (rows 8 g .. 8 g + 7, keys c, c + 16, c + 32, c + 48) and the same rows
// of O in columns c, c + 16, ...; the sixteen threads of a row group are half a warp, so the row
// maxima are shuffles and P goes through shared memory inside one warp. 32 products need 12
// shared-memory words: bound by the FP32 pipe. Warps whose sixteen rows hold no query skip the
// arithmetic.
#include <cuda_runtime.h>

#include "common.cuh"
#include "kernels.h"
#include "launch.cuh"

namespace vit {
namespace {

constexpr int CF_ROWS = 64, CF_KEYS = 64, CF_THREADS = 128;

template <int DH> struct CfLayout {
    static constexpr int LD = DH + 4;             // padded rows: 16-byte columns of eight keys in different banks
    static constexpr int LDP = CF_KEYS + 4;
    static constexpr int TILE = CF_KEYS * LD;     // floats of one K or V tile
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_K = OFF_Q + CF_ROWS * LD;
    static constexpr int OFF_V = OFF_K + 2 * TILE;
    static constexpr int OFF_P = OFF_V + 2 * TILE;
    static constexpr int SMEM = (OFF_P + CF_ROWS * LDP) * 4;
    static_assert(SMEM <= 227 * 1024, "shared memory");
};

// 16 bytes global -> shared, zeros when !ok (nothing is read then).
__device__ __forceinline__ void cp_async16(float* dst, const float* src, bool ok) {
    const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <int DH>
__global__ void __launch_bounds__(CF_THREADS)
cross_f32_kernel(const __grid_constant__ CrossDesc d, float scale_log2, int qtiles) {
    using L = CfLayout<DH>;
    constexpr int LD = L::LD, NC = DH / 16, V4 = DH / 4;
    extern __shared__ __align__(16) float sm[];
    float* sQ = sm + L::OFF_Q;
    float* sK = sm + L::OFF_K;
    float* sV = sm + L::OFF_V;
    float* sP = sm + L::OFF_P;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, c = lane & 15, r0 = warp * 16 + (lane >> 4) * 8;
    const int G = (int)(d.H / d.Hkv);
    const int64_t rows = d.Tq * G;   // packed rows of one key head
    const int qt = blockIdx.x % qtiles;
    const int64_t bh = blockIdx.x / qtiles, b = bh / d.Hkv, h = bh % d.Hkv, first = (int64_t)qt * CF_ROWS;
    griddep_wait();
    griddep_launch_dependents();

    const float* k = static_cast<const float*>(d.k) + b * d.ks[0] + h * d.ks[2];
    const float* v = static_cast<const float*>(d.v) + b * d.vs[0] + h * d.vs[2];
    int64_t len = d.Tk;
    if (d.kv_lens) len = min((int64_t)max(__ldg(d.kv_lens + b), 0), d.Tk);
    const int tiles = (int)((len + CF_KEYS - 1) / CF_KEYS);
    auto fetch = [&](int tile) {
        float* dk = sK + (tile & 1) * L::TILE;
        float* dv = sV + (tile & 1) * L::TILE;
        for (int i = tid; i < CF_KEYS * V4; i += CF_THREADS) {
            const int u = i / V4, x = (i - u * V4) * 4;
            const int64_t key = (int64_t)tile * CF_KEYS + u;
            const bool ok = key < len;   // rows past the length are zeros, whatever they hold
            cp_async16(dk + u * LD + x, k + (ok ? key : 0) * d.ks[1] + x, ok);
            cp_async16(dv + u * LD + x, v + (ok ? key : 0) * d.vs[1] + x, ok);
        }
        cp_async_commit();
    };
    if (tiles > 0) fetch(0);
    for (int i = tid; i < CF_ROWS * V4; i += CF_THREADS) {
        const int r = i / V4, x = (i - r * V4) * 4;
        const int64_t row = first + r;
        float4 q = make_float4(0.f, 0.f, 0.f, 0.f);
        if (row < rows)
            q = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(d.q) + b * d.qs[0] + (row / G) * d.qs[1] +
                                                      (h * G + row % G) * d.qs[2] + x));
        *reinterpret_cast<float4*>(sQ + r * LD + x) = q;
    }

    const bool live = first + warp * 16 < rows;
    float o[8][NC], m[8], l[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int j = 0; j < NC; ++j) o[i][j] = 0.f;
    }
    for (int t = 0; t < tiles; ++t) {
        if (t + 1 < tiles) {
            fetch(t + 1);
            cp_async_wait<1>();
        } else {
            cp_async_wait<0>();
        }
        __syncthreads();   // this tile (and, the first time, Q) is in place
        if (live) {
            const float* tk = sK + (t & 1) * L::TILE;
            const float* tv = sV + (t & 1) * L::TILE;
            float s[8][4] = {};
#pragma unroll 4
            for (int x = 0; x < DH; x += 4) {
                float4 kv[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) kv[j] = *reinterpret_cast<const float4*>(tk + (c + 16 * j) * LD + x);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float4 q = *reinterpret_cast<const float4*>(sQ + (r0 + i) * LD + x);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        s[i][j] = fmaf(q.x, kv[j].x, s[i][j]);
                        s[i][j] = fmaf(q.y, kv[j].y, s[i][j]);
                        s[i][j] = fmaf(q.z, kv[j].z, s[i][j]);
                        s[i][j] = fmaf(q.w, kv[j].w, s[i][j]);
                    }
                }
            }
            const int64_t valid = len - (int64_t)t * CF_KEYS;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float mx = m[i];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[i][j] = c + 16 * j < valid ? s[i][j] * scale_log2 : -INFINITY;
                    mx = fmaxf(mx, s[i][j]);
                }
#pragma unroll
                for (int w = 8; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
                const float base = mx == -INFINITY ? 0.f : mx;   // only infinite scores so far: weights of zero
                const float alpha = exp2_approx(m[i] - base);
                m[i] = mx;
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float p = exp2_approx(s[i][j] - base);
                    sum += p;
                    sP[(r0 + i) * L::LDP + c + 16 * j] = p;
                }
                l[i] = l[i] * alpha + sum;   // this thread's keys; joined at the end
#pragma unroll
                for (int j = 0; j < NC; ++j) o[i][j] *= alpha;
            }
            __syncwarp();
#pragma unroll 2
            for (int u = 0; u < CF_KEYS; u += 4) {
                float vv[4][NC];
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int j = 0; j < NC; ++j) vv[e][j] = tv[(u + e) * LD + c + 16 * j];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float4 p = *reinterpret_cast<const float4*>(sP + (r0 + i) * L::LDP + u);
#pragma unroll
                    for (int j = 0; j < NC; ++j) {
                        o[i][j] = fmaf(p.x, vv[0][j], o[i][j]);
                        o[i][j] = fmaf(p.y, vv[1][j], o[i][j]);
                        o[i][j] = fmaf(p.z, vv[2][j], o[i][j]);
                        o[i][j] = fmaf(p.w, vv[3][j], o[i][j]);
                    }
                }
            }
        }
        __syncthreads();   // the tile has been read: its buffer takes the one after the next
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma unroll
        for (int w = 8; w > 0; w >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], w);
        const int64_t row = first + r0 + i;
        if (row < rows) {
            float* at = static_cast<float*>(d.o) + ((b * d.Tq + row / G) * d.H + h * G + row % G) * DH;
            const float inv = 1.f / l[i];
#pragma unroll
            for (int j = 0; j < NC; ++j) at[c + 16 * j] = tiles > 0 ? o[i][j] * inv : 0.f;
        }
    }
}

template <int DH> cudaError_t launch_cf(const CrossDesc& d, cudaStream_t s) {
    using L = CfLayout<DH>;
    static std::atomic<uint64_t> attr{0};
    const cudaError_t e = set_smem_limit_once(cross_f32_kernel<DH>, L::SMEM, attr);
    if (e != cudaSuccess) return e;
    const int64_t qtiles = (d.Tq * (d.H / d.Hkv) + CF_ROWS - 1) / CF_ROWS;
    return launch_dependent(cross_f32_kernel<DH>, dim3((unsigned)(d.B * d.Hkv * qtiles)), dim3(CF_THREADS), L::SMEM, s, d,
                            (float)(d.scale * 1.4426950408889634), (int)qtiles);
}

}  // namespace

bool cross_f32_supported(const CrossDesc& d) {
    if (d.dt != DT_F32 || d.dh % 16 != 0 || d.dh < 32 || d.dh > 128) return false;
    const int64_t lim = 0x7fffffff, qtiles = (d.Tq * (d.H / d.Hkv) + CF_ROWS - 1) / CF_ROWS;
    if (d.Tk > lim - 65536 || qtiles > lim || d.B > lim / (d.Hkv * qtiles) || d.Hkv > lim / qtiles) return false;
    const struct { const void* p; const int64_t* st; } in[] = {{d.q, d.qs}, {d.k, d.ks}, {d.v, d.vs}};
    for (const auto& i : in)
        if ((reinterpret_cast<uintptr_t>(i.p) & 15) || i.st[0] % 4 || i.st[1] % 4 || i.st[2] % 4) return false;
    return true;
}

cudaError_t launch_cross_f32(const CrossDesc& d, cudaStream_t s) {
    switch (d.dh) {
        case 32: return launch_cf<32>(d, s);
        case 48: return launch_cf<48>(d, s);
        case 64: return launch_cf<64>(d, s);
        case 80: return launch_cf<80>(d, s);
        case 96: return launch_cf<96>(d, s);
        case 112: return launch_cf<112>(d, s);
        case 128: return launch_cf<128>(d, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace vit
