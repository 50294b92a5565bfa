// attention_cross_f32.cu -- cross attention in fp32: the mathematics of attention_cross.cu for head
// widths up to 128 in steps of 4.
//
// Products are 3xTF32 (hi hi + hi lo + lo hi, hi rounded to the 11 bits that the tensor cores read,
// lo the rest) on mma.m16n8k8, and sums longer than 16 keys are fp32 additions: the outputs of 8 x 197
// queries over 288 to 577 keys are off by 3.7e-7 in the 2-norm, and by 3.3e-6 when O is summed on the
// tensor cores, which cut sums off instead of rounding them. 53 us at 12 heads of 64 (36 TFLOP/s): bound by each
// warp's own chain of dependent steps, with one or two warps to a scheduler and the tensor pipe of mma.sync 50 % active. It
// is the simple form; attention_tf32.cu, on tcgen05, reaches twice that rate in self attention. A CUDA-core kernel
// took 103 us. Heads wider than 64 and 96 columns spill with sixteen rows to a warp (20 and 196 bytes a thread written, 76
// and 344 read back).
//
// A CTA of four warps walks the keys of one (sequence, key head) 64 at a time, K and V tiles by TMA in
// a ring that all warps read. Query rows are the n side of the products, S^T = K Q^T and
// O^T = V^T P^T, eight or sixteen to a warp (packed row = token * G + head of the group):
//   64 rows per CTA, sixteen to each warp;
//   a CTA with at most 32 or 16 rows (decoding, or the last of a head) is split along the keys: two or four
//   warps share the rows and take every second or fourth group of 16 keys, joined at the end through
//   shared memory. The last five of 197 rows took three quarters of a full CTA's time before, and 100 x
//   20 queries over 577 keys 149 us instead of 107. (Two warps for full CTAs too, of 32 rows, fetch K and V
//   twice as often: 32 x 197 queries 223 us instead of 163.)
// CTAs whose rows four warps share come last, before them all others, of each kind the longest sequences first: 16 x 100
// queries over 1025 keys of 16 heads of 80 221 -> 186 us, 4 x 500 over 577 of 12 heads of 64 75 -> 62. All keys of a
// (sequence, key head) are walked by one CTA: one query over 1100 keys of 12 heads of 64, on 12 SMs, takes 18 us.
// Operands are read 16 bytes at a time from the 128-byte swizzled tiles without bank conflicts:
// the order of the columns in a dot product is free, so thread c takes four consecutive columns
// of its key for two k-steps; so is which column a row of V^T means; and P^T comes out of S^T by
// 8 x 8 transposes of its upper and lower halves.
#include <cuda.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "cross_maps.cuh"
#include "kernels.h"
#include "launch.cuh"
#include "ptx.cuh"

namespace vit {
namespace {

constexpr int CF_KEYS = 64, CF_WARPS = 4, CF_ROWS = 64, CF_BOX = CF_KEYS * 128;   // a box: 32 columns of 64 keys
constexpr int CF_SORT = 128;   // sequences that are put in order of their lengths, at most
static_assert(CF_SORT <= CF_WARPS * 32, "a sequence per thread");

template <int DHT> struct CfLayout {
    static constexpr int NB = DHT / 32;                 // boxes of a K or V tile
    static constexpr int STAGE = 2 * NB * CF_BOX;
    static constexpr int STAGES = DHT <= 64 ? 3 : 2;
    static constexpr int SMEM = STAGES * STAGE + 1024;
    static_assert(SMEM <= 227 * 1024, "shared memory");
};

__device__ __forceinline__ void mma_tf32(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// x as hi + lo: hi its 11 leading bits, rounded to nearest (an infinity stays one), lo exact.
__device__ __forceinline__ void split_tf32(uint32_t x, uint32_t& hi, uint32_t& lo) {
    hi = (x + 0x1000u) & 0xFFFFE000u;
    lo = __float_as_uint(__uint_as_float(x) - __uint_as_float(hi));
}
__device__ __forceinline__ void split_tf32(const uint32_t (&x)[4], uint32_t (&hi)[4], uint32_t (&lo)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) split_tf32(x[i], hi[i], lo[i]);
}

// Lane (r, c) holds row r, columns 2c and 2c + 1 of an 8 x 8 matrix: the same of the transpose.
__device__ __forceinline__ void transpose_8x8_f32(float& x, float& y) {
    const uint32_t a = __float_as_uint(x), b = __float_as_uint(y);
    uint32_t l = __byte_perm(a, b, 0x5410), h = __byte_perm(a, b, 0x7632);
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %0;" : "+r"(l));
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %0;" : "+r"(h));
    x = __uint_as_float(__byte_perm(l, h, 0x5410));
    y = __uint_as_float(__byte_perm(l, h, 0x7632));
}

template <int DHT, int NR>
__global__ void __launch_bounds__(CF_WARPS * 32, DHT <= 64 ? 2 : 1)
cross_f32_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                 const __grid_constant__ CrossDesc d, float scale_log2, int sms, uint32_t* err) {
    using L = CfLayout<DHT>;
    constexpr int NB = L::NB, STAGES = L::STAGES;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t full[STAGES], empty[STAGES];
    __shared__ int abort_word;
    __shared__ uint8_t order[CF_SORT];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    volatile int* abort_flag = &abort_word;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c4 = lane & 3, r8 = lane >> 2;
    const int G = (int)(d.H / d.Hkv), dh = (int)d.dh;
    const int64_t rows = d.Tq * G;
    if (threadIdx.x == 0) {
        for (int i = 0; i < STAGES; ++i) {
            ptx::mbar_init(full + i, 1);
            ptx::mbar_init(empty + i, CF_WARPS);
        }
        abort_word = 0;
        ptx::fence_mbar_init();
        ptx::prefetch_tensormap(&tmK);
        ptx::prefetch_tensormap(&tmV);
    }
    __syncthreads();
    griddep_wait();
    griddep_launch_dependents();

    // Work in order: tiles of more than NR * 8 rows, then the last ones of all heads that have fewer and that four warps
    // share; of each, the longest sequences first. The CTAs that come to sit beside the first on each SM go backwards through theirs.
    const bool sorted = sms > 0;
    if (sorted) {
        int* lens = reinterpret_cast<int*>(smem);   // before anything is copied there
        const int i = threadIdx.x, n = (int)d.B;
        if (i < n) lens[i] = min(max(__ldg(d.kv_lens + i), 0), (int)d.Tk);
        __syncthreads();
        int before = 0;
        if (i < n)
            for (int j = 0; j < n; ++j) before += lens[j] > lens[i] || (lens[j] == lens[i] && j < i);
        if (i < n) order[before] = (uint8_t)i;
        ptx::fence_proxy_async_smem();
        __syncthreads();
    }
    int at = blockIdx.x;
    if (sorted && DHT <= 64 && at >= sms && at < 2 * sms) at = sms + min(2 * sms, (int)gridDim.x) - 1 - at;
    const int heads = (int)(d.B * d.Hkv), whole = (int)((rows - NR * 8 + CF_ROWS - 1) / CF_ROWS);   // tiles before the last kind
    int qt, bh;
    if (at < whole * heads) {
        bh = at / whole;
        qt = at - bh * whole;
    } else {
        bh = at - whole * heads;
        qt = whole;
    }
    const int b = sorted ? order[bh / (int)d.Hkv] : bh / (int)d.Hkv, h = bh % (int)d.Hkv;
    const int64_t tile0 = (int64_t)qt * CF_ROWS;
    const int W = rows - tile0 <= NR * 8 ? 4 : rows - tile0 <= NR * 16 ? 2 : 1;   // warps that share rows
    const int64_t first = tile0 + warp / W * (NR * 8);

    int len = (int)d.Tk;
    if (d.kv_lens) len = min(max(__ldg(d.kv_lens + b), 0), (int)d.Tk);
    const int tiles = (len + CF_KEYS - 1) / CF_KEYS;
    const int kb = d.ks[0] ? b : 0, kh = d.ks[2] ? h : 0, vb = d.vs[0] ? b : 0, vh = d.vs[2] ? h : 0;
    auto request = [&](int t) {   // thread 0
        uint8_t* dst = smem + (t % STAGES) * L::STAGE;
        uint64_t* bar = full + t % STAGES;
        ptx::mbar_arrive_expect_tx(bar, L::STAGE);
#pragma unroll
        for (int x = 0; x < NB; ++x) {
            ptx::tma_load_4d(dst + x * CF_BOX, &tmK, bar, x * 32, kh, t * CF_KEYS, kb);
            ptx::tma_load_4d(dst + (NB + x) * CF_BOX, &tmV, bar, x * 32, vh, t * CF_KEYS, vb);
        }
    };
    if (threadIdx.x == 0)
        for (int t = 0; t < STAGES && t < tiles; ++t) request(t);

    // query rows first + 8 i + r8: columns 32 x + 4 (2 c4 + u) + {0 .. 3}
    uint4 q[NR][2 * NB];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        const int64_t r = first + 8 * i + r8;
        const float* qr = static_cast<const float*>(d.q) + b * d.qs[0] + (r / G) * d.qs[1] + (h * G + r % G) * d.qs[2];
#pragma unroll
        for (int c = 0; c < 2 * NB; ++c) {
            const int col = (c >> 1) * 32 + (2 * c4 + (c & 1)) * 4;
            q[i][c] = r < rows && col < dh ? __ldg(reinterpret_cast<const uint4*>(qr + col)) : make_uint4(0, 0, 0, 0);
        }
    }
    // rows 8 i + 2 c4 + e: maximum, this thread's part of the sum; O^T of the two m-tiles of each box
    float o[NR][2 * NB][4], m[NR][2], l[NR][2];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        m[i][0] = m[i][1] = -INFINITY;
        l[i][0] = l[i][1] = 0.f;
#pragma unroll
        for (int j = 0; j < 2 * NB; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][j][e] = 0.f;
    }
    const bool live = first < rows;
    bool ok = true;
    int t = 0;
    for (; t < tiles; ++t) {
        const uint32_t st = t % STAGES, par = (t / STAGES) & 1;
        ok = __all_sync(0xffffffffu, ptx::mbar_wait_bounded(full + st, par, abort_flag));
        if (!ok) break;
        const uint8_t* sk = smem + st * L::STAGE;
        const uint8_t* sv = sk + NB * CF_BOX;
        // 16 keys at a time; the key groups of a warp
        const int share = CF_KEYS / 16 / W, g0 = warp % W * share, g1 = g0 + share;
#pragma unroll 1
        for (int g = g0; g < g1; ++g) {
            const int valid = len - t * CF_KEYS - g * 16;
            if (!live || valid <= 0) break;
            // hi hi, lo hi and hi lo apart: shorter chains of dependent products
            float s[NR][4] = {}, s2[NR][4] = {}, s3[NR][4] = {};
#pragma unroll
            for (int c = 0; c < 2 * NB; ++c) {
                // 16-byte unit i of key u at i ^ (u % 8)
                const uint8_t* at = sk + (c >> 1) * CF_BOX + (g * 16 + r8) * 128 + (((2 * c4 + (c & 1)) ^ r8) << 4);
                const uint4 k0 = *reinterpret_cast<const uint4*>(at), k1 = *reinterpret_cast<const uint4*>(at + 1024);
                uint32_t a0[4], a1[4], l0[4], l1[4];
                split_tf32({k0.x, k1.x, k0.y, k1.y}, a0, l0);
                split_tf32({k0.z, k1.z, k0.w, k1.w}, a1, l1);
#pragma unroll
                for (int i = 0; i < NR; ++i) {
                    uint32_t x[4], y[4];
                    split_tf32({q[i][c].x, q[i][c].y, q[i][c].z, q[i][c].w}, x, y);
                    mma_tf32(s[i], a0, x[0], x[1]);
                    mma_tf32(s2[i], l0, x[0], x[1]);
                    mma_tf32(s3[i], a0, y[0], y[1]);
                    mma_tf32(s[i], a1, x[2], x[3]);
                    mma_tf32(s2[i], l1, x[2], x[3]);
                    mma_tf32(s3[i], a1, y[2], y[3]);
                }
            }
            float alpha[NR][2];
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                float mx[2] = {m[i][0], m[i][1]};
#pragma unroll
                for (int e = 0; e < 4; ++e) {   // key r8 + 8 (e / 2), row 2 c4 + e % 2
                    // an infinite hi hi stands as it is: the low part of an infinity is NaN
                    if (fabsf(s[i][e]) < INFINITY) s[i][e] += s2[i][e] + s3[i][e];
                    // rounded like the maximum that is taken off below: behind an exact product a maximum of 2^31
                    // and more is off by more than the exponential's range
                    s[i][e] = __fmul_rn(s[i][e], scale_log2);
                    if (r8 + 8 * (e >> 1) < valid) mx[e & 1] = fmaxf(mx[e & 1], s[i][e]);
                }
#pragma unroll
                for (int w = 4; w < 32; w *= 2) {
                    mx[0] = fmaxf(mx[0], __shfl_xor_sync(0xffffffffu, mx[0], w));
                    mx[1] = fmaxf(mx[1], __shfl_xor_sync(0xffffffffu, mx[1], w));
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    alpha[i][e] = mx[e] > m[i][e] ? exp2_approx(m[i][e] - mx[e]) : 1.f;
                    m[i][e] = mx[e];
                    if (mx[e] == -INFINITY) mx[e] = 0.f;   // only infinite scores so far: weights of zero
                }
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    s[i][e] = r8 + 8 * (e >> 1) < valid ? exp2_approx(s[i][e] - mx[e & 1]) : 0.f;
                l[i][0] = l[i][0] * alpha[i][0] + (s[i][0] + s[i][2]);
                l[i][1] = l[i][1] * alpha[i][1] + (s[i][1] + s[i][3]);
                transpose_8x8_f32(s[i][0], s[i][1]);   // now row r8, keys 2 c4 and 2 c4 + 1
                transpose_8x8_f32(s[i][2], s[i][3]);   // and 8 on
            }
            // the tensor cores cut sums off instead of rounding them, which adds up over hundreds of
            // keys: the 16 keys' products start from zero and are added to O here
#pragma unroll
            for (int x = 0; x < NB; ++x) {
                float y[NR][2][4] = {};
#pragma unroll
                for (int k = 0; k < 2; ++k) {   // eight keys
                    const int u = g * 16 + k * 8 + 2 * c4;
                    const uint8_t* at = sv + x * CF_BOX + u * 128;
                    uint4 v0 = *reinterpret_cast<const uint4*>(at + ((r8 ^ (u & 7)) << 4));
                    uint4 v1 = *reinterpret_cast<const uint4*>(at + 128 + ((r8 ^ ((u + 1) & 7)) << 4));
                    if (valid < 16) {   // rows past the length may hold anything, and 0 * NaN is NaN
                        if (k * 8 + 2 * c4 >= valid) v0 = make_uint4(0, 0, 0, 0);
                        if (k * 8 + 2 * c4 + 1 >= valid) v1 = make_uint4(0, 0, 0, 0);
                    }
                    uint32_t a0[4], a1[4], l0[4], l1[4];
                    split_tf32({v0.x, v0.y, v1.x, v1.y}, a0, l0);
                    split_tf32({v0.z, v0.w, v1.z, v1.w}, a1, l1);
#pragma unroll
                    for (int i = 0; i < NR; ++i) {
                        uint32_t p0, p1, n0, n1;
                        split_tf32(__float_as_uint(s[i][2 * k]), p0, n0);
                        split_tf32(__float_as_uint(s[i][2 * k + 1]), p1, n1);
                        mma_tf32(y[i][0], l0, p0, p1);
                        mma_tf32(y[i][1], l1, p0, p1);
                        mma_tf32(y[i][0], a0, n0, n1);
                        mma_tf32(y[i][1], a1, n0, n1);
                        mma_tf32(y[i][0], a0, p0, p1);
                        mma_tf32(y[i][1], a1, p0, p1);
                    }
                }
#pragma unroll
                for (int i = 0; i < NR; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            o[i][2 * x + j][e] = fmaf(o[i][2 * x + j][e], alpha[i][e & 1], y[i][j][e]);
            }
        }
        __syncwarp();   // this warp has read the stage
        if (lane == 0) ptx::mbar_arrive(empty + st);
        if (threadIdx.x == 0 && t > 0 && t - 1 + STAGES < tiles) {   // the tile before: the other warps are done too
            ok = ptx::mbar_wait_bounded(empty + (t - 1) % STAGES, ((t - 1) / STAGES) & 1, abort_flag);
            if (ok) request(t - 1 + STAGES);
        }
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
    }
    if (!ok) {
        if (lane == 0 && err) atomicOr(err, ERRBIT_TIMEOUT_ATTENTION);
        *abort_flag = 1;
        // copies in flight land before the CTA can exit
        if (threadIdx.x == 0)
            for (int i = t; i < t + STAGES && i < tiles; ++i)
                ptx::mbar_wait_bounded(full + i % STAGES, (i / STAGES) & 1, nullptr);
    }

#pragma unroll
    for (int i = 0; i < NR; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int w = 4; w < 32; w *= 2) l[i][e] += __shfl_xor_sync(0xffffffffu, l[i][e], w);
    auto out = [&](int64_t r) {
        return static_cast<float*>(d.o) + ((b * d.Tq + r / G) * d.H + h * G + r % G) * dh;
    };
    // [0] and [2] of m-tile j are columns 16 j' ..: 32 x + 4 r8 + 2 (j % 2) and the next, row 2 c4; [1] and [3]
    // the same of row 2 c4 + 1
    if (W == 1) {
#pragma unroll
        for (int i = 0; i < NR; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int64_t r = first + 8 * i + 2 * c4 + e;
                if (r >= rows) continue;
                const float inv = tiles > 0 ? 1.f / l[i][e] : 0.f;
                float* at = out(r);
#pragma unroll
                for (int x = 0; x < NB; ++x) {
                    const int col = 32 * x + 4 * r8;
                    const float v[4] = {o[i][2 * x][e], o[i][2 * x][2 + e], o[i][2 * x + 1][e], o[i][2 * x + 1][2 + e]};
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (col + j < dh) at[col + j] = tiles > 0 ? v[j] * inv : 0.f;
                }
            }
    } else {
        // join the warps that share rows: O, m and l of each over the ring, which nobody reads any more
        constexpr int PIECE = NR * 8 * (DHT + 2);
        float* sm = reinterpret_cast<float*>(smem);
        static_assert(CF_WARPS * PIECE * 4 <= L::STAGES * L::STAGE, "join");
        __syncthreads();
        float* w0 = sm + warp * PIECE;
#pragma unroll
        for (int i = 0; i < NR; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = 8 * i + 2 * c4 + e;
#pragma unroll
                for (int x = 0; x < NB; ++x) {
                    float* at = w0 + r * DHT + 32 * x + 4 * r8;
                    at[0] = o[i][2 * x][e];
                    at[1] = o[i][2 * x][2 + e];
                    at[2] = o[i][2 * x + 1][e];
                    at[3] = o[i][2 * x + 1][2 + e];
                }
                if (r8 == 0) {
                    w0[NR * 8 * DHT + r] = m[i][e];
                    w0[NR * 8 * DHT + NR * 8 + r] = l[i][e];
                }
            }
        __syncthreads();
        for (int x = threadIdx.x; x < (int)(rows - tile0) * dh; x += CF_WARPS * 32) {
            const int rt = x / dh, c = x - rt * dh, r = rt % (NR * 8);
            const float* sg = sm + rt / (NR * 8) * W * PIECE;
            float mw[CF_WARPS], mx = -INFINITY;
#pragma unroll
            for (int w = 0; w < CF_WARPS; ++w) {
                mw[w] = w < W ? sg[w * PIECE + NR * 8 * DHT + r] : -INFINITY;
                mx = fmaxf(mx, mw[w]);
            }
            const float base = mx == -INFINITY ? 0.f : mx;
            float acc = 0.f, sum = 0.f;
#pragma unroll
            for (int w = 0; w < CF_WARPS; ++w) {
                if (w >= W) break;
                const float f = exp2_approx(mw[w] - base);
                acc = fmaf(f, sg[w * PIECE + r * DHT + c], acc);
                sum = fmaf(f, sg[w * PIECE + NR * 8 * DHT + NR * 8 + r], sum);
            }
            out(tile0 + rt)[c] = tiles > 0 ? acc / sum : 0.f;
        }
    }
}

template <int DHT, int NR> cudaError_t launch_cf_inst(const CrossDesc& d, const DeviceInfo& dev, cudaStream_t s) {
    using L = CfLayout<DHT>;
    auto k = cross_f32_kernel<DHT, NR>;
    static std::atomic<uint64_t> attr{0};
    const cudaError_t e = set_smem_limit_once(k, L::SMEM, attr);
    if (e != cudaSuccess) return e;
    alignas(64) CUtensorMap mk, mv;
    if (!ct_map_f32(&mk, d.k, d.ks, d.B, d.Tk, d.Hkv, d.dh, CF_KEYS) ||
        !ct_map_f32(&mv, d.v, d.vs, d.B, d.Tk, d.Hkv, d.dh, CF_KEYS))
        return cudaErrorInvalidValue;
    const int64_t qtiles = (d.Tq * (d.H / d.Hkv) + CF_ROWS - 1) / CF_ROWS;
    const bool sorted = d.kv_lens && d.B > 1 && d.B <= CF_SORT && d.B * d.Hkv * qtiles > dev.num_sms;
    return launch_dependent(k, dim3((unsigned)(d.B * d.Hkv * qtiles)), dim3(CF_WARPS * 32), L::SMEM, s, mk, mv, d,
                            (float)(d.scale * 1.4426950408889634),
                            sorted ? dev.num_sms : 0, dev.err_word);
}

template <int DHT> cudaError_t launch_cf(const CrossDesc& d, const DeviceInfo& dev, cudaStream_t s) {
    return d.Tq * (d.H / d.Hkv) <= 8 ? launch_cf_inst<DHT, 1>(d, dev, s) : launch_cf_inst<DHT, 2>(d, dev, s);
}

}  // namespace

bool cross_f32_supported(const CrossDesc& d) {
    if (d.dt != DT_F32 || d.dh % 4 != 0 || d.dh > 128) return false;
    const int64_t lim = 0x7fffffff, qtiles = (d.Tq * (d.H / d.Hkv) + CF_ROWS - 1) / CF_ROWS;
    if (d.Tk > lim - 65536 || qtiles > lim || d.Hkv > lim / qtiles || d.B > lim / (d.Hkv * qtiles)) return false;
    if ((reinterpret_cast<uintptr_t>(d.q) & 15) || d.qs[0] % 4 || d.qs[1] % 4 || d.qs[2] % 4) return false;
    return ct_strides_ok(d.k, d.ks, d.Tk, 4) && ct_strides_ok(d.v, d.vs, d.Tk, 4) && ct_encode_fn() != nullptr;
}

cudaError_t launch_cross_f32(const CrossDesc& d, const DeviceInfo& dev, cudaStream_t s) {
    if (d.dh <= 32) return launch_cf<32>(d, dev, s);
    if (d.dh <= 64) return launch_cf<64>(d, dev, s);
    if (d.dh <= 96) return launch_cf<96>(d, dev, s);
    return launch_cf<128>(d, dev, s);
}

}  // namespace vit
