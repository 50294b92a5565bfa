// attention_cross_rows.cu -- cross attention of few queries (decoding): the mathematics of
// attention_cross.cu where one key head serves at most 16 query rows (Tq * G <= 16), bf16,
// head width up to 128 in steps of 8.
//
// Bound by reading K and V once. The keys of a (sequence, key head) are dealt out in tiles of 16
// to the warps of one CTA or of a cluster of CTAs; every warp keeps its own running maximum, sum
// and output rows, joined at the end through shared memory and, between the CTAs of a cluster,
// distributed shared memory: no workspace, one launch, the same order of additions every time.
//
// 32 sequences of 288 to 577 keys, 16 heads of 64: 12.9 us (4.3 TB/s); 64 of 577 keys: 27 us (5.6 TB/s).
//
// The weights are rounded to bf16 for the second product (their sum is not): the matrix instruction takes both operands
// in one type, and V is bf16. The outputs' error in the 2-norm becomes 2.1e-3 instead of the 1.7e-3 of rounding them alone.
//
// Each warp streams its tiles through a ring of its own in shared memory: its lane 0 asks for the
// tile two or three ahead by TMA as soon as the warp has used up a stage.
//
// Products are mma.m16n8k16 with the query rows as the n side, S^T = K Q^T and O^T = V^T P^T: eight
// rows (NR = 1) or sixteen, where the m side would compute sixteen for one. Operands are read
// 16 bytes at a time from the 128-byte swizzled tiles, without bank conflicts and without
// transposing V:
//  - the order of the columns in a dot product is free, so the thread that owns columns 2c, 2c+1,
//    2c+8, 2c+9 of a k-step takes 8 consecutive columns of its key (two k-steps), and the same
//    ones of its query row: units 2c and 2c+1 of the row's eight;
//  - so is which output column a row of V^T means: thread r reads columns 8r to 8r+7 of four
//    keys, interleaves key pairs with byte permutes, and columns 8r + 2t, 8r + 2t + 1 become rows
//    r and r + 8 of m-tile t;
//  - P^T comes out of S^T by one 8 x 8 transpose (movmatrix) per 8 keys.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "cross_maps.cuh"
#include "kernels.h"
#include "launch.cuh"
#include "mma_rows.cuh"
#include "ptx.cuh"

namespace vit {
namespace {

constexpr int CR_ROWS = 16, CR_MAXZ = 8;

// DHT: the head width rounded up to 64 or 128; columns past dh are zeros.
template <int DHT, int NR, int NW, int KEYS, int CR_STAGES, int MINB>
__global__ void __launch_bounds__(NW * 32, MINB)
cross_rows_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                  const __grid_constant__ CrossDesc d, float scale_log2, int Z, uint32_t* err) {
    constexpr int NCH = DHT / 64, NT = KEYS / 16, CR_STAGE = KEYS * NCH * 256;
    constexpr int BOX = KEYS * 128;   // 64 columns of one tile
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t bars[NW][CR_STAGES];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c4 = lane & 3, r8 = lane >> 2;
    const int z = Z > 1 ? (int)ptx::cluster_ctarank() : 0;
    const int bh = blockIdx.x / Z, b = bh / (int)d.Hkv, h = bh % (int)d.Hkv;
    const int G = (int)(d.H / d.Hkv), R = (int)d.Tq * G, dh = (int)d.dh;
    uint64_t* bar = bars[warp];
    uint8_t* ring = smem + warp * CR_STAGES * CR_STAGE;
    // once a warp's keys are done, over its ring: O (R x dh), m and l (R each); behind the rings
    // this CTA's joined O, m and l
    constexpr int piece = CR_STAGES * CR_STAGE / 4;
    float* sm = reinterpret_cast<float*>(smem);
    float* wO = sm + warp * piece;
    float* jO = sm + NW * piece;
    static_assert(NR * 8 * (DHT + 2) <= piece, "output rows in a ring");
    if (lane == 0) {
        for (int i = 0; i < CR_STAGES; ++i) ptx::mbar_init(bar + i, 1);
        ptx::fence_mbar_init();
        ptx::prefetch_tensormap(&tmK);
        ptx::prefetch_tensormap(&tmV);
    }
    __syncwarp();
    griddep_wait();
    griddep_launch_dependents();

    int len = (int)d.Tk;
    if (d.kv_lens) len = min(max(__ldg(d.kv_lens + b), 0), (int)d.Tk);
    // tiles of this warp: first, first + stride, ...
    const int tiles = (len + KEYS - 1) / KEYS, first = z * NW + warp, stride = Z * NW;
    const int kb = d.ks[0] ? b : 0, kh = d.ks[2] ? h : 0, vb = d.vs[0] ? b : 0, vh = d.vs[2] ? h : 0;
    auto request = [&](int tile, int st) {   // lane 0
        uint8_t* dst = ring + st * CR_STAGE;
        ptx::mbar_arrive_expect_tx(bar + st, CR_STAGE);
#pragma unroll
        for (int c = 0; c < NCH; ++c) ptx::tma_load_4d(dst + c * BOX, &tmK, bar + st, c * 64, kh, tile * KEYS, kb);
#pragma unroll
        for (int c = 0; c < NCH; ++c)
            ptx::tma_load_4d(dst + CR_STAGE / 2 + c * BOX, &tmV, bar + st, c * 64, vh, tile * KEYS, vb);
    };
    if (lane == 0)
        for (int i = 0; i < CR_STAGES; ++i)
            if (first + i * stride < tiles) request(first + i * stride, i);

    // query rows 8 i + r8; packed row = token * G + head of the group
    uint4 q[NR][2 * NCH];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        const int r = r8 + 8 * i;
        const __nv_bfloat16* qr = static_cast<const __nv_bfloat16*>(d.q) + b * d.qs[0] + (r / G) * d.qs[1] +
                                  (int64_t)(h * G + r % G) * d.qs[2];
#pragma unroll
        for (int c = 0; c < 2 * NCH; ++c) {
            const int col = (c >> 1) * 64 + (2 * c4 + (c & 1)) * 8;
            q[i][c] = r < R && col < dh ? *reinterpret_cast<const uint4*>(qr + col) : make_uint4(0, 0, 0, 0);
        }
    }

    // rows 8 i + 2 c4 + e: maximum, this thread's part of the sum; O^T of m-tile t of piece c
    float o[NR][NCH * 4][4], m[NR][2], l[NR][2];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        m[i][0] = m[i][1] = -INFINITY;
        l[i][0] = l[i][1] = 0.f;
#pragma unroll
        for (int j = 0; j < NCH * 4; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][j][e] = 0.f;
    }

    uint32_t it = 0;
    bool ok = true;
    for (int tile = first; tile < tiles; tile += stride, ++it) {
        const uint32_t st = it % CR_STAGES;
        ok = __all_sync(0xffffffffu, ptx::mbar_wait_bounded(bar + st, (it / CR_STAGES) & 1, nullptr));
        if (!ok) break;
        const uint8_t* sk = ring + st * CR_STAGE;
        const uint8_t* sv = sk + CR_STAGE / 2;
        const int valid = len - tile * KEYS;
        // s[i][t]: keys 16 t + r8 (0, 1) and 16 t + 8 + r8 (2, 3), rows 8 i + 2 c4 + {0, 1}
        float s[NR][NT][4];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            float sp[NR][2][4] = {};   // even and odd k-steps: shorter chains of dependent products
#pragma unroll
            for (int c = 0; c < 2 * NCH; ++c) {
                // 16-byte unit i of key u at i ^ (u % 8)
                const uint8_t* at = sk + (c >> 1) * BOX + (t * 16 + r8) * 128 + (((2 * c4 + (c & 1)) ^ r8) << 4);
                const uint4 k0 = *reinterpret_cast<const uint4*>(at), k1 = *reinterpret_cast<const uint4*>(at + 1024);
                const uint32_t a0[4] = {k0.x, k1.x, k0.y, k1.y}, a1[4] = {k0.z, k1.z, k0.w, k1.w};
#pragma unroll
                for (int i = 0; i < NR; ++i) {
                    mma_16816(sp[i][0], a0, q[i][c].x, q[i][c].y);
                    mma_16816(sp[i][1], a1, q[i][c].z, q[i][c].w);
                }
            }
#pragma unroll
            for (int i = 0; i < NR; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[i][t][e] = __fmul_rn(sp[i][0][e] + sp[i][1][e], scale_log2);   // rounded like the maximum
        }
        if (valid < KEYS) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (t * 16 + (e >> 1) * 8 + r8 >= valid)
#pragma unroll
                        for (int i = 0; i < NR; ++i) s[i][t][e] = -INFINITY;
        }
        uint32_t pt[NR][NT][2];   // P^T: row 8 i + r8, keys 16 t + 2 c4 + {0, 1} and + 8
        bool grew = false;
        float alpha[NR][2];
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            float mx[2] = {m[i][0], m[i][1]};
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) mx[e & 1] = fmaxf(mx[e & 1], s[i][t][e]);
#pragma unroll
            for (int w = 4; w < 32; w *= 2) {
                mx[0] = fmaxf(mx[0], __shfl_xor_sync(0xffffffffu, mx[0], w));
                mx[1] = fmaxf(mx[1], __shfl_xor_sync(0xffffffffu, mx[1], w));
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                alpha[i][e] = mx[e] > m[i][e] ? exp2_approx(m[i][e] - mx[e]) : 1.f;
                grew = grew || mx[e] > m[i][e];
                m[i][e] = mx[e];
                if (mx[e] == -INFINITY) mx[e] = 0.f;   // only infinite scores so far: weights of zero
            }
            float sum[2] = {0.f, 0.f};
#pragma unroll
            for (int t = 0; t < NT; ++t) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    s[i][t][e] = exp2_approx(s[i][t][e] - mx[e & 1]);
                    sum[e & 1] += s[i][t][e];
                }
                pt[i][t][0] = transpose_8x8(pack_bf16x2(s[i][t][0], s[i][t][1]));
                pt[i][t][1] = transpose_8x8(pack_bf16x2(s[i][t][2], s[i][t][3]));
            }
            l[i][0] = l[i][0] * alpha[i][0] + sum[0];
            l[i][1] = l[i][1] * alpha[i][1] + sum[1];
        }
        if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
            for (int i = 0; i < NR; ++i)
#pragma unroll
                for (int j = 0; j < NCH * 4; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[i][j][e] *= alpha[i][e & 1];
        }
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int c = 0; c < NCH; ++c) {
                uint4 w[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {   // keys 2 c4, 2 c4 + 1, 2 c4 + 8, 2 c4 + 9 of this 16
                    const int u = t * 16 + 2 * c4 + (k & 1) + 8 * (k >> 1);
                    w[k] = *reinterpret_cast<const uint4*>(sv + c * BOX + u * 128 + ((r8 ^ (u & 7)) << 4));
                }
                if (valid < KEYS) {   // rows past the length may hold anything, and 0 * NaN is NaN
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (t * 16 + 2 * c4 + (k & 1) + 8 * (k >> 1) >= valid) w[k] = make_uint4(0, 0, 0, 0);
                }
                const uint32_t* w0 = reinterpret_cast<const uint32_t*>(&w[0]);
                const uint32_t* w1 = reinterpret_cast<const uint32_t*>(&w[1]);
                const uint32_t* w2 = reinterpret_cast<const uint32_t*>(&w[2]);
                const uint32_t* w3 = reinterpret_cast<const uint32_t*>(&w[3]);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t a[4] = {__byte_perm(w0[e], w1[e], 0x5410), __byte_perm(w0[e], w1[e], 0x7632),
                                           __byte_perm(w2[e], w3[e], 0x5410), __byte_perm(w2[e], w3[e], 0x7632)};
#pragma unroll
                    for (int i = 0; i < NR; ++i) mma_16816(o[i][c * 4 + e], a, pt[i][t][0], pt[i][t][1]);
                }
            }
        __syncwarp();   // the stage has been read
        const int next = tile + CR_STAGES * stride;
        if (lane == 0 && next < tiles) request(next, st);
    }
    if (!ok && lane == 0) {
        if (err) atomicOr(err, ERRBIT_TIMEOUT_ATTENTION);
        // copies in flight land before the CTA can exit
        for (uint32_t i = it; i < it + CR_STAGES; ++i)
            if (first + (int)i * stride < tiles) ptx::mbar_wait_bounded(bar + i % CR_STAGES, (i / CR_STAGES) & 1, nullptr);
    }
    __syncwarp();

    // this warp's rows: [0], [2] are columns 8 r8 + 2 t, + 1 of row 8 i + 2 c4; [1], [3] of the next row
#pragma unroll
    for (int i = 0; i < NR; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int w = 4; w < 32; w *= 2) l[i][e] += __shfl_xor_sync(0xffffffffu, l[i][e], w);
            const int r = 8 * i + 2 * c4 + e;
            if (r >= R) continue;
#pragma unroll
            for (int c = 0; c < NCH; ++c)
                if (c * 64 + r8 * 8 < dh) {
                    float* at = wO + r * dh + c * 64 + r8 * 8;
                    *reinterpret_cast<float2*>(at) = make_float2(o[i][c * 4][e], o[i][c * 4][2 + e]);
                    *reinterpret_cast<float2*>(at + 2) = make_float2(o[i][c * 4 + 1][e], o[i][c * 4 + 1][2 + e]);
                    *reinterpret_cast<float2*>(at + 4) = make_float2(o[i][c * 4 + 2][e], o[i][c * 4 + 2][2 + e]);
                    *reinterpret_cast<float2*>(at + 6) = make_float2(o[i][c * 4 + 3][e], o[i][c * 4 + 3][2 + e]);
                }
            if (r8 == 0) {
                wO[R * dh + r] = m[i][e];
                wO[R * dh + R + r] = l[i][e];
            }
        }
    __syncthreads();

    // join the warps' rows, two columns per thread and step, every operand asked for at once
    auto store = [&](int r, int col, float x, float y) {
        __nv_bfloat16* at = static_cast<__nv_bfloat16*>(d.o) + (((int64_t)b * d.Tq + r / G) * d.H + h * G + r % G) * dh + col;
        if ((reinterpret_cast<uintptr_t>(at) & 3) == 0) {
            *reinterpret_cast<uint32_t*>(at) = pack_bf16x2(x, y);
        } else {
            at[0] = __float2bfloat16_rn(x);
            at[1] = __float2bfloat16_rn(y);
        }
    };
    for (int i = threadIdx.x * 2; i < R * dh; i += NW * 64) {
        const int r = i / dh;
        float mw[NW], mx = -INFINITY;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            mw[w] = sm[w * piece + R * dh + r];
            mx = fmaxf(mx, mw[w]);
        }
        const float base = mx == -INFINITY ? 0.f : mx;
        float2 acc = make_float2(0.f, 0.f);
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const float f = exp2_approx(mw[w] - base);
            const float2 v = *reinterpret_cast<const float2*>(sm + w * piece + i);
            acc.x = fmaf(f, v.x, acc.x);
            acc.y = fmaf(f, v.y, acc.y);
            sum = fmaf(f, sm[w * piece + R * dh + R + r], sum);
        }
        if (Z == 1) {
            const float inv = len > 0 ? 1.f / sum : 0.f;
            store(r, i - r * dh, len > 0 ? acc.x * inv : 0.f, len > 0 ? acc.y * inv : 0.f);
        } else {
            *reinterpret_cast<float2*>(jO + i) = acc;
            if (i == r * dh) {
                jO[R * dh + r] = mx;
                jO[R * dh + R + r] = sum;
            }
        }
    }
    if (Z > 1) {
        ptx::cluster_sync();   // every CTA's joined rows are in place
        const uint32_t own = ptx::smem_addr(jO);
        for (int i = (z * NW * 32 + threadIdx.x) * 2; i < R * dh; i += Z * NW * 64) {
            const int r = i / dh;
            float mz[CR_MAXZ], lz[CR_MAXZ];
            float2 oz[CR_MAXZ];
#pragma unroll
            for (int y = 0; y < CR_MAXZ; ++y) {
                const uint32_t at = ptx::mapa_shared(own, y < Z ? y : 0);
                mz[y] = ptx::ld_cluster_f32(at + (R * dh + r) * 4);
                lz[y] = ptx::ld_cluster_f32(at + (R * dh + R + r) * 4);
                oz[y].x = ptx::ld_cluster_f32(at + i * 4);
                oz[y].y = ptx::ld_cluster_f32(at + i * 4 + 4);
                if (y >= Z) mz[y] = -INFINITY;
            }
            float mx = -INFINITY;
#pragma unroll
            for (int y = 0; y < CR_MAXZ; ++y) mx = fmaxf(mx, mz[y]);
            const float base = mx == -INFINITY ? 0.f : mx;
            float ax = 0.f, ay = 0.f, sum = 0.f;
#pragma unroll
            for (int y = 0; y < CR_MAXZ; ++y) {
                if (y >= Z) break;
                const float f = exp2_approx(mz[y] - base);
                ax = fmaf(f, oz[y].x, ax);
                ay = fmaf(f, oz[y].y, ay);
                sum = fmaf(f, lz[y], sum);
            }
            const float inv = 1.f / sum;
            store(r, i - r * dh, len > 0 ? ax * inv : 0.f, len > 0 ? ay * inv : 0.f);
        }
        __syncwarp();
        ptx::cluster_sync();   // no CTA leaves while another reads its shared memory
    }
}

template <int DHT, int NR, int NW, int KEYS, int CR_STAGES, int MINB>
cudaError_t launch_rows(const CrossDesc& d, const DeviceInfo& dev, int Z, cudaStream_t s) {
    constexpr int CR_STAGE = KEYS * (DHT / 64) * 256;
    auto k = cross_rows_kernel<DHT, NR, NW, KEYS, CR_STAGES, MINB>;
    static std::atomic<uint64_t> attr{0};
    constexpr int smem = NW * CR_STAGES * CR_STAGE + NR * 8 * (DHT + 2) * 4 + 1024;
    cudaError_t e = set_smem_limit_once(k, smem, attr);
    if (e != cudaSuccess) return e;
    alignas(64) CUtensorMap mk, mv;
    if (!ct_map(&mk, d.k, d.ks, d.B, d.Tk, d.Hkv, d.dh, 1, KEYS, CU_TENSOR_MAP_L2_PROMOTION_L2_256B) ||
        !ct_map(&mv, d.v, d.vs, d.B, d.Tk, d.Hkv, d.dh, 1, KEYS, CU_TENSOR_MAP_L2_PROMOTION_L2_256B))
        return cudaErrorInvalidValue;
    const float sl2 = (float)(d.scale * 1.4426950408889634);
    const dim3 grid((unsigned)(d.B * d.Hkv * Z)), block(NW * 32);
    if (Z == 1) return launch_dependent(k, grid, block, smem, s, mk, mv, d, sl2, 1, dev.err_word);
    return launch_dependent_cluster(k, grid, block, Z, smem, s, mk, mv, d, sl2, Z, dev.err_word);
}

}  // namespace

bool cross_rows_supported(const CrossDesc& d) {
    if (d.dt != DT_BF16 || d.dh % 8 != 0 || d.dh > 128 || d.Tq * (d.H / d.Hkv) > CR_ROWS) return false;
    if (d.B > 0x7fffffff / 8 / d.Hkv || d.Tk > 0x7fffffff - 65536) return false;
    if ((reinterpret_cast<uintptr_t>(d.q) & 15) || d.qs[0] % 8 || d.qs[1] % 8 || d.qs[2] % 8) return false;
    return ct_strides_ok(d.k, d.ks, d.Tk) && ct_strides_ok(d.v, d.vs, d.Tk) && ct_encode_fn() != nullptr;
}

cudaError_t launch_cross_rows(const CrossDesc& d, const DeviceInfo& dev, cudaStream_t s) {
    // A warp takes 0.64 us for a tile, whatever the latency of its copies, so what counts is to
    // have some four warps on every SM or more, each with two tiles at least. Measured at 8192 keys
    // (us at 1 / 2 / 4 / 8 CTAs per key head): 64 heads of 64, four warps: 54 / 30 / 23.0 / 25; 16
    // heads of 128, eight warps: 52 / 30 / 18.1 / 25. Clusters of eight CTAs that fill an SM each do
    // not pack into the GPU's SM groups, hence the smaller limit for them. 512 heads of 64, 577 keys
    // (one wave of four CTAs per SM): 13.1 / 18 / 22 / 37.
    const int64_t heads = d.B * d.Hkv, sms = dev.num_sms;
    const bool narrow = d.dh <= 64;
    const int warps = narrow || heads > sms / 2 ? 4 : 8;
    const int64_t ctas = narrow || warps == 4 ? 2 * sms : sms;   // aimed at; more CTAs only add joins
    int Z = 1;
    while (Z < CR_MAXZ && heads * Z * 2 <= ctas && d.Tk >= (int64_t)Z * 2 * warps * 16 * 2) Z *= 2;
    if (warps == 8 && Z == 8 && heads * 8 > sms / 2) Z = 4;
    if (d.Tq * (d.H / d.Hkv) > 8)
        return narrow ? launch_rows<64, 2, 4, 16, 3, 3>(d, dev, Z, s)
                      : warps == 8 ? launch_rows<128, 2, 8, 16, 2, 1>(d, dev, Z, s)
                                   : launch_rows<128, 2, 4, 16, 3, 2>(d, dev, Z, s);
    return narrow ? launch_rows<64, 1, 4, 16, 3, 4>(d, dev, Z, s)
                  : warps == 8 ? launch_rows<128, 1, 8, 16, 2, 1>(d, dev, Z, s)
                               : launch_rows<128, 1, 4, 16, 3, 2>(d, dev, Z, s);
}

}  // namespace vit
