// gemm_fp8.cu -- the 8-bit matrix product with a scale for each block of 128:
//   z[m, n] = sum_b sa[m, b] sw[n / 128, b] sum_{k in block b} a[m, k] w[n, k]   (+ bias[n])
//   out     = z,  GELU_tanh(z)  or  residual + z
// a (M, K) and w (N, K) are e4m3, sa (M, ceil(K / 128)) and sw (ceil(N / 128), ceil(K / 128))
// fp32. Products of e4m3 values are exact in fp32; a block's sum and the sum over blocks are
// fp32. An e4m3 output takes one scale for each 128 columns of a row (fp8.cuh).
//
// Pair kernel (many rows): a persistent CTA pair makes a 256 x BN tile with
// tcgen05.mma.cta_group::2 kind::f8f6f4. One ring stage is one block of 128 along K, both operands
// K-major with the 128-byte swizzle. A block's scales differ from row to row, so its sum cannot
// stay in one accumulator with the others': each block gets an accumulator of its own in TMEM
// (512 / BN, in turn), and the epilogue warps add scale * block sum to fp32 registers while the
// tensor cores make the next ones. With four in turn instead of two 577 x 5120 -> 5120 (BN 128) takes
// 34.1 us instead of 34.7. At BN 256 a block takes some 1160 cycles of which the products
// need 512 (36928 x 4096 -> 4096: 564 us, 2.20 PFLOP/s, near the power limit). No one part of it bounds that: without the
// additions 546 us, without the loads from TMEM too 473, with every tile's operands in L2 559 (BN 128: 803, 703, 684 and
// 798); what is left is the handing over between ring, products and sums, block by block. Measured and slower: loads of 64
// columns, 642 us; sixteen epilogue warps of 64 columns each with loads of 16, 780 us; products of 128 columns with
// accumulators handed over by halves, 573 us. The BN 128 instances spill 28 bytes a thread (100 read back).
//   warp 0       MMA issue (one lane of the leader CTA's)
//   warps 1-3    TMA: a stage is four boxes, A and B rows in halves, dealt out to the three warps in
//                turn (one thread's copies run one after another: with A's 16 KB on one warp the
//                stages came in at half the rate)
//   warps 4-11   promotion and epilogue: warp (quarter, half) keeps 32 rows x BN / 2 columns in
//                registers, one row per thread, so the row's scale is one register and an e4m3
//                output's 128-column scale needs no exchange (BN 256)
//
// Rows kernel (few rows): bound by the weight's bytes and by latency. The weight is the M side,
// out^T = w a^T: a CTA takes 128 weight rows (one scale block) against 16 or 32 rows of a, and a
// cluster of CTAs shares the blocks along K, so that a decoding step's product streams its weight
// with most of the SMs. The CTAs' fp32 sums meet in distributed shared memory and are added in
// rank order: no workspace, one launch, the same result every time. 8 x 1024 -> 4096 with GELU to
// e4m3 takes 5.0 us, 8 x 5120 -> 5120 7.4 (the pair kernel 7.2 and 20.2).
//
// Generic kernel: CUDA cores, any size and alignment; a CTA makes 16 rows x 128 columns (one
// output block per row), a thread eight columns of one row.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <mutex>

#include "common.cuh"
#include "fp8.cuh"
#include "kernels.h"
#include "launch.cuh"
#include "ptx.cuh"

namespace vit {
namespace {

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn f8_encode_fn() {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* q = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &q, 12000, cudaEnableDefault, &r) == cudaSuccess &&
            r == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(q);
    });
    return fn;
}

// Row-major (rows, cols) of `es`-byte elements; boxes of box_rows rows of 128 bytes, 128B swizzle.
bool f8_map(CUtensorMap* m, const void* base, CUtensorMapDataType dt, int es, int64_t rows, int64_t cols,
            uint32_t box_rows, CUtensorMapL2promotion l2) {
    EncodeTiledFn fn = f8_encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)(cols * es)};
    const cuuint32_t box[2] = {(cuuint32_t)(128 / es), box_rows};
    const cuuint32_t estr[2] = {1, 1};
    return fn(m, dt, 2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, l2, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

CUtensorMapDataType f8_map_type(int dt) {
    return dt == DT_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                        : dt == DT_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8;
}

__device__ __forceinline__ float load_f32(const void* p, bool f32, int64_t i) {
    return f32 ? static_cast<const float*>(p)[i] : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}

__device__ __forceinline__ void f8_error(uint32_t* err, uint32_t bit) {
    if (err) atomicOr(err, bit);
}

// ------------------------------------------------------------------------ pair kernel
constexpr int FP_THREADS = 384, FP_EPI_WARPS = 8, FP_TILE_M = 256;
constexpr int FP_A_BYTES = 128 * kFp8Block;      // this CTA's 128 rows of one block
constexpr int FP_STG = 32 * 128;                 // staging: 32 rows of 128 bytes per warp
constexpr int FP_REGS_IO = 56, FP_REGS_EPI = 224;   // of 168 x 3 warpgroups at launch

template <int BN> struct FpLayout {
    static constexpr int B_BYTES = BN / 2 * kFp8Block;
    static constexpr int STAGE = FP_A_BYTES + B_BYTES;
    static constexpr int STAGES = BN == 256 ? 5 : 6;
    static constexpr int NB = 512 / BN;                  // block sums in TMEM
    static constexpr int OFF_EPI = STAGES * STAGE;
    static constexpr int OFF_MAX = OFF_EPI + FP_EPI_WARPS * FP_STG;   // row maxima, BN 128 with e4m3
    static constexpr int OFF_BIAS = OFF_MAX + 2 * 2 * 128 * 4;        // per warp: its columns' bias
    static constexpr int OFF_BAR = OFF_BIAS + FP_EPI_WARPS * BN / 2 * 4;
    static constexpr int SMEM = OFF_BAR + 256 + 1024;
    static_assert(SMEM <= 227 * 1024, "shared memory");
};

struct FpParams {
    Fp8GemmDesc d;
    uint32_t* err;
    int out_tma;
};

// 32 sums of this thread's row from column `col` on, as 16 packed pairs: GELU or residual.
template <int EPI>
__device__ __forceinline__ void f8_finish32(const Fp8GemmDesc& d, int64_t row, int64_t col, unsigned long long (&v)[16]) {
    if constexpr (EPI == TC_EPI_GELU) {
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = gelu_tanh_exp2(v[j]);
    }
    if constexpr (EPI == TC_EPI_RESID) {
        if (row < d.M) {
            const int64_t at = row * d.N + col;
            const bool whole = col + 32 <= d.N;
            if (d.residual_f32) {
                const float* r = static_cast<const float*>(d.residual) + at;
                if (whole && (reinterpret_cast<uintptr_t>(r) & 15) == 0) {
#pragma unroll
                    for (int j = 0; j < 16; j += 2) {
                        const float4 u = *reinterpret_cast<const float4*>(r + 2 * j);
                        v[j] = f2_add(v[j], f2_pack(u.x, u.y));
                        v[j + 1] = f2_add(v[j + 1], f2_pack(u.z, u.w));
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        v[j] = f2_add(v[j], f2_pack(col + 2 * j < d.N ? r[2 * j] : 0.f, col + 2 * j + 1 < d.N ? r[2 * j + 1] : 0.f));
                }
            } else {
                const __nv_bfloat16* r = static_cast<const __nv_bfloat16*>(d.residual) + at;
                if (whole && (reinterpret_cast<uintptr_t>(r) & 15) == 0) {
#pragma unroll
                    for (int j = 0; j < 16; j += 4) {
                        const uint4 u = *reinterpret_cast<const uint4*>(r + 2 * j);
                        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            v[j + q] = f2_add(v[j + q], f2_pack(__uint_as_float(w[q] << 16), __uint_as_float(w[q] & 0xFFFF0000u)));
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        v[j] = f2_add(v[j], f2_pack(col + 2 * j < d.N ? __bfloat162float(r[2 * j]) : 0.f,
                                                    col + 2 * j + 1 < d.N ? __bfloat162float(r[2 * j + 1]) : 0.f));
                }
            }
        }
    }
}

// 16-byte unit u of staging row r, 128-byte rows with the 128-byte swizzle.
__device__ __forceinline__ uint4* f8_unit(uint8_t* stage, int r, int u) {
    return reinterpret_cast<uint4*>(stage + r * 128 + ((u ^ (r & 7)) << 4));
}

template <int BN, int EPI, int OUT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(FP_THREADS, 1)
gemm_fp8_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                     const __grid_constant__ CUtensorMap tmOut, const __grid_constant__ FpParams p) {
    using L = FpLayout<BN>;
    constexpr int STAGES = L::STAGES, NB = L::NB, COLS = BN / 2;   // columns per epilogue warp
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);
    uint64_t* empty = full + STAGES;
    uint64_t* tfull = empty + STAGES;
    uint64_t* tempty = tfull + NB;
    uint64_t* done = tempty + NB;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const Fp8GemmDesc& d = p.d;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = ptx::cluster_ctarank();
    const int cluster = blockIdx.x >> 1, nclusters = gridDim.x >> 1;
    const int n_tiles = (int)((d.N + BN - 1) / BN);
    const int tiles = (int)((d.M + FP_TILE_M - 1) / FP_TILE_M) * n_tiles;
    const int kblocks = (int)((d.K + kFp8Block - 1) / kFp8Block);

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            ptx::mbar_init(full + s, 1);
            ptx::mbar_init(empty + s, 1);
        }
        for (int a = 0; a < NB; ++a) {
            ptx::mbar_init(tfull + a, 1);
            ptx::mbar_init(tempty + a, 2 * FP_EPI_WARPS);
        }
        ptx::mbar_init(done, 1);
        *abort_flag = 0;
        ptx::fence_mbar_init();
    }
    if (warp == 1 && lane == 0) {
        ptx::prefetch_tensormap(&tmA);
        ptx::prefetch_tensormap(&tmB);
        if (p.out_tma) ptx::prefetch_tensormap(&tmOut);
    }
    if (warp == 0) {
        ptx::tmem_alloc_pair(tmem_slot, 512);
        ptx::tmem_relinquish_pair();
    }
    ptx::tc_fence_before();
    ptx::cluster_sync();   // barriers of both CTAs initialised before any remote arrive
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    griddep_wait();
    griddep_launch_dependents();

    if (warp < 4) {
        ptx::setmaxnreg_dec<FP_REGS_IO>();
        if (warp > 0 && lane == 0) {
            // ------------------------------------------------ TMA producers (both CTAs)
            const uint32_t full0 = ptx::mapa_shared(ptx::smem_addr(full), 0);   // the leader's
            uint32_t it = 0;
            bool ok = true;
            for (int t = cluster; t < tiles && ok; t += nclusters) {
                const int m0 = (t / n_tiles) * FP_TILE_M + (int)rank * 128;
                const int n0 = (t % n_tiles) * BN + (int)rank * (BN / 2);
                for (int kb = 0; kb < kblocks; ++kb, ++it) {
                    const uint32_t s = it % STAGES, u = it / STAGES;
                    if (!ptx::mbar_wait_bounded<true>(empty + s, (u & 1) ^ 1, abort_flag)) { ok = false; break; }
                    if (warp == 1 && rank == 0) ptx::mbar_arrive_expect_tx(full + s, 2 * L::STAGE);
                    uint8_t* st = smem + s * L::STAGE;
#pragma unroll
                    for (int x = 0; x < 4; ++x) {   // A rows 0-63, 64-127, then B's halves
                        if ((it * 4 + x) % 3 != (uint32_t)(warp - 1)) continue;
                        if (x < 2)
                            ptx::tma_load_2d_pair(st + x * (FP_A_BYTES / 2), &tmA, full0 + s * 8, kb * kFp8Block, m0 + x * 64);
                        else
                            ptx::tma_load_2d_pair(st + FP_A_BYTES + (x - 2) * (L::B_BYTES / 2), &tmB, full0 + s * 8,
                                                  kb * kFp8Block, n0 + (x - 2) * (BN / 4));
                    }
                }
            }
            if (!ok) {
                f8_error(p.err, ERRBIT_TIMEOUT_PRODUCER);
                *abort_flag = 1;
            }
            if (warp == 1 && rank == 0) {
                // the copies of both CTAs complete on these barriers: let them land
                for (uint32_t s = 0; s < (uint32_t)STAGES; ++s)
                    if (it > s && !ptx::mbar_wait_bounded(full + s, ((it - 1 - s) / STAGES) & 1, nullptr))
                        f8_error(p.err, ERRBIT_TIMEOUT_TEARDOWN);
            }
        } else if (warp == 0 && rank == 0) {
            // ------------------------------------------------ MMA issue (leader), one lane of a warp
            // that stays together (see elect_one): from lane 0 alone each issue took some 100 cycles
            constexpr uint32_t idesc = ptx::idesc_e4m3_f32(FP_TILE_M, BN);
            const uint64_t a0 = ptx::smem_desc_sw128(ptx::smem_addr(smem), 16, 1024);
            const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
            uint32_t it = 0, s = 0, round = 0;
            bool ok = true;
            for (int t = cluster; t < tiles && ok; t += nclusters) {
                for (int kb = 0; kb < kblocks; ++kb, ++it) {
                    const uint32_t acc = it % NB;
                    ok = ptx::mbar_wait_bounded(tempty + acc, ((it / NB) & 1) ^ 1, abort_flag) &&
                         ptx::mbar_wait_bounded(full + s, round & 1, abort_flag);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    ptx::tc_fence_after();
                    // descriptors count 16-byte units
                    const uint64_t ad = a0 + s * (L::STAGE >> 4), bd = ad + (FP_A_BYTES >> 4);
                    if (ptx::elect_one()) {
#pragma unroll
                        for (int k = 0; k < kFp8Block / 32; ++k)
                            ptx::mma_f8_ss_pair(tm + acc * BN, ad + k * 2, bd + k * 2, idesc, k != 0);
                        ptx::mma_commit_pair_mc(empty + s, 0x3);
                        ptx::mma_commit_pair_mc(tfull + acc, 0x3);
                    }
                    __syncwarp();
                    if (++s == (uint32_t)STAGES) {
                        s = 0;
                        ++round;
                    }
                }
            }
            if (ptx::elect_one()) {
                if (!ok) {
                    f8_error(p.err, ERRBIT_TIMEOUT_MMA);
                    *abort_flag = 1;
                }
                ptx::mma_commit_pair(done);
                if (!ptx::mbar_wait_bounded(done, 0, nullptr)) f8_error(p.err, ERRBIT_TIMEOUT_TEARDOWN);
            }
        }
    } else {
        // ------------------------------------------------ promotion and epilogue
        ptx::setmaxnreg_inc<FP_REGS_EPI>();
        const int quarter = warp & 3, half = (warp - 4) >> 2;
        const uint32_t tempty0 = ptx::mapa_shared(ptx::smem_addr(tempty), 0);
        const uint32_t t_lane = tmem + half * COLS + ((uint32_t)(quarter * 32) << 16);
        uint8_t* stage = smem + L::OFF_EPI + (warp - 4) * FP_STG;
        const int64_t nblk = (d.N + kFp8Block - 1) / kFp8Block;
        uint32_t it = 0, tcount = 0;   // block sums, tiles so far
        bool failed = false;   // a wait ran out: go on without waiting, store nothing
        // scales of block kb of tile t for this thread's row and this warp's columns
        auto scale_of = [&](int t, int kb) -> float {
            if (t >= tiles || kb >= kblocks) return 0.f;
            const int64_t row = (int64_t)(t / n_tiles) * FP_TILE_M + rank * 128 + quarter * 32 + lane;
            int64_t nb = ((int64_t)(t % n_tiles) * BN + half * COLS) / kFp8Block;
            if (nb > nblk - 1) nb = nblk - 1;
            const float sa = row < d.M ? __ldg(d.a_scales + row * kblocks + kb) : 0.f;
            return sa * __ldg(d.w_scales + nb * kblocks + kb);
        };
        float s0 = scale_of(cluster, 0), s1 = scale_of(cluster, 1);
        float bl[COLS / 32];
        auto load_bias = [&](int t) {
            if (!d.bias || t >= tiles) return;
#pragma unroll
            for (int j = 0; j < COLS / 32; ++j) {
                const int64_t c = (int64_t)(t % n_tiles) * BN + half * COLS + lane * (COLS / 32) + j;
                bl[j] = c < d.N ? load_f32(d.bias, d.bias_f32, c) : 0.f;
            }
        };
        load_bias(cluster);
        for (int t = cluster; t < tiles; t += nclusters, ++tcount) {
            const int64_t row0 = (int64_t)(t / n_tiles) * FP_TILE_M + rank * 128 + quarter * 32, row = row0 + lane;
            const int64_t n0 = (int64_t)(t % n_tiles) * BN + half * COLS;
            // sums start from the bias, COLS / 32 columns per lane, which arrived during the last tile
            unsigned long long acc[COLS / 2];
            if (d.bias) {
                float* sb = reinterpret_cast<float*>(smem + L::OFF_BIAS) + (warp - 4) * COLS;
                __syncwarp();   // the previous tile's have been read
#pragma unroll
                for (int j = 0; j < COLS / 32; ++j) sb[lane * (COLS / 32) + j] = bl[j];
                __syncwarp();
#pragma unroll
                for (int j = 0; j < COLS / 4; ++j) {
                    const float4 b = *reinterpret_cast<const float4*>(sb + 4 * j);
                    acc[2 * j] = f2_pack(b.x, b.y);
                    acc[2 * j + 1] = f2_pack(b.z, b.w);
                }
            } else {
#pragma unroll
                for (int j = 0; j < COLS / 2; ++j) acc[j] = 0ull;
            }
            // 32 columns at a time; the next 32 (of this block sum or of the next) are on their way
            // from TMEM while these are added
            constexpr int CH = COLS / 32;
            uint32_t ra[32], rb[32];
            auto ready = [&]() {   // the next block's sum is complete
                if (!failed && !__all_sync(0xffffffffu, ptx::mbar_wait_bounded(tfull + it % NB, (it / NB) & 1, abort_flag))) {
                    failed = true;
                    if (lane == 0) f8_error(p.err, ERRBIT_TIMEOUT_EPILOGUE);
                    *abort_flag = 1;
                }
                ptx::tc_fence_after();
            };
            auto add = [&](int c, const uint32_t (&r)[32], unsigned long long ss) {
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    acc[c * 16 + j] = f2_fma(f2_pack(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1])), ss,
                                             acc[c * 16 + j]);
            };
            ready();
            ptx::tmem_ld_32x32b_x32(t_lane + it % NB * BN, ra);
            for (int kb = 0; kb < kblocks; ++kb) {
                const float s2 = scale_of(t, kb + 2);   // two blocks ahead
                const unsigned long long ss = f2_pack(s0, s0);
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    uint32_t(&cur)[32] = (c & 1) ? rb : ra;
                    uint32_t(&nxt)[32] = (c & 1) ? ra : rb;
                    ptx::tmem_ld_wait_for(cur);
                    if (c + 1 < CH) {
                        ptx::tmem_ld_32x32b_x32(t_lane + it % NB * BN + (c + 1) * 32, nxt);
                    } else {
                        // this sum is in registers: its accumulator is free
                        ptx::tc_fence_before();
                        __syncwarp();
                        if (lane == 0) ptx::mbar_arrive_cluster_relaxed(tempty0 + it % NB * 8);   // orders TMEM reads only
                        ++it;
                        if (kb + 1 < kblocks) {
                            ready();
                            ptx::tmem_ld_32x32b_x32(t_lane + it % NB * BN, nxt);
                        }
                    }
                    add(c, cur, ss);
                }
                s0 = s1;
                s1 = s2;
            }
            // the next tile's first scales and bias travel while this one is stored
            s0 = scale_of(t + nclusters, 0);
            s1 = scale_of(t + nclusters, 1);
            load_bias(t + nclusters);
            if (n0 >= d.N && !(OUT == DT_E4M3 && BN == 128)) continue;   // (there the two halves meet below)
            if constexpr (OUT == DT_E4M3) {
                float amax = 0.f;
#pragma unroll
                for (int c = 0; c < COLS / 32; ++c) {
                    unsigned long long(&v)[16] = *reinterpret_cast<unsigned long long(*)[16]>(&acc[c * 16]);
                    f8_finish32<EPI>(d, row, n0 + c * 32, v);
                    // columns past N are products with zero rows: 0 (or NaN, which fmaxf drops)
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        float a, b;
                        f2_unpack(v[j], a, b);
                        amax = fmaxf(amax, fmaxf(fabsf(a), fabsf(b)));
                    }
                }
                if constexpr (BN == 128) {   // a block of 128 columns is two warps' halves
                    float* mx = reinterpret_cast<float*>(smem + L::OFF_MAX) + (tcount & 1) * 256;
                    mx[half * 128 + quarter * 32 + lane] = amax;
                    ptx::named_bar_sync(1 + quarter, 64);
                    amax = fmaxf(amax, mx[(half ^ 1) * 128 + quarter * 32 + lane]);
                }
                const float sc = fp8_block_scale(amax), inv = fp8_inverse(sc);
                const unsigned long long inv2 = f2_pack(inv, inv);
                if (row < d.M && n0 < d.N && (BN == 256 || half == 0) && !failed)
                    d.out_scales[row * nblk + n0 / kFp8Block] = sc;
                if (p.out_tma) {
                    if (lane == 0) ptx::bulk_wait_group_read<0>();
                    __syncwarp();
                }
#pragma unroll
                for (int u = 0; u < COLS / 16; ++u) {
                    uint32_t w[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        float a, b, c, e;
                        f2_unpack(f2_mul(acc[u * 8 + q * 2], inv2), a, b);
                        f2_unpack(f2_mul(acc[u * 8 + q * 2 + 1], inv2), c, e);
                        w[q] = fp8_pack4(a, b, c, e);
                    }
                    if (p.out_tma) {
                        if constexpr (BN == 256) *f8_unit(stage, lane, u) = make_uint4(w[0], w[1], w[2], w[3]);
                        else   // rows of 64 bytes, 64-byte swizzle
                            *reinterpret_cast<uint4*>(stage + lane * 64 + ((u ^ ((lane >> 1) & 3)) << 4)) =
                                make_uint4(w[0], w[1], w[2], w[3]);
                    } else if (row < d.M && !failed) {
                        uint8_t* o = static_cast<uint8_t*>(d.out) + row * d.N + n0 + u * 16;
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            if (n0 + u * 16 + j < d.N) o[j] = (uint8_t)(w[j >> 2] >> ((j & 3) * 8));
                    }
                }
                if (p.out_tma) {
                    ptx::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0 && !failed && n0 < d.N) {
                        ptx::tma_store_2d(&tmOut, stage, (int32_t)n0, (int32_t)row0);
                        ptx::bulk_commit_group();
                    }
                }
            } else {
                // 128 bytes of each row at a time: 32 fp32 or 64 bf16 columns
                constexpr int UNIT = OUT == DT_F32 ? 32 : 64;
#pragma unroll
                for (int c = 0; c < COLS / 32; ++c) {
                    const int64_t col = n0 + c * 32;
                    f8_finish32<EPI>(d, row, col, *reinterpret_cast<unsigned long long(*)[16]>(&acc[c * 16]));
                    float v[32];
#pragma unroll
                    for (int j = 0; j < 16; ++j) f2_unpack(acc[c * 16 + j], v[2 * j], v[2 * j + 1]);
                    if (p.out_tma) {
                        if ((c * 32) % UNIT == 0) {
                            if (lane == 0) ptx::bulk_wait_group_read<0>();
                            __syncwarp();
                        }
                        if constexpr (OUT == DT_F32) {
#pragma unroll
                            for (int u = 0; u < 8; ++u)
                                *f8_unit(stage, lane, u) =
                                    make_uint4(__float_as_uint(v[4 * u]), __float_as_uint(v[4 * u + 1]),
                                               __float_as_uint(v[4 * u + 2]), __float_as_uint(v[4 * u + 3]));
                        } else {
#pragma unroll
                            for (int u = 0; u < 4; ++u)
                                *f8_unit(stage, lane, (c & 1) * 4 + u) =
                                    make_uint4(pack_bf16x2(v[8 * u], v[8 * u + 1]), pack_bf16x2(v[8 * u + 2], v[8 * u + 3]),
                                               pack_bf16x2(v[8 * u + 4], v[8 * u + 5]),
                                               pack_bf16x2(v[8 * u + 6], v[8 * u + 7]));
                        }
                        if ((c * 32 + 32) % UNIT == 0) {
                            ptx::fence_proxy_async_smem();
                            __syncwarp();
                            const int64_t first = n0 + c * 32 + 32 - UNIT;
                            if (lane == 0 && !failed && first < d.N) {
                                ptx::tma_store_2d(&tmOut, stage, (int32_t)first, (int32_t)row0);
                                ptx::bulk_commit_group();
                            }
                        }
                    } else if (row < d.M && !failed) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            if (col + j >= d.N) continue;
                            if constexpr (OUT == DT_F32) static_cast<float*>(d.out)[row * d.N + col + j] = v[j];
                            else static_cast<__nv_bfloat16*>(d.out)[row * d.N + col + j] = __float2bfloat16_rn(v[j]);
                        }
                    }
                }
            }
        }
        if (lane == 0) ptx::bulk_wait_group<0>();   // stores complete before the CTA exits
    }

    __syncthreads();
    ptx::cluster_sync();   // no CTA leaves while its peer may still touch its memory
    if (warp == 0) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc_pair(tmem, 512);
    }
}

// A row stride that TMA takes, from a 16-byte aligned base.
inline bool f8_tma_ok(const void* p, int64_t row_bytes) {
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && row_bytes % 16 == 0;
}

template <int BN, int EPI, int OUT>
cudaError_t launch_pair_inst(const Fp8GemmDesc& d, const DeviceInfo& dev, cudaStream_t s) {
    using L = FpLayout<BN>;
    auto k = gemm_fp8_pair_kernel<BN, EPI, OUT>;
    // setmaxnreg hands out the registers of the launch: the split must fit in them
    static const bool fits = [&] {
        cudaFuncAttributes a;
        return cudaFuncGetAttributes(&a, k) == cudaSuccess &&
               a.numRegs * 3 >= FP_REGS_IO + 2 * FP_REGS_EPI;
    }();
    if (!fits) return cudaErrorNotSupported;
    static std::atomic<uint64_t> attr{0};
    cudaError_t e = set_smem_limit_once(k, L::SMEM, attr);
    if (e != cudaSuccess) return e;
    alignas(64) CUtensorMap ma, mb, mo;
    if (!f8_map(&ma, d.a, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, d.M, d.K, 64, CU_TENSOR_MAP_L2_PROMOTION_L2_256B) ||
        !f8_map(&mb, d.w, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, d.N, d.K, BN / 4, CU_TENSOR_MAP_L2_PROMOTION_L2_256B))
        return cudaErrorInvalidValue;
    FpParams p{d, dev.err_word, 0};
    const int es = (int)dt_size(OUT);
    mo = ma;
    if (f8_tma_ok(d.out, d.N * es)) {
        p.out_tma = 1;
        if (OUT == DT_E4M3 && BN == 128) {
            const cuuint64_t dims[2] = {(cuuint64_t)d.N, (cuuint64_t)d.M};
            const cuuint64_t strides[1] = {(cuuint64_t)d.N};
            const cuuint32_t box[2] = {64, 32}, estr[2] = {1, 1};
            if (f8_encode_fn()(&mo, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, d.out, dims, strides, box, estr,
                               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
                return cudaErrorInvalidValue;
        } else if (!f8_map(&mo, d.out, f8_map_type(OUT), es, d.M, d.N, 32, CU_TENSOR_MAP_L2_PROMOTION_NONE)) {
            return cudaErrorInvalidValue;
        }
    }
    const int64_t tiles = ((d.M + FP_TILE_M - 1) / FP_TILE_M) * ((d.N + BN - 1) / BN);
    const int64_t clusters = tiles < dev.num_sms / 2 ? tiles : dev.num_sms / 2;
    return launch_dependent(k, dim3((unsigned)(2 * clusters)), dim3(FP_THREADS), L::SMEM, s, ma, mb, mo, p);
}

template <int BN, int EPI>
cudaError_t launch_pair_out(const Fp8GemmDesc& d, const DeviceInfo& dev, cudaStream_t s) {
    switch (d.out_dt) {
        case DT_BF16: return launch_pair_inst<BN, EPI, DT_BF16>(d, dev, s);
        case DT_F32: return launch_pair_inst<BN, EPI, DT_F32>(d, dev, s);
        case DT_E4M3: return launch_pair_inst<BN, EPI, DT_E4M3>(d, dev, s);
    }
    return cudaErrorInvalidValue;
}

template <int BN> cudaError_t launch_pair(const Fp8GemmDesc& d, const DeviceInfo& dev, cudaStream_t s) {
    switch (d.epi) {
        case TC_EPI_STORE: return launch_pair_out<BN, TC_EPI_STORE>(d, dev, s);
        case TC_EPI_GELU: return launch_pair_out<BN, TC_EPI_GELU>(d, dev, s);
        case TC_EPI_RESID: return launch_pair_out<BN, TC_EPI_RESID>(d, dev, s);
    }
    return cudaErrorInvalidValue;
}

// Tensor-core kernels: 16-byte aligned operands and rows, extents and tile counts in 32 bits.
bool f8_tc_ok(const Fp8GemmDesc& d, const DeviceInfo& dev) {
    const int64_t lim = 0x7fffffff - 512;
    return f8_tma_ok(d.a, d.K) && f8_tma_ok(d.w, d.K) && d.M <= lim && d.N <= lim && d.K <= lim &&
           ((d.M + 255) / 256) * ((d.N + 127) / 128) <= lim && dev.num_sms >= 2 && f8_encode_fn() != nullptr;
}

// ------------------------------------------------------------------------ rows kernel
constexpr int FR_THREADS = 224;   // warp 0: weight loads, 1: MMA, 2-5: sums and epilogue, 6: loads of a
constexpr int FR_BUFS = 4;        // block sums in TMEM
constexpr int FR_MAXZ = 8;

template <int TN> struct FrLayout {
    static constexpr int W_BYTES = 128 * kFp8Block;
    static constexpr int STAGE = W_BYTES + TN * kFp8Block;
    static constexpr int STAGES = 5;   // two CTAs fit an SM
    static constexpr int OFF_SC = STAGES * STAGE;                    // per warp: two sets of TN scales
    static constexpr int OFF_MAX = OFF_SC + 4 * 2 * TN * 4;          // per token: four warps' maxima
    static constexpr int OFF_BAR = OFF_MAX + 4 * TN * 4;
    static constexpr int SMEM = OFF_BAR + 512 + 1024;
    static_assert(TN * 128 * 4 <= STAGES * STAGE, "sums over the ring");
    static_assert(SMEM <= 227 * 1024, "shared memory");
};

template <int TN, int EPI, int OUT>
__global__ void __launch_bounds__(FR_THREADS, 1)
gemm_fp8_rows_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmA,
                     const __grid_constant__ FpParams p, int Z, int mtiles) {
    using L = FrLayout<TN>;
    constexpr int STAGES = L::STAGES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);
    uint64_t* empty = full + STAGES;
    uint64_t* tfull = empty + STAGES;
    uint64_t* tempty = tfull + FR_BUFS;
    uint64_t* done = tempty + FR_BUFS;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const Fp8GemmDesc& d = p.d;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int z = Z > 1 ? (int)ptx::cluster_ctarank() : 0, tile = blockIdx.x / Z;
    const int nt = tile / mtiles, mt = tile - nt * mtiles;
    const int kblocks = (int)((d.K + kFp8Block - 1) / kFp8Block);
    // this CTA's share of the blocks
    const int per = (kblocks + Z - 1) / Z, kb0 = min(z * per, kblocks), nkb = min(kb0 + per, kblocks) - kb0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            ptx::mbar_init(full + s, 2);
            ptx::mbar_init(empty + s, 1);
        }
        for (int b = 0; b < FR_BUFS; ++b) {
            ptx::mbar_init(tfull + b, 1);
            ptx::mbar_init(tempty + b, 4);
        }
        ptx::mbar_init(done, 1);
        *abort_flag = 0;
        ptx::fence_mbar_init();
        ptx::prefetch_tensormap(&tmW);
        ptx::prefetch_tensormap(&tmA);
    }
    if (warp == 1) {
        ptx::tmem_alloc(tmem_slot, FR_BUFS * TN);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
    griddep_wait();
    griddep_launch_dependents();

    bool failed = false;
    float acc[TN];
    if (warp == 0 || warp == 6) {
        if (lane == 0) {
            bool ok = true;
            int i = 0;
            for (; i < nkb; ++i) {
                const int s = i % STAGES;
                if (!ptx::mbar_wait_bounded<true>(empty + s, ((i / STAGES) & 1) ^ 1, abort_flag)) { ok = false; break; }
                uint8_t* st = smem + s * L::STAGE;
                if (warp == 0) {
                    ptx::mbar_arrive_expect_tx(full + s, L::W_BYTES);
                    ptx::tma_load_2d(st, &tmW, full + s, (kb0 + i) * kFp8Block, nt * 128);
                } else {
                    ptx::mbar_arrive_expect_tx(full + s, TN * kFp8Block);
                    ptx::tma_load_2d(st + L::W_BYTES, &tmA, full + s, (kb0 + i) * kFp8Block, mt * TN);
                }
            }
            if (!ok) {
                f8_error(p.err, ERRBIT_TIMEOUT_PRODUCER);
                *abort_flag = 1;
                // copies in flight land before the CTA can exit
                for (int j = i > STAGES ? i - STAGES : 0; j < i; ++j)
                    if (!ptx::mbar_wait_bounded(full + j % STAGES, (j / STAGES) & 1, nullptr))
                        f8_error(p.err, ERRBIT_TIMEOUT_TEARDOWN);
            }
        }
    } else if (warp == 1) {
        constexpr uint32_t idesc = ptx::idesc_e4m3_f32(128, TN);
        const uint64_t w0 = ptx::smem_desc_sw128(ptx::smem_addr(smem), 16, 1024);
        bool ok = true;
        for (int i = 0; i < nkb; ++i) {
            const uint32_t s = i % STAGES, buf = i % FR_BUFS;
            ok = ptx::mbar_wait_bounded(tempty + buf, ((i / FR_BUFS) & 1) ^ 1, abort_flag) &&
                 ptx::mbar_wait_bounded(full + s, (i / STAGES) & 1, abort_flag);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            ptx::tc_fence_after();
            const uint64_t wd = w0 + s * (L::STAGE >> 4), ad = wd + (L::W_BYTES >> 4);
            if (ptx::elect_one()) {
#pragma unroll
                for (int k = 0; k < kFp8Block / 32; ++k)
                    ptx::mma_f8_ss(tmem + buf * TN, wd + k * 2, ad + k * 2, idesc, k != 0);
                ptx::mma_commit(empty + s);
                ptx::mma_commit(tfull + buf);
            }
            __syncwarp();
        }
        if (ptx::elect_one()) {
            if (!ok) {
                f8_error(p.err, ERRBIT_TIMEOUT_MMA);
                *abort_flag = 1;
            }
            ptx::mma_commit(done);
            if (!ptx::mbar_wait_bounded(done, 0, nullptr)) f8_error(p.err, ERRBIT_TIMEOUT_TEARDOWN);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------ sums: a weight row per thread, TN tokens
        const int quarter = warp & 3;
        const uint32_t t_lane = tmem + ((uint32_t)(quarter * 32) << 16);
        float* sc = reinterpret_cast<float*>(smem + L::OFF_SC) + quarter * 2 * TN;
        constexpr int PER = (TN + 31) / 32;
        // products of a block's scales for this lane's tokens
        auto scales = [&](int i, float (&v)[PER]) {
            const float w = i < nkb ? __ldg(d.w_scales + (int64_t)nt * kblocks + kb0 + i) : 0.f;
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                const int64_t m = (int64_t)mt * TN + j * 32 + lane;
                v[j] = i < nkb && j * 32 + lane < TN && m < d.M ? w * __ldg(d.a_scales + m * kblocks + kb0 + i) : 0.f;
            }
        };
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[j] = 0.f;
        float v0[PER], v1[PER];
        scales(0, v0);
        scales(1, v1);
        for (int i = 0; i < nkb; ++i) {
            const uint32_t buf = i % FR_BUFS;
            float* set = sc + (i & 1) * TN;
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                if (j * 32 + lane < TN) set[j * 32 + lane] = v0[j];
                v0[j] = v1[j];
            }
            scales(i + 2, v1);
            __syncwarp();   // two sets in turn: nobody is still reading the one that is written next
            if (!failed && !__all_sync(0xffffffffu, ptx::mbar_wait_bounded(tfull + buf, (i / FR_BUFS) & 1, abort_flag))) {
                failed = true;
                if (lane == 0) f8_error(p.err, ERRBIT_TIMEOUT_EPILOGUE);
                *abort_flag = 1;
            }
            ptx::tc_fence_after();
#pragma unroll
            for (int c = 0; c < TN / 16; ++c) {
                uint32_t r[16];
                ptx::tmem_ld_32x32b_x16(t_lane + buf * TN + c * 16, r);
                ptx::tmem_ld_wait_for(r);
#pragma unroll
                for (int j = 0; j < 16; j += 4) {
                    const float4 f = *reinterpret_cast<const float4*>(set + c * 16 + j);
                    acc[c * 16 + j] = fmaf(f.x, __uint_as_float(r[j]), acc[c * 16 + j]);
                    acc[c * 16 + j + 1] = fmaf(f.y, __uint_as_float(r[j + 1]), acc[c * 16 + j + 1]);
                    acc[c * 16 + j + 2] = fmaf(f.z, __uint_as_float(r[j + 2]), acc[c * 16 + j + 2]);
                    acc[c * 16 + j + 3] = fmaf(f.w, __uint_as_float(r[j + 3]), acc[c * 16 + j + 3]);
                }
            }
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(tempty + buf);
        }
    }
    // ---------------------------------------------------- the CTAs' sums over the ring, [token][weight row]
    float* part = reinterpret_cast<float*>(smem);
    __syncthreads();   // every block of this CTA has been multiplied and added
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, FR_BUFS * TN);
    }
    const bool sums = warp >= 2 && warp <= 5;
    const int n = (warp & 3) * 32 + lane;
    if (sums && Z > 1) {
#pragma unroll
        for (int j = 0; j < TN; ++j) part[j * 128 + n] = acc[j];
    }
    if (Z > 1) ptx::cluster_sync();
    if (sums) {
        const int64_t col = (int64_t)nt * 128 + n, nblk = (d.N + kFp8Block - 1) / kFp8Block;
        const float bias = d.bias && col < d.N ? load_f32(d.bias, d.bias_f32, col) : 0.f;
        float* mx = reinterpret_cast<float*>(smem + L::OFF_MAX);
        // this CTA's tokens: all of them, or its share of the cluster's
        const int share = (TN + Z - 1) / Z, j0 = z * share, j1 = min(j0 + share, TN);
        auto finish = [&](int j, float v) -> float {
            const int64_t m = (int64_t)mt * TN + j;
            v += bias;
            if constexpr (EPI == TC_EPI_GELU) v = gelu_tanh_exp1(v);
            if constexpr (EPI == TC_EPI_RESID)
                if (m < d.M && col < d.N) v += load_f32(d.residual, d.residual_f32, m * d.N + col);
            return v;
        };
        auto store = [&](int j, float v) {
            const int64_t m = (int64_t)mt * TN + j;
            if (m >= d.M || col >= d.N || failed) return;
            if constexpr (OUT == DT_F32) static_cast<float*>(d.out)[m * d.N + col] = v;
            else if constexpr (OUT == DT_BF16) static_cast<__nv_bfloat16*>(d.out)[m * d.N + col] = __float2bfloat16_rn(v);
            else static_cast<uint8_t*>(d.out)[m * d.N + col] = fp8_pack1(v);
        };
        if (Z == 1) {
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                acc[j] = finish(j, acc[j]);
                if constexpr (OUT == DT_E4M3) {
                    const float w = warp_max(fabsf(acc[j]));
                    if (lane == 0) mx[(warp & 3) * TN + j] = w;
                } else {
                    store(j, acc[j]);
                }
            }
            if constexpr (OUT == DT_E4M3) {
                ptx::named_bar_sync(1, 128);
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    const float s = fp8_block_scale(fmaxf(fmaxf(mx[j], mx[TN + j]), fmaxf(mx[2 * TN + j], mx[3 * TN + j])));
                    const int64_t m = (int64_t)mt * TN + j;
                    if (n == 0 && m < d.M && !failed) d.out_scales[m * nblk + nt] = s;
                    store(j, acc[j] * fp8_inverse(s));
                }
            }
        } else {
            // the cluster's sums in rank order, four tokens' values asked for at once
            uint32_t at[FR_MAXZ];
#pragma unroll
            for (int y = 0; y < FR_MAXZ; ++y) at[y] = ptx::mapa_shared(ptx::smem_addr(part + n), y < Z ? y : 0);
            for (int j4 = j0; j4 < j1; j4 += 4) {
                float v[4][FR_MAXZ];
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int y = 0; y < FR_MAXZ; ++y)
                        v[e][y] = y < Z && j4 + e < j1 ? ptx::ld_cluster_f32(at[y] + (j4 + e) * 512) : 0.f;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int j = j4 + e;
                    if (j >= j1) break;
                    float t = 0.f;
#pragma unroll
                    for (int y = 0; y < FR_MAXZ; ++y)
                        if (y < Z) t += v[e][y];
                    t = finish(j, t);
                    if constexpr (OUT == DT_E4M3) {
                        part[j * 128 + n] = t;   // of this CTA's sums of this token, only this thread read [n]
                        const float w = warp_max(fabsf(t));
                        if (lane == 0) mx[(warp & 3) * TN + j] = w;
                    } else {
                        store(j, t);
                    }
                }
            }
            if constexpr (OUT == DT_E4M3) {
                ptx::named_bar_sync(1, 128);
                for (int j = j0; j < j1; ++j) {
                    const float s = fp8_block_scale(fmaxf(fmaxf(mx[j], mx[TN + j]), fmaxf(mx[2 * TN + j], mx[3 * TN + j])));
                    const int64_t m = (int64_t)mt * TN + j;
                    if (n == 0 && m < d.M && !failed) d.out_scales[m * nblk + nt] = s;
                    store(j, part[j * 128 + n] * fp8_inverse(s));
                }
            }
        }
    }
    __syncwarp();
    if (Z > 1) ptx::cluster_sync();   // no CTA leaves while another reads its sums
}

template <int TN, int EPI, int OUT>
cudaError_t launch_rows_inst(const Fp8GemmDesc& d, const DeviceInfo& dev, int Z, cudaStream_t s) {
    using L = FrLayout<TN>;
    auto k = gemm_fp8_rows_kernel<TN, EPI, OUT>;
    static std::atomic<uint64_t> attr{0};
    const cudaError_t e = set_smem_limit_once(k, L::SMEM, attr);
    if (e != cudaSuccess) return e;
    alignas(64) CUtensorMap mw, ma;
    if (!f8_map(&mw, d.w, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, d.N, d.K, 128, CU_TENSOR_MAP_L2_PROMOTION_L2_256B) ||
        !f8_map(&ma, d.a, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, d.M, d.K, TN, CU_TENSOR_MAP_L2_PROMOTION_L2_256B))
        return cudaErrorInvalidValue;
    const FpParams p{d, dev.err_word, 0};
    const int mtiles = (int)((d.M + TN - 1) / TN);
    const int64_t tiles = mtiles * ((d.N + 127) / 128);
    if (Z == 1)
        return launch_dependent(k, dim3((unsigned)tiles), dim3(FR_THREADS), L::SMEM, s, mw, ma, p, 1, mtiles);
    return launch_dependent_cluster(k, dim3((unsigned)(tiles * Z)), dim3(FR_THREADS), Z, L::SMEM, s, mw, ma, p, Z, mtiles);
}

template <int TN, int EPI> cudaError_t launch_rows_out(const Fp8GemmDesc& d, const DeviceInfo& dev, int Z, cudaStream_t s) {
    switch (d.out_dt) {
        case DT_BF16: return launch_rows_inst<TN, EPI, DT_BF16>(d, dev, Z, s);
        case DT_F32: return launch_rows_inst<TN, EPI, DT_F32>(d, dev, Z, s);
        case DT_E4M3: return launch_rows_inst<TN, EPI, DT_E4M3>(d, dev, Z, s);
    }
    return cudaErrorInvalidValue;
}

template <int TN> cudaError_t launch_rows(const Fp8GemmDesc& d, const DeviceInfo& dev, cudaStream_t s) {
    // One block along K at least for each CTA; a second CTA on an SM only for eight or more (us with
    // one / two per SM: 8 x 5120 x 5120 9.7 / 7.4, 256 x 4096 x 1024 10.8 / 8.8, but 512 x 1024 x 1024,
    // four blocks each, 5.3 / 8.0).
    const int64_t tiles = ((d.M + TN - 1) / TN) * ((d.N + 127) / 128), kblocks = (d.K + kFp8Block - 1) / kFp8Block;
    int Z = 1;
    while (Z < FR_MAXZ && tiles * Z * 2 <= 2 * (int64_t)dev.num_sms &&
           kblocks >= Z * 2 * (tiles * Z * 2 <= dev.num_sms ? 1 : 8))
        Z *= 2;
    switch (d.epi) {
        case TC_EPI_STORE: return launch_rows_out<TN, TC_EPI_STORE>(d, dev, Z, s);
        case TC_EPI_GELU: return launch_rows_out<TN, TC_EPI_GELU>(d, dev, Z, s);
        case TC_EPI_RESID: return launch_rows_out<TN, TC_EPI_RESID>(d, dev, Z, s);
    }
    return cudaErrorInvalidValue;
}

// ------------------------------------------------------------------------ generic kernel
constexpr int GG_ROWS = 16, GG_COLS = 128, GG_THREADS = 256;

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
            if (d.out_dt == DT_E4M3) static_cast<uint8_t*>(d.out)[at] = fp8_pack1(acc[j] * fp8_inverse(sc));
            else if (d.out_dt == DT_F32) static_cast<float*>(d.out)[at] = acc[j];
            else static_cast<__nv_bfloat16*>(d.out)[at] = __float2bfloat16_rn(acc[j]);
        }
    }
}

}  // namespace

cudaError_t launch_gemm_fp8(const Fp8GemmDesc& d, const DeviceInfo& dev, cudaStream_t s) {
    if (f8_tc_ok(d, dev)) {
        // Up to 32 rows the rows kernel reads the weight once, with every SM. Beyond, 32 rows at a time,
        // while its tiles are one wave of CTAs: it then has more CTAs than the pair kernel has pairs
        // with work. Measured, rows / pair kernel, us (rows x K x N): 8 x 5120 x 5120 7.4 / 20.2;
        // 100 x 4096 x 1024 6.9 / 15.1; 512 x 1024 x 1024 5.3 / 6.5; and past one wave
        // 200 x 1024 x 4096 6.5 / 6.5; 1000 x 1280 x 1280 12.2 / 7.6.
        if (d.M <= 16) return launch_rows<16>(d, dev, s);
        if (d.M <= 32 || ((d.M + 31) / 32) * ((d.N + 127) / 128) <= dev.num_sms) return launch_rows<32>(d, dev, s);
        // A 256-wide tile takes 1.4 times a 128-wide one (0.55 to 0.60 us and 0.40 to 0.45 per block along K), so what
        // counts is in how many rounds the pairs get through them. Measured, 128 / 256 wide, us (rows x K x N):
        // 2308 x 4096 x 1024 27.1 / 20.7 (2 rounds / 1), 577 x 5120 x 5120 33.7 / 24.4 (2 / 1), 1154 x 4096 x 1024
        // 15.7 / 20.5 (1 / 1), 2308 x 1024 x 4096 20.6 / 18.1 (5 / 3), 9232 x 4096 x 1024 55.9 / 40.0 (4 / 2).
        const int64_t pairs = dev.num_sms / 2, high = (d.M + FP_TILE_M - 1) / FP_TILE_M;
        const int64_t wide = (high * ((d.N + 255) / 256) + pairs - 1) / pairs;
        const int64_t narrow = (high * ((d.N + 127) / 128) + pairs - 1) / pairs;
        return narrow * 5 <= wide * 7 ? launch_pair<128>(d, dev, s) : launch_pair<256>(d, dev, s);
    }
    int64_t grid = ((d.M + GG_ROWS - 1) / GG_ROWS) * ((d.N + GG_COLS - 1) / GG_COLS);
    if (grid > 8 * (int64_t)dev.num_sms) grid = 8 * (int64_t)dev.num_sms;
    return launch_dependent(gemm_fp8_generic_kernel, dim3((unsigned)grid), dim3(GG_THREADS), 0, s, d);
}

}  // namespace vit
