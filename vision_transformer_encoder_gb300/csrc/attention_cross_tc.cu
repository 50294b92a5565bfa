// attention_cross_tc.cu -- cross attention of many queries on the sm_103a tensor cores
// (tcgen05 / TMEM / TMA), bf16 in and out, fp32 softmax: the mathematics of
// attention_cross.cu for head widths 64, 80, 96 and 128.
//
// A tile is up to 128 query rows of ONE key head: TT tokens x the G query heads that share it
// (TT = 128 / G), packed row = token * G + head by one 4-D TMA box, so K and V are read once for
// the whole head group. A work item is (sequence, key head, pair of tiles); a persistent CTA per
// SM walks the items.
//   warps 10, 11  TMA: Q and K tiles, V tiles, 128 keys each, rings of their own
//   warps 1, 0    MMA issue for softmax group 0, 1, 64 keys (half a tile) at a time: S = Q K^T
//                 (M 128, N 64, K dh), then O += P V (M 128, N dh, K 64) with P read from TMEM and V
//                 MN-major
//   warps 2-5, 6-9  softmax groups 0 and 1, one query row per thread
// Each group has two S buffers of 64 columns in TMEM, and P overwrites the S that it came from: while
// the softmax works on one half tile, the scores of the next are there already and P V of the one
// before runs. (With 128 keys at a time S, P and O of both groups fill TMEM, so that the scores
// wait for P V and the softmax for the scores: a pair of tiles of 128 x 128 took 3960 cycles at dh 128
// where its products take 2048. P in columns of its own, which fit up to dh 96, with scores made as
// soon as the softmax holds the last ones, measured slower: 2 x 1024 queries over 8192 keys of 16
// heads of 64, 111 us instead of 97.) A half tile now takes 1440 cycles at dh 64 and 1725 at dh 128:
// some 960 in the softmax, half of them exponentials, the rest waiting for scores.
// Heads wider than 64 columns are two 64-column boxes; columns past dh are zero-filled on load and
// cut off on store by the tensor map, so 80 and 96 run as they are.
//
// The weights P are rounded to bf16 for the second product (their sum is not): one MMA has both operands in one type, and
// V is bf16. The outputs' error in the 2-norm becomes 2.3e-3 instead of the 1.7e-3 of rounding them alone.
//
// The running maximum is only raised when a row's scores exceed it by more than 8 (in log2): until
// then weights of up to 2^8 are carried, exactly as good in bf16 and far inside fp32, and the
// accumulator in TMEM is not touched. Keys past the sequence's length get weight 0 by position,
// and the V rows that the last tile holds past it are cleared before they meet those zeros.
//
// Few items over many keys (SPLIT): the CTAs of a cluster take a part of an item's key tiles each and
// join O, the maxima and the sums through distributed shared memory, every CTA a share of the rows.
// Every wait is bounded; on expiry the kernel records an error bit and unwinds.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "cross_maps.cuh"
#include "kernels.h"
#include "launch.cuh"
#include "ptx.cuh"

namespace vit {
namespace {

constexpr int CT_ROWS = 128, CT_KEYS = 128, CT_SUB = 64, CT_THREADS = 384;
constexpr int CT_BOX = CT_ROWS * 128;      // 64 columns x 128 rows: 16 KB
constexpr int CT_MAXZ = 8;
constexpr int CT_SORT = 128;               // sequences that are put in order of their lengths, at most
constexpr float CT_SLACK = 8.f;            // log2 of the weights that are carried before a rescale
// Weights are exp2(fma(s, scale, -m)): the product exact, m the rounded product of the largest score, so that the
// largest weight is 2 to the power of up to half of m's last place. From here on that may be more than 2, and past 2^31 it
// overflows: such rows round their products as m was rounded. (One vote with the rescaling, 0 to 1 % of the time.)
constexpr float CT_COARSE = 16777216.f;

template <int DH> struct CtLayout {
    static_assert(DH % 16 == 0 && DH >= 64 && DH <= 128, "head width");
    static constexpr int NCH = (DH + 63) / 64;           // 64-column boxes per tile
    static constexpr int TILE = NCH * CT_BOX;
    static constexpr int QBUF = NCH == 2 ? 1 : 2;        // buffers of two query tiles
    static constexpr int KVS = NCH == 2 ? 2 : 4;         // stages of each ring
    static constexpr int OFF_K = QBUF * 2 * TILE;
    static constexpr int OFF_V = OFF_K + KVS * TILE;
    static constexpr int OFF_O = OFF_V + KVS * TILE;     // per group: one 64-column box of O on its way out
    static constexpr int OFF_BAR = OFF_O + 2 * CT_BOX;
    static constexpr int OFF_LENS = OFF_BAR + 512;       // lengths while the sequences are put in order
    static constexpr int SMEM = OFF_LENS + CT_SORT * 4 + 1024;
    static_assert(SMEM <= 227 * 1024, "shared memory");
};

struct CtParams {
    const int32_t* kv_lens;
    int B, Tq, Tk, Hkv, G, TT;
    int npairs, items;
    int kb, kh, vb, vh, qb;      // 0 where the tensor has one sequence (key head) for all
    int Z;                       // CTAs per item (SPLIT)
    int sorted;                  // items by falling length
    int H;
    __nv_bfloat16* o;            // SPLIT: rows are stored directly
    float scale_log2;
    uint32_t* err;
};

struct CtBars {
    uint64_t q_full[2], q_empty[2];
    uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4];
    // two of each for the half tiles in turn: a waiter may be one phase behind, never two
    uint64_t s_full[2][2], p_full[2][2], o_done[2][2], o_free[2], ost_full[2], ost_free[2];
    uint64_t done;
    uint32_t tmem_slot;
    int abort_flag;
    uint8_t order[CT_SORT];      // sequences, the longest first
};
static_assert(sizeof(CtBars) <= 512, "barriers");

__device__ __forceinline__ void ct_error(uint32_t* err, uint32_t bit) {
    if (err) atomicOr(err, bit);
}

struct CtItem {
    int b, h, t0, nact, len;
    int nkt, nst;   // key tiles, half tiles
    int kt0;        // first key tile (SPLIT)
    bool any;       // the sequence has keys at all
};

template <bool SPLIT> __device__ __forceinline__ CtItem ct_item(const CtParams& p, int item, const uint8_t* order) {
    CtItem x;
    const int pair = item % p.npairs, bh = item / p.npairs;
    x.h = bh % p.Hkv;
    x.b = bh / p.Hkv;
    if (!SPLIT && p.sorted) x.b = order[x.b];
    x.t0 = pair * 2 * p.TT;
    x.nact = x.t0 + p.TT < p.Tq ? 2 : 1;
    x.len = p.kv_lens ? min(max(__ldg(p.kv_lens + x.b), 0), p.Tk) : p.Tk;
    x.any = x.len > 0;
    x.kt0 = 0;
    if (SPLIT) {   // this CTA's part of the tiles
        const int all = (x.len + CT_KEYS - 1) / CT_KEYS, per = (all + p.Z - 1) / p.Z;
        x.kt0 = min((int)ptx::cluster_ctarank() * per, all);
        x.len = min(x.len - x.kt0 * CT_KEYS, per * CT_KEYS);
    }
    x.nkt = (x.len + CT_KEYS - 1) / CT_KEYS;
    x.nst = (x.len + CT_SUB - 1) / CT_SUB;
    return x;
}

template <int DH, bool SPLIT>
__global__ void __launch_bounds__(CT_THREADS, 1)
cross_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmO, const CtParams p) {
    using L = CtLayout<DH>;
    constexpr int KVS = L::KVS, QB = L::QBUF, NCH = L::NCH;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    uint8_t* sQ = smem;
    uint8_t* sK = smem + L::OFF_K;
    uint8_t* sV = smem + L::OFF_V;
    CtBars* bars = reinterpret_cast<CtBars*>(smem + L::OFF_BAR);
    volatile int* abort_flag = &bars->abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&bars->q_full[i], 1);
            ptx::mbar_init(&bars->q_empty[i], 2);     // both MMA issuers
            for (int b = 0; b < 2; ++b) {
                ptx::mbar_init(&bars->s_full[i][b], 1);
                ptx::mbar_init(&bars->p_full[i][b], 4);   // one arrival per softmax warp
                ptx::mbar_init(&bars->o_done[i][b], 1);
            }
            ptx::mbar_init(&bars->o_free[i], 4);
            ptx::mbar_init(&bars->ost_full[i], 4);
            ptx::mbar_init(&bars->ost_free[i], 1);
        }
        for (int i = 0; i < 4; ++i) {
            ptx::mbar_init(&bars->k_full[i], 1);
            ptx::mbar_init(&bars->k_empty[i], 2);
            ptx::mbar_init(&bars->v_full[i], 1);
            ptx::mbar_init(&bars->v_empty[i], 2);
        }
        ptx::mbar_init(&bars->done, 2);
        bars->abort_flag = 0;
        ptx::fence_mbar_init();
    }
    if (warp == 10 && lane == 0) {
        ptx::prefetch_tensormap(&tmQ);
        ptx::prefetch_tensormap(&tmK);
        ptx::prefetch_tensormap(&tmV);
        ptx::prefetch_tensormap(&tmO);
    }
    if (warp == 1) {
        ptx::tmem_alloc(&bars->tmem_slot, 512);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, bars->tmem_slot, 0);
    griddep_wait();
    griddep_launch_dependents();
    // item of round i: there and back over the CTAs where the items fall in length
    const int item0 = SPLIT ? blockIdx.x / p.Z : blockIdx.x, step = SPLIT ? p.items : gridDim.x;
    auto item_of = [&](int i) -> int64_t {
        return (int64_t)i * step + (!SPLIT && p.sorted && (i & 1) ? step - 1 - item0 : item0);
    };
    if (!SPLIT && p.sorted) {
        int* lens = reinterpret_cast<int*>(smem + L::OFF_LENS);
        const int b = threadIdx.x;
        if (b < p.B) lens[b] = min(max(__ldg(p.kv_lens + b), 0), p.Tk);
        __syncthreads();
        if (b < p.B) {
            int before = 0;
            for (int i = 0; i < p.B; ++i) before += lens[i] > lens[b] || (lens[i] == lens[b] && i < b);
            bars->order[before] = (uint8_t)b;
        }
        __syncthreads();
    }
    float m = -INFINITY, l = 0.f;   // softmax warps: this row's maximum and sum
    // TMEM columns: S_g at 128 g, two buffers of 64 with P over each; O_g at 256 + 128 g

    if (warp >= 10) {
        if (lane == 0) {
            // ------------------------------------------------ TMA producers
            const bool kq = warp == 10;
            uint64_t* full = kq ? bars->k_full : bars->v_full;
            uint64_t* empty = kq ? bars->k_empty : bars->v_empty;
            uint8_t* ring = kq ? sK : sV;
            const CUtensorMap* tm = kq ? &tmK : &tmV;
            uint32_t it = 0, ii = 0;
            bool ok = true;
            for (int i = 0; item_of(i) < p.items && ok; ++i) {
                const CtItem x = ct_item<SPLIT>(p, (int)item_of(i), bars->order);
                if (x.nkt == 0) continue;
                if (kq) {
                    const uint32_t qb = ii % QB;
                    if (!ptx::mbar_wait_bounded<true>(&bars->q_empty[qb], ((ii / QB) & 1) ^ 1, abort_flag)) { ok = false; break; }
                    ptx::mbar_arrive_expect_tx(&bars->q_full[qb], x.nact * NCH * p.G * p.TT * 128);
                    for (int g = 0; g < x.nact; ++g)
                        for (int c = 0; c < NCH; ++c)
                            ptx::tma_load_4d(sQ + (qb * 2 + g) * L::TILE + c * CT_BOX, &tmQ, &bars->q_full[qb], c * 64,
                                             x.h * p.G, x.t0 + g * p.TT, x.b * p.qb);
                }
                ++ii;
                const int b = x.b * (kq ? p.kb : p.vb), h = x.h * (kq ? p.kh : p.vh);
                for (int j = 0; j < x.nkt; ++j, ++it) {
                    const uint32_t st = it % KVS;
                    if (!ptx::mbar_wait_bounded<true>(empty + st, ((it / KVS) & 1) ^ 1, abort_flag)) { ok = false; break; }
                    ptx::mbar_arrive_expect_tx(full + st, L::TILE);
                    for (int c = 0; c < NCH; ++c)
                        ptx::tma_load_4d(ring + st * L::TILE + c * CT_BOX, tm, full + st, c * 64, h, (x.kt0 + j) * CT_KEYS, b);
                }
            }
            if (!ok) {
                ct_error(p.err, ERRBIT_TIMEOUT_ATTENTION);
                *abort_flag = 1;
            }
            // copies in flight land before the CTA can exit
            if (kq)
                for (uint32_t i = 0; i < (uint32_t)QB; ++i)
                    if (ii > i && !ptx::mbar_wait_bounded(&bars->q_full[(ii - 1 - i) % QB], ((ii - 1 - i) / QB) & 1, nullptr))
                        ct_error(p.err, ERRBIT_TIMEOUT_TEARDOWN);
            for (uint32_t i = 0; i < (uint32_t)KVS; ++i)
                if (it > i && !ptx::mbar_wait_bounded(full + (it - 1 - i) % KVS, ((it - 1 - i) / KVS) & 1, nullptr))
                    ct_error(p.err, ERRBIT_TIMEOUT_TEARDOWN);
        }
    } else if (warp <= 1) {
        // ---------------------------------------------------- MMA issue, one lane; the others wait
        // alongside and help to clear V rows
        const int g = warp == 1 ? 0 : 1;
        constexpr uint32_t idS = ptx::idesc_bf16_f32(CT_ROWS, CT_SUB, false, false);
        constexpr uint32_t idO = ptx::idesc_bf16_f32(CT_ROWS, DH, false, true);
        const uint32_t tS = tmem + g * 128, tO = tmem + 256 + g * 128;
        uint32_t base = 0, ii = 0, pc = 0, ic = 0;   // key tiles, items with keys, half tiles, own items so far
        bool ok = true;
        auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
            return __all_sync(0xffffffffu, ptx::mbar_wait_bounded(bar, parity, abort_flag));
        };
        // S of half tile j of this item, n half tiles after the first of this group
        auto issue_S = [&](int j, uint32_t n, uint32_t qb, bool last_of_stage) -> bool {
            const uint32_t it = base + (j >> 1), st = it % KVS;
            if (!wait(&bars->k_full[st], (it / KVS) & 1)) return false;
            ptx::tc_fence_after();
            // descriptors count 16-byte units: those of later steps are sums
            const uint64_t qd = ptx::smem_desc(ptx::smem_addr(sQ + (qb * 2 + g) * L::TILE), 16, 1024, ptx::kLayoutSw128);
            const uint64_t kd = ptx::smem_desc(ptx::smem_addr(sK + st * L::TILE + (j & 1) * (CT_SUB * 128)), 16, 1024,
                                               ptx::kLayoutSw128);
            const uint32_t tD = tS + (n & 1) * CT_SUB;
            if (ptx::elect_one()) {
#pragma unroll
                for (int kk = 0; kk < DH / 16; ++kk) {
                    const uint64_t off = ((kk >> 2) * CT_BOX + (kk & 3) * 32) >> 4;
                    ptx::mma_bf16_ss(tD, qd + off, kd + off, idS, kk > 0);
                }
                ptx::mma_commit(&bars->s_full[g][n & 1]);
                if (last_of_stage) ptx::mma_commit(&bars->k_empty[st]);
            }
            __syncwarp();
            return true;
        };
        for (int i = 0; item_of(i) < p.items && ok; ++i) {
            const CtItem x = ct_item<SPLIT>(p, (int)item_of(i), bars->order);
            if (x.nkt == 0) continue;
            const uint32_t qb = ii % QB;
            ok = wait(&bars->q_full[qb], (ii / QB) & 1);
            ++ii;
            if (!ok) break;
            if (g >= x.nact) {
                // no tile for this group: release what the other issuer uses, each once it has landed
                if (ptx::elect_one()) ptx::mma_commit(&bars->q_empty[qb]);
                for (int j = 0; j < x.nkt && ok; ++j) {
                    const uint32_t it = base + j, st = it % KVS;
                    ok = wait(&bars->k_full[st], (it / KVS) & 1);
                    if (ok && ptx::elect_one()) ptx::mma_commit(&bars->k_empty[st]);
                    ok = ok && wait(&bars->v_full[st], (it / KVS) & 1);
                    if (ok && ptx::elect_one()) ptx::mma_commit(&bars->v_empty[st]);
                }
                base += x.nkt;
                continue;
            }
            auto scores = [&](int j) -> bool {   // and what their last user releases
                if (!issue_S(j, pc + j, qb, (j & 1) || j + 1 == x.nst)) return false;
                if (j + 1 == x.nst && ptx::elect_one()) ptx::mma_commit(&bars->q_empty[qb]);
                return true;
            };
            // the first scores overwrite the last item's P: after its last P V has read it
            ok = (pc == 0 || wait(&bars->o_done[g][(pc - 1) & 1], ((pc - 1) >> 1) & 1)) && scores(0) && (x.nst < 2 || scores(1));
            for (int j = 0; j < x.nst && ok; ++j) {
                const uint32_t it = base + (j >> 1), st = it % KVS, n = pc + j;
                if (!(ok = wait(&bars->v_full[st], (it / KVS) & 1))) break;
                const int valid = x.len - j * CT_SUB;
                uint8_t* v = sV + st * L::TILE + (j & 1) * (CT_SUB * 128);
                if (valid < CT_SUB) {
                    // rows past the length may hold anything, and 0 * NaN is NaN. Both issuers clear
                    // the same rows: the second finds zeros and writes zeros.
                    for (int i = valid * 8 + lane; i < CT_SUB * 8; i += 32)
#pragma unroll
                        for (int c = 0; c < NCH; ++c)
                            *reinterpret_cast<uint4*>(v + c * CT_BOX + i * 16) = make_uint4(0, 0, 0, 0);
                    ptx::fence_proxy_async_smem();
                    __syncwarp();
                }
                if (!(ok = wait(&bars->p_full[g][n & 1], (n >> 1) & 1))) break;
                if (j == 0 && ic > 0 && !(ok = wait(&bars->o_free[g], (ic - 1) & 1))) break;
                ptx::tc_fence_after();
                const uint64_t vd = ptx::smem_desc(ptx::smem_addr(v), CT_BOX, 1024, ptx::kLayoutSw128);
                const uint32_t tP = tS + (n & 1) * CT_SUB;
                if (ptx::elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < CT_SUB / 16; ++kk)   // 16 keys: 16 rows of V, 8 columns of bf16 pairs of P
                        ptx::mma_bf16_ts(tO, tP + kk * 8, vd + kk * (2048 >> 4), idO, j > 0 || kk > 0);
                    ptx::mma_commit(&bars->o_done[g][n & 1]);
                    if ((j & 1) || j + 1 == x.nst) ptx::mma_commit(&bars->v_empty[st]);
                }
                __syncwarp();
                if (j + 2 < x.nst) {
                    // the scores two on overwrite P: after P V has read it; the next ones are there
                    if (!(ok = wait(&bars->o_done[g][n & 1], (n >> 1) & 1))) break;
                    ok = scores(j + 2);
                }
            }
            ++ic;
            pc += x.nst;
            base += x.nkt;
        }
        if (!ok && lane == 0) {
            ct_error(p.err, ERRBIT_TIMEOUT_MMA);
            *abort_flag = 1;
        }
        __syncwarp();
        if (ptx::elect_one()) {
            ptx::mma_commit(&bars->done);
            if (!ptx::mbar_wait_bounded(&bars->done, 0, nullptr)) ct_error(p.err, ERRBIT_TIMEOUT_TEARDOWN);
        }
    } else {
        // ---------------------------------------------------- softmax groups
        const int g = (warp - 2) >> 2, quarter = warp & 3, r = quarter * 32 + lane;
        const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
        const uint32_t tO = tmem + 256 + g * 128 + lane_off;
        uint8_t* stage = smem + L::OFF_O + g * CT_BOX;
        const bool storer = quarter == 2 && lane == 0;
        const float sl2 = p.scale_log2;
        uint32_t tt = 0, sc = 0;   // half tiles, staged boxes of this group so far
        bool ok = true;
        auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
            return __all_sync(0xffffffffu, ptx::mbar_wait_bounded(bar, parity, abort_flag));
        };
        for (int i = 0; item_of(i) < p.items && ok; ++i) {
            const CtItem x = ct_item<SPLIT>(p, (int)item_of(i), bars->order);
            if (g >= x.nact) continue;
            const int t0 = x.t0 + g * p.TT;
            // a warp whose 32 rows hold no query only keeps the barrier protocol
            const bool live = quarter * 32 < min(p.TT, p.Tq - t0) * p.G;
            m = -INFINITY;
            l = 0.f;
            for (int j = 0; j < x.nst; ++j, ++tt) {
                if (!(ok = wait(&bars->s_full[g][tt & 1], (tt >> 1) & 1))) break;
                ptx::tc_fence_after();
                const uint32_t tS = tmem + g * 128 + (tt & 1) * CT_SUB + lane_off;
                if (live) {
                    uint32_t sv[CT_SUB];   // S, then P packed in place
                    ptx::tmem_ld_32x32b_x32(tS, *reinterpret_cast<uint32_t(*)[32]>(&sv[0]));
                    ptx::tmem_ld_32x32b_x32(tS + 32, *reinterpret_cast<uint32_t(*)[32]>(&sv[32]));
                    ptx::tmem_ld_wait();
                    const int valid = x.len - j * CT_SUB;
                    if (valid < CT_SUB) {
#pragma unroll
                        for (int e = 0; e < CT_SUB; ++e)
                            if (e >= valid) sv[e] = __float_as_uint(-INFINITY);
                    }
                    float mx[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) mx[e] = __uint_as_float(sv[e]);
#pragma unroll
                    for (int e = 8; e < CT_SUB; ++e) mx[e & 7] = fmaxf(mx[e & 7], __uint_as_float(sv[e]));
                    const float mrow = fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])),
                                             fmaxf(fmaxf(mx[4], mx[5]), fmaxf(mx[6], mx[7]))) * sl2;
                    float alpha = 1.f;
                    if (mrow > m + CT_SLACK || m == -INFINITY) {   // raise the maximum
                        const float m_new = fmaxf(m, mrow);
                        if (m_new > -INFINITY) alpha = exp2_approx(m - m_new);
                        m = m_new;
                    }
                    const float base = m == -INFINITY ? 0.f : m;   // only infinite scores so far: weights of zero
                    const bool coarse = fabsf(base) > CT_COARSE;
                    if (__any_sync(0xffffffffu, (j > 0 && alpha != 1.f) || coarse)) {
                        if (j > 0) {
                            // P V of the half tile before writes O
                            if (!(ok = wait(&bars->o_done[g][(tt - 1) & 1], ((tt - 1) >> 1) & 1))) break;
                            ptx::tc_fence_after();
#pragma unroll
                            for (int c = 0; c < DH / 16; ++c) {
                                uint32_t ov[16];
                                ptx::tmem_ld_32x32b_x16(tO + c * 16, ov);
                                ptx::tmem_ld_wait();
#pragma unroll
                                for (int e = 0; e < 16; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
                                ptx::tmem_st_32x32b_x16(tO + c * 16, ov);
                            }
                        }
                        const float f = coarse ? sl2 : 1.f;
#pragma unroll
                        for (int e = 0; e < CT_SUB; ++e) sv[e] = __float_as_uint(__fmul_rn(__uint_as_float(sv[e]), f));
                    }
                    const float mul = coarse ? 1.f : sl2;
                    const unsigned long long s2 = f2_pack(mul, mul), nm = f2_pack(-base, -base);
                    unsigned long long ls[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
                    for (int e = 0; e < CT_SUB; e += 2) {
                        float x0, x1;
                        f2_unpack(f2_fma(f2_pack(__uint_as_float(sv[e]), __uint_as_float(sv[e + 1])), s2, nm), x0, x1);
                        const float p0 = exp2_approx(x0), p1 = exp2_approx(x1);
                        ls[(e >> 1) & 3] = f2_add(ls[(e >> 1) & 3], f2_pack(p0, p1));
                        sv[e >> 1] = pack_bf16x2(p0, p1);
                    }
                    ptx::tmem_st_32x32b_x32(tS, *reinterpret_cast<uint32_t(*)[32]>(&sv[0]));
                    float a0, a1, b0, b1;
                    f2_unpack(f2_add(ls[0], ls[1]), a0, a1);
                    f2_unpack(f2_add(ls[2], ls[3]), b0, b1);
                    l = l * alpha + ((a0 + a1) + (b0 + b1));
                    ptx::tmem_st_wait();
                }
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&bars->p_full[g][tt & 1]);
            }
            if (!ok) break;
            if (x.nkt > 0) {
                if (!(ok = wait(&bars->o_done[g][(tt - 1) & 1], ((tt - 1) >> 1) & 1))) break;
                ptx::tc_fence_after();
            }
            if (SPLIT) continue;   // joined below
            const float inv = 1.f / l;
#pragma unroll 1
            for (int c = 0; c < NCH; ++c, ++sc) {
                // the previous store has read the staging box
                if (sc > 0 && !(ok = wait(&bars->ost_free[g], (sc - 1) & 1))) break;
                if (live) {
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        uint32_t ov[16];
                        if (x.nkt > 0 && c * 64 + u * 16 < DH) {
                            ptx::tmem_ld_32x32b_x16(tO + c * 64 + u * 16, ov);
                            ptx::tmem_ld_wait();
                        } else {
#pragma unroll
                            for (int e = 0; e < 16; ++e) ov[e] = 0u;
                        }
                        uint32_t w[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const float lo = __uint_as_float(ov[2 * e]), hi = __uint_as_float(ov[2 * e + 1]);
                            w[e] = x.nkt > 0 ? pack_bf16x2(lo * inv, hi * inv) : 0u;
                        }
                        // 16-byte unit i of row r at i ^ (r % 8)
                        *reinterpret_cast<uint4*>(stage + r * 128 + (((2 * u) ^ (r & 7)) << 4)) =
                            make_uint4(w[0], w[1], w[2], w[3]);
                        *reinterpret_cast<uint4*>(stage + r * 128 + (((2 * u + 1) ^ (r & 7)) << 4)) =
                            make_uint4(w[4], w[5], w[6], w[7]);
                    }
                }
                ptx::fence_proxy_async_smem();
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (c == NCH - 1 && x.nkt > 0) ptx::mbar_arrive(&bars->o_free[g]);   // O has been read
                    ptx::mbar_arrive(&bars->ost_full[g]);
                }
                bool sok = true;
                if (storer) {
                    sok = ptx::mbar_wait_bounded(&bars->ost_full[g], sc & 1, abort_flag);
                    if (sok) {
                        ptx::tma_store_4d(&tmO, stage, c * 64, x.h * p.G, t0, x.b);
                        ptx::bulk_commit_group();
                        ptx::bulk_wait_group_read<0>();
                        ptx::mbar_arrive(&bars->ost_free[g]);
                    }
                }
                if (!(ok = __all_sync(0xffffffffu, sok))) break;
            }
        }
        if (storer) ptx::bulk_wait_group<0>();   // the group's last store has completed
        if (!ok) {
            if (lane == 0) ct_error(p.err, ERRBIT_TIMEOUT_ATTENTION);
            *abort_flag = 1;
        }
    }

    __syncthreads();
    if constexpr (SPLIT) {
        // O, m and l of both groups over the K and V rings, which nobody reads any more; rows of
        // DH + 4 floats keep the 16-byte writes of eight rows in different banks
        constexpr int LD = DH + 4;
        float* jO = reinterpret_cast<float*>(sK);
        float* jm = jO + 2 * CT_ROWS * LD;
        static_assert((2 * CT_ROWS * LD + 4 * CT_ROWS) * 4 <= L::OFF_BAR - L::OFF_K, "join");
        const CtItem x = ct_item<true>(p, item0, nullptr);
        if (warp >= 2 && warp <= 9) {
            const int g = (warp - 2) >> 2, quarter = warp & 3, r = quarter * 32 + lane;
            float* row = jO + (g * CT_ROWS + r) * LD;
            ptx::tc_fence_after();
#pragma unroll
            for (int c = 0; c < DH / 16; ++c) {
                uint32_t ov[16];
                ptx::tmem_ld_32x32b_x16(tmem + 256 + g * 128 + ((uint32_t)(quarter * 32) << 16) + c * 16, ov);
                ptx::tmem_ld_wait_for(ov);
#pragma unroll
                for (int e = 0; e < 16; e += 4) {   // a part without keys adds nothing
                    const uint4 v = x.nkt > 0 ? make_uint4(ov[e], ov[e + 1], ov[e + 2], ov[e + 3]) : make_uint4(0, 0, 0, 0);
                    *reinterpret_cast<uint4*>(row + c * 16 + e) = v;
                }
            }
            jm[g * CT_ROWS + r] = m;
            jm[2 * CT_ROWS + g * CT_ROWS + r] = l;
            ptx::tc_fence_before();
        }
        ptx::cluster_sync();   // every part is in place
        const uint32_t own = ptx::smem_addr(jO), own_m = ptx::smem_addr(jm);
        const int rows = x.nact * CT_ROWS, share = (rows + p.Z - 1) / p.Z, z = (int)ptx::cluster_ctarank();
        const bool clean = *abort_flag == 0;
        for (int i = threadIdx.x; i < share * (DH / 4); i += CT_THREADS) {
            const int gr = z * share + i / (DH / 4), c = (i % (DH / 4)) * 4;   // group * 128 + row, column
            const int r = gr % CT_ROWS, t = x.t0 + (gr / CT_ROWS) * p.TT + r / p.G;
            if (gr >= rows || r >= p.TT * p.G || t >= p.Tq) continue;
            float mz[CT_MAXZ], lz[CT_MAXZ];
            float4 oz[CT_MAXZ];
#pragma unroll
            for (int y = 0; y < CT_MAXZ; ++y) {
                if (y >= p.Z) break;
                mz[y] = ptx::ld_cluster_f32(ptx::mapa_shared(own_m + gr * 4, y));
                lz[y] = ptx::ld_cluster_f32(ptx::mapa_shared(own_m + (2 * CT_ROWS + gr) * 4, y));
                oz[y] = ptx::ld_cluster_f32x4(ptx::mapa_shared(own + (gr * LD + c) * 4, y));
            }
            float mx = -INFINITY;
#pragma unroll
            for (int y = 0; y < CT_MAXZ; ++y)
                if (y < p.Z) mx = fmaxf(mx, mz[y]);
            const float base = mx == -INFINITY ? 0.f : mx;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            float sum = 0.f;
#pragma unroll
            for (int y = 0; y < CT_MAXZ; ++y) {
                if (y >= p.Z) break;
                const float f = exp2_approx(mz[y] - base);
                acc.x = fmaf(f, oz[y].x, acc.x);
                acc.y = fmaf(f, oz[y].y, acc.y);
                acc.z = fmaf(f, oz[y].z, acc.z);
                acc.w = fmaf(f, oz[y].w, acc.w);
                sum = fmaf(f, lz[y], sum);
            }
            const float inv = 1.f / sum;
            if (clean)
                *reinterpret_cast<uint2*>(p.o + (((int64_t)x.b * p.Tq + t) * p.H + x.h * p.G + r % p.G) * DH + c) =
                    x.any ? make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv))
                          : make_uint2(0u, 0u);
        }
        __syncwarp();
        ptx::cluster_sync();   // no CTA leaves while another reads its shared memory
    }
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, 512);
    }
}

template <int DH>
cudaError_t launch_ct(const CrossDesc& d, const DeviceInfo& dev, cudaStream_t s) {
    using L = CtLayout<DH>;
    const int G = (int)(d.H / d.Hkv), TT = CT_ROWS / G;
    const int64_t os[3] = {d.Tq * d.H * d.dh, d.H * d.dh, d.dh};
    alignas(64) CUtensorMap mq, mk, mv, mo;
    if (!ct_map(&mq, d.q, d.qs, d.B, d.Tq, d.H, d.dh, G, TT, CU_TENSOR_MAP_L2_PROMOTION_L2_128B) ||
        !ct_map(&mk, d.k, d.ks, d.B, d.Tk, d.Hkv, d.dh, 1, CT_KEYS, CU_TENSOR_MAP_L2_PROMOTION_L2_128B) ||
        !ct_map(&mv, d.v, d.vs, d.B, d.Tk, d.Hkv, d.dh, 1, CT_KEYS, CU_TENSOR_MAP_L2_PROMOTION_L2_128B) ||
        !ct_map(&mo, d.o, os, d.B, d.Tq, d.H, d.dh, G, TT, CU_TENSOR_MAP_L2_PROMOTION_NONE))
        return cudaErrorInvalidValue;
    CtParams p;
    p.kv_lens = d.kv_lens;
    p.B = (int)d.B;
    p.Tq = (int)d.Tq;
    p.Tk = (int)d.Tk;
    p.Hkv = (int)d.Hkv;
    p.G = G;
    p.TT = TT;
    p.npairs = (int)((d.Tq + 2 * TT - 1) / (2 * TT));
    p.items = (int)(d.B * d.Hkv * p.npairs);
    p.qb = d.qs[0] != 0;
    p.kb = d.ks[0] != 0;
    p.kh = d.ks[2] != 0;
    p.vb = d.vs[0] != 0;
    p.vh = d.vs[2] != 0;
    p.scale_log2 = (float)(d.scale * 1.4426950408889634);
    p.err = dev.err_word;
    p.H = (int)d.H;
    p.o = static_cast<__nv_bfloat16*>(d.o);
    // Items that fill at most half the SMs are split along the keys, each part four tiles at least. CTAs
    // fill an SM each, and clusters of eight of them do not pack into the GPU's SM groups.
    const int64_t nkt = (d.Tk + CT_KEYS - 1) / CT_KEYS;
    int Z = 1;
    while (Z < CT_MAXZ && (int64_t)p.items * Z * 2 <= (Z < 4 ? dev.num_sms : dev.num_sms / 2) && nkt >= Z * 2 * 4) Z *= 2;
    p.Z = Z;
    p.sorted = 0;
    if (Z > 1) {
        static std::atomic<uint64_t> attr{0};
        const cudaError_t e = set_smem_limit_once(cross_tc_kernel<DH, true>, L::SMEM, attr);
        if (e != cudaSuccess) return e;
        return launch_dependent_cluster(cross_tc_kernel<DH, true>, dim3(p.items * Z), dim3(CT_THREADS), Z, L::SMEM, s, mq, mk,
                                        mv, mo, p);
    }
    static std::atomic<uint64_t> attr{0};
    const cudaError_t e = set_smem_limit_once(cross_tc_kernel<DH, false>, L::SMEM, attr);
    if (e != cudaSuccess) return e;
    const int grid = p.items < dev.num_sms ? p.items : dev.num_sms;
    // Sequences of different lengths: the longest first, dealt out there and back, so that no CTA gets the
    // long ones of every round. Lengths from Tk / 2 to Tk, us in the order given / sorted: 16 x 500 queries over
    // 1025 keys, 16 heads of 80, 58.3 / 50.4; 8 of these with heads of 64, 29.0 / 25.3; 64 x 577 over 577, 140.7 /
    // 135.8. With many more sequences the rounds even out.
    p.sorted = p.kv_lens && d.B > 1 && d.B <= CT_SORT && p.items > grid;
    return launch_dependent(cross_tc_kernel<DH, false>, dim3(grid), dim3(CT_THREADS), L::SMEM, s, mq, mk, mv, mo, p);
}

}  // namespace

bool cross_tc_supported(const CrossDesc& d) {
    if (d.dt != DT_BF16 || (d.dh != 64 && d.dh != 80 && d.dh != 96 && d.dh != 128)) return false;
    const int64_t G = d.H / d.Hkv, lim = 0x7fffffff;
    // positive scales only: the row maximum is taken before scaling
    if (!((float)(d.scale * 1.4426950408889634) > 0.f) || G > CT_ROWS) return false;
    // the query producer may wait for a whole item: 2^26 keys take half of the wait's limit
    if (d.Tq > lim - 1024 || d.Tk > (1 << 26) || d.H > lim || d.B > lim) return false;
    if (d.B > lim / (d.Hkv * ((d.Tq * G + 1) / 2 + 1))) return false;   // items, at two rows each
    if (d.H > 1 && d.qs[2] == 0) return false;
    const int64_t os[3] = {d.Tq * d.H * d.dh, d.H * d.dh, d.dh};
    return ct_strides_ok(d.q, d.qs, d.Tq) && ct_strides_ok(d.k, d.ks, d.Tk) && ct_strides_ok(d.v, d.vs, d.Tk) &&
           ct_strides_ok(d.o, os, d.Tq) && ct_encode_fn() != nullptr;
}

cudaError_t launch_cross_tc(const CrossDesc& d, const DeviceInfo& dev, cudaStream_t s) {
    switch (d.dh) {
        case 64: return launch_ct<64>(d, dev, s);
        case 80: return launch_ct<80>(d, dev, s);
        case 96: return launch_ct<96>(d, dev, s);
        case 128: return launch_ct<128>(d, dev, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace vit
