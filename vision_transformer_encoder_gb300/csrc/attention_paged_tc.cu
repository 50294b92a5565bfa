// attention_paged_tc.cu -- paged attention on the sm_103a tensor cores (tcgen05 / TMEM / TMA), bf16 in and out, fp32
// softmax: the mathematics of attention_paged.cu for head widths 64, 80, 96 and 128 and pages of a multiple of 16 tokens.
//
// A tile is up to 128 query rows of ONE key head: TT tokens x the G query heads that share it (TT = 128 / G), packed
// row = token * G + head. A work item is a pair of tiles and a range of key tiles (128 keys each), of one of two kinds:
//   prefix  the tokens of all sequences of a group in turn, over the group's prefix: its keys are read and scored once
//   own     the tokens of one sequence over its own keys, up to the last that the tile sees, behind the prefix where that is
//           not worked off apart
// Ranges of keys leave parts (PagedParts), whole ones are stored. A persistent CTA per SM walks the items, the longest first.
//   warps 10, 11  TMA: Q and K tiles, V tiles, rings of their own; a tile is a box for each page in it (or for each 128
//                 of its tokens), every lane looking up and asking for one
//   warps 1, 0    MMA issue for softmax group 0, 1, 64 keys (half a tile) at a time: S = Q K^T (M 128, N 64, K dh), then
//                 O += P V (M 128, N dh, K 64) with P read from TMEM and V MN-major
//   warps 2-5, 6-9  softmax groups 0 and 1, one query row per thread
// With two tiles each group has one, and both use every key tile up to their last. With one tile (few rows, as in decoding
// behind a shared prefix) the groups take every other key tile each, and group 0 joins both accumulators from TMEM. What a
// group does not use of the rings the producers release for it.
//
// Scores, weights and the slack on the running maximum are those of attention_cross_tc.cu: P is rounded to bf16 for the
// second product, as one tcgen05.mma has both operands in one type and V is bf16 (its sum is not): outputs are off by 2.3e-3 in the
// 2-norm where their own rounding alone leaves 1.7e-3; P as two numbers of bf16 would take that back at twice the second
// product. Exponentials are the hardware's, good to 2^-22. Keys past a row's limit and on absent pages get weight 0 by position; V rows past the
// last key are cleared, and absent pages read as zeros. Weights of zero still meet the values of later tokens: a row of O that is
// not finite, where not all rows see all keys, is made again key by key.
//
// Bound by the matrix unit and, at widths below 128, by the softmax's instructions: 4 x 2048 queries behind 8200 keys, 16 heads of
// 128 on 2 key heads, 540 us (1.14 PFLOP/s; a half tile of both groups 1720 cycles, its products 1280 of them); 2 x 1025 queries over 4100
// keys, 12 heads of 64, 56 us (0.40 PFLOP/s: one round of 120 items, 1450 cycles to a half tile). With few rows, by HBM: 64 x 3
// queries behind 16 prefixes of up to 8200 keys, 39.9 us with the own keys and the join.
//
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

constexpr int PT_ROWS = 128, PT_KEYS = 128, PT_SUB = 64, PT_THREADS = 384;
constexpr int PT_BOX = PT_ROWS * 128;      // 64 columns x 128 rows: 16 KB
constexpr int PT_SORT = 128;               // sequences that are put in order of their lengths, at most
constexpr float PT_SLACK = 8.f;            // log2 of the weights that are carried before a rescale
constexpr float PT_COARSE = 16777216.f;    // maxima from which products are rounded before the maximum is taken off

// NARROW: items of one tile only, which leave room for deeper rings.
template <int DH, bool NARROW> struct PtLayout {
    static_assert(DH % 16 == 0 && DH >= 64 && DH <= 128, "head width");
    static constexpr int NCH = (DH + 63) / 64;           // 64-column boxes per tile
    static constexpr int TILE = NCH * PT_BOX;
    static constexpr int QT = NARROW ? 1 : 2;            // query tiles of a buffer
    static constexpr int QBUF = NCH == 2 ? 1 : 2;
    static constexpr int KS = NCH == 2 ? 2 : NARROW ? 5 : 4;               // stages of the rings
    static constexpr int VS = NCH == 2 ? (NARROW ? 3 : 2) : NARROW ? 6 : 4;
    static constexpr int OFF_K = QBUF * QT * TILE;
    static constexpr int OFF_V = OFF_K + KS * TILE;
    static constexpr int OFF_BAR = OFF_V + VS * TILE;
    static constexpr int OFF_ML = OFF_BAR + 1024;        // group 1's maxima and sums for group 0; lengths while sorting
    static constexpr int SMEM = OFF_ML + 1024 + 1024;
    static_assert(SMEM <= 227 * 1024, "shared memory");
};

struct PtParams {
    PagedDesc d;
    PagedParts parts;            // n 0: rows are stored
    int G, TT, S;                // S sequences to a group
    int unit;                    // tokens of a box
    int with_prefix;             // own items take the prefix along
    int prefix_items, items;     // prefix items first
    int prefix_pairs, own_pairs, prefix_parts, own_parts;
    int qb, qpb;                 // 0 where the queries have one sequence (group) for all
    int sorted;                  // own items by falling length
    float scale_log2;
    uint32_t* err;
};

struct PtBars {
    uint64_t q_full[2], q_empty[2];
    uint64_t k_full[6], k_empty[6], v_full[6], v_empty[6];
    // two of each for the half tiles in turn: a waiter may be one phase behind, never two
    uint64_t s_full[2][2], p_full[2][2], o_done[2][2], o_free[2];
    uint64_t ml_full;            // group 1's part of a shared tile is there
    uint64_t x_full[2], x_empty[2];   // items, as the producer of keys makes them out ahead of the others
    uint64_t done;
    uint32_t tmem_slot;
    int abort_flag;
    uint8_t order[PT_SORT];      // sequences, the longest first
};

struct alignas(16) PtItem {
    bool prefix;                 // kind
    int at, h, z;                // sequence or group, key head, part
    int t0, tokens;              // first token of the pair, tokens of the sequence (group)
    int live;                    // tiles with queries that are worked off: 0, 1, 2
    int len0, len1;              // keys of the prefix, and of its own up to the last that the pair sees
    int n0;                      // key tiles of the prefix
    int low, new_;               // query t sees own keys before low + t; new tokens
    int kt0;                     // first key tile of the range
    int count0, count1;          // key tiles of it that tile 0, tile 1 see
    bool gaps;                   // some page of the range is absent: half tiles are looked at one by one then
    const int32_t *table0, *table1;

    __device__ __forceinline__ int count(int g) const { return g ? count1 : count0; }
    __device__ __forceinline__ int tiles() const { return max(count0, count1); }
    __device__ __forceinline__ bool shared() const { return live == 1; }
    // key tiles and half tiles of group g
    __device__ __forceinline__ int own_tiles(int g) const { return shared() ? (count0 + 1 - g) >> 1 : count(g); }
    __device__ __forceinline__ int tile(int g, int j) const { return shared() ? 2 * j + g : j; }
    // keys of key tile j (of the range) in front of its end, for query tile g: more than 128 where all are
    __device__ __forceinline__ int keys(int j, int limit) const {
        const int t = kt0 + j;
        return t < n0 ? len0 - t * PT_KEYS : limit - (t - n0) * PT_KEYS;
    }
    // own keys that some row of query tile g sees
    __device__ __forceinline__ int limit(const PtParams& p, int g) const {
        if (prefix || t0 + g * p.TT >= new_) return 0;
        return max(0, low + min(t0 + (g + 1) * p.TT, new_) - 1);
    }
    __device__ __forceinline__ int halves(const PtParams& p, int g) const {
        const int n = own_tiles(g), q = shared() ? 0 : g;
        if (n == 0) return 0;
        const int j = tile(g, n - 1);
        // only the last key tile of all may end in its first half
        return 2 * n - (j == count(q) - 1 && keys(j, limit(p, q)) <= PT_SUB);
    }
};

struct PtShared {
    PtBars bars;
    PtItem items[2];
};
static_assert(sizeof(PtShared) <= 1024, "barriers and items");

__device__ __forceinline__ PtItem pt_item(const PtParams& p, int item, const uint8_t* order) {
    const PagedDesc& d = p.d;
    PtItem x;
    x.prefix = item < p.prefix_items;
    int i = x.prefix ? item : item - p.prefix_items;
    const int Hkv = (int)d.Hkv, Tq = (int)d.Tq;
    const int ahead = x.prefix || p.with_prefix;
    if (x.prefix) {
        x.z = i % p.prefix_parts;
        i /= p.prefix_parts;
        x.h = i % Hkv;
        i /= Hkv;
        x.t0 = i % p.prefix_pairs * 2 * p.TT;
        x.at = i / p.prefix_pairs;
        x.tokens = p.S * Tq;
        x.new_ = x.tokens;
        x.low = 0;
        x.len1 = 0;
        x.table1 = nullptr;
    } else {
        // the last pairs, which see the most keys, first
        x.z = i % p.own_parts;
        i /= p.own_parts;
        x.h = i % Hkv;
        i /= Hkv;
        x.at = i % (int)d.B;
        x.t0 = (p.own_pairs - 1 - i / (int)d.B) * 2 * p.TT;
        if (p.sorted) x.at = order[x.at];
        x.tokens = Tq;
        x.new_ = d.q_lens ? min(max(load(d.q_lens + x.at), 0), Tq) : Tq;
        const int len = min(max(load(d.kv_lens + x.at), 0), (int)(d.table_pages * d.page));
        x.low = len - (x.new_ - 1);
        x.table1 = d.table + (int64_t)x.at * d.table_pages;
    }
    x.live = x.t0 >= x.new_ ? 0 : x.t0 + p.TT >= x.new_ ? 1 : 2;
    x.len0 = 0;
    x.table0 = nullptr;
    if (ahead) {
        const int g = x.prefix ? x.at : x.at / p.S;
        x.len0 = min(max(load(d.prefix_lens + g), 0), (int)(d.prefix_pages * d.page));
        x.table0 = d.prefix_table + (int64_t)g * d.prefix_pages;
    }
    x.n0 = (x.len0 + PT_KEYS - 1) / PT_KEYS;
    if (!x.prefix) x.len1 = max(x.limit(p, 0), x.limit(p, 1));
    const int seen0 = x.live > 0 ? x.n0 + (x.limit(p, 0) + PT_KEYS - 1) / PT_KEYS : 0;
    const int seen1 = x.live > 1 ? x.n0 + (x.limit(p, 1) + PT_KEYS - 1) / PT_KEYS : 0;
    const int all = max(seen0, seen1), Z = x.prefix ? p.prefix_parts : p.own_parts, per = (all + Z - 1) / Z;
    x.kt0 = min(x.z * per, all);
    const int end = min(x.kt0 + per, all);
    x.count0 = max(0, min(seen0, end) - x.kt0);
    x.count1 = max(0, min(seen1, end) - x.kt0);
    return x;
}

// One row from the definition, over the key tiles of the item's range: only where a product with a weight of zero was not a
// number. False where no value that the row does not see is to blame. acc: dh sums, their maximum and sum of weights, all
// of these scores: the products' own are rounded differently, and far from zero that makes another weight. 16 keys, which
// lie in one page, at a time: 21 ms for 256 rows x 4096 keys of 128.
__device__ __noinline__ bool pt_row(const PtParams& p, const PtItem& x, int t, int head, int lim, float* acc) {
    const PagedDesc& d = p.d;
    const int dh = (int)d.dh, page = (int)d.page, tiles = x.tiles();
    auto row = [&](const void* pool, const int64_t (&st)[3], bool ahead, int u) -> const __nv_bfloat16* {
        const int pg = load((ahead ? x.table0 : x.table1) + u / page);
        if (pg < 0 || pg >= d.pages) return nullptr;
        return static_cast<const __nv_bfloat16*>(pool) + pg * st[0] + u % page * st[1] + x.h * st[2];
    };
    auto unit = [](const __nv_bfloat16* from, float (&to)[8]) {
        const uint4 raw = *reinterpret_cast<const uint4*>(from);
        const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = unpack_bf16x2(w[i]);
            to[2 * i] = f.x;
            to[2 * i + 1] = f.y;
        }
    };
    bool blame = false;
    for (int u = max(lim, 0); u < x.len1 && !blame; ++u) {
        const __nv_bfloat16* v = row(d.v, d.vs, false, u);
        for (int c = 0; v && c < dh; ++c) blame = blame || !isfinite(__bfloat162float(v[c]));
    }
    if (!blame) return false;
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(d.q) + head * d.qs[2] + x.at * d.qs[0] + t * d.qs[1];
    float m = -INFINITY, l = 0.f;
    for (int c = 0; c < dh; ++c) acc[c] = 0.f;
    for (int j = 0; j < tiles; ++j) {
        const bool ahead = x.kt0 + j < x.n0;
        const int first = (ahead ? x.kt0 + j : x.kt0 + j - x.n0) * PT_KEYS, last = min(PT_KEYS, x.keys(j, lim));
        for (int u = 0; u < last; u += 16) {
            const __nv_bfloat16 *k = row(d.k, d.ks, ahead, first + u), *v = row(d.v, d.vs, ahead, first + u);
            if (!k) continue;
            float s[16] = {};
            for (int c = 0; c < dh; c += 8) {
                float a[8];
                unit(q + c, a);
#pragma unroll
                for (int y = 0; y < 16; ++y) {
                    if (u + y >= last) continue;
                    float b[8];
                    unit(k + y * d.ks[1] + c, b);
#pragma unroll
                    for (int e = 0; e < 8; ++e) s[y] = fmaf(a[e], b[e], s[y]);
                }
            }
            float top = m;
#pragma unroll
            for (int y = 0; y < 16; ++y) {
                s[y] = u + y < last ? __fmul_rn(s[y], p.scale_log2) : -INFINITY;
                top = fmaxf(top, s[y]);
            }
            const float base = top == -INFINITY ? 0.f : top, alpha = exp2_approx(m - base);
            m = top;
            l *= alpha;
#pragma unroll
            for (int y = 0; y < 16; ++y) {
                s[y] = exp2_approx(s[y] - base);
                l += s[y];
            }
            bool over = l != 0.f;   // nothing can change any more
            for (int c = 0; c < dh; c += 8) {
                float a[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) a[e] = acc[c + e] * alpha;
#pragma unroll
                for (int y = 0; y < 16; ++y) {
                    if (u + y >= last) continue;
                    float b[8];
                    unit(v + y * d.vs[1] + c, b);
#pragma unroll
                    for (int e = 0; e < 8; ++e) a[e] = fmaf(s[y], b[e], a[e]);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    acc[c + e] = a[e];
                    over = over && a[e] != a[e];
                }
            }
            if (over) j = tiles, u = last;
        }
    }
    acc[dh] = m;
    acc[dh + 1] = l;
    return true;
}

__device__ __forceinline__ void pt_error(uint32_t* err, uint32_t bit) {
    if (err) atomicOr(err, bit);
}

template <int DH, bool NARROW>
__global__ void __launch_bounds__(PT_THREADS, 1)
paged_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmQP,
                const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const __grid_constant__ PtParams p) {
    using L = PtLayout<DH, NARROW>;
    constexpr int KS = L::KS, VS = L::VS, QB = L::QBUF, QT = L::QT, NCH = L::NCH;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    uint8_t* sQ = smem;
    uint8_t* sK = smem + L::OFF_K;
    uint8_t* sV = smem + L::OFF_V;
    PtShared* shared = reinterpret_cast<PtShared*>(smem + L::OFF_BAR);
    PtBars* bars = &shared->bars;
    float* sml = reinterpret_cast<float*>(smem + L::OFF_ML);
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
            ptx::mbar_init(&bars->x_full[i], 1);
            ptx::mbar_init(&bars->x_empty[i], 11);    // every other warp
        }
        for (int i = 0; i < 6; ++i) {
            ptx::mbar_init(&bars->k_full[i], 1);
            ptx::mbar_init(&bars->k_empty[i], 2);     // both groups, or the producer for one that does not use the stage
            ptx::mbar_init(&bars->v_full[i], 1);
            ptx::mbar_init(&bars->v_empty[i], 2);
        }
        ptx::mbar_init(&bars->ml_full, 4);
        ptx::mbar_init(&bars->done, 2);
        bars->abort_flag = 0;
        ptx::fence_mbar_init();
    }
    if (warp == 10 && lane == 0) {
        ptx::prefetch_tensormap(&tmQ);
        ptx::prefetch_tensormap(&tmQP);
        ptx::prefetch_tensormap(&tmK);
        ptx::prefetch_tensormap(&tmV);
    }
    if (warp == 1) {
        ptx::tmem_alloc(&bars->tmem_slot, 512);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, bars->tmem_slot, 0);
    // While the kernel in front ends: lengths and page tables, of which the first item needs one after the other, go to L2.
    // They may still change, and are read behind the wait. (Looking keys up by them, for L2 too, held the warp up for
    // longer than it gained: 32 x 1 over 64 keys behind 1025, 13.5 -> 15.8 us.)
    if (warp == 2) {
        const int32_t* lens[3] = {p.d.kv_lens, p.d.q_lens, p.d.prefix_lens};
        for (int i = 0; i < 3; ++i)
            if (lens[i])
                for (int b = lane * 32; b < (i < 2 ? p.d.B : p.d.groups) && b < 4096; b += 1024) prefetch_l2(lens[i] + b);
        if (p.items > p.prefix_items)
            for (int b = lane; b < p.d.B && b < 128; b += 32) prefetch_l2(p.d.table + b * p.d.table_pages);
        if (p.d.prefix_table)
            for (int b = lane; b < p.d.groups && b < 128; b += 32) prefetch_l2(p.d.prefix_table + b * p.d.prefix_pages);
    }
    griddep_wait();
    griddep_launch_dependents();
    // item of round i: there and back over the CTAs, as the items fall in length
    const int item0 = blockIdx.x, step = gridDim.x;
    auto item_of = [&](int i) -> int64_t { return (int64_t)i * step + (i & 1 ? step - 1 - item0 : item0); };
    if (p.sorted) {
        int* lens = reinterpret_cast<int*>(sml);
        const int b = threadIdx.x, B = (int)p.d.B;
        if (b < B) lens[b] = max(load(p.d.kv_lens + b), 0);
        __syncthreads();
        if (b < B) {
            int before = 0;
            for (int i = 0; i < B; ++i) before += lens[i] > lens[b] || (lens[i] == lens[b] && i < b);
            bars->order[before] = (uint8_t)b;
        }
        __syncthreads();
    }
    // The i-th item of this CTA, for every warp but the one that makes it out; false where the wait gave up.
    auto take = [&](int i, PtItem& x) -> bool {
        if (!__all_sync(0xffffffffu, ptx::mbar_wait_bounded(&bars->x_full[i & 1], (i >> 1) & 1, abort_flag))) return false;
        x = shared->items[i & 1];
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&bars->x_empty[i & 1]);
        return true;
    };
    // TMEM columns: S_g at 128 g, two buffers of 64 with P over each; O_g at 256 + 128 g

    if (warp >= 10) {
        // ---------------------------------------------------- TMA producers, a lane to a box
        const bool kq = warp == 10;
        const uint32_t KVS = kq ? KS : VS;
        uint64_t* full = kq ? bars->k_full : bars->v_full;
        uint64_t* empty = kq ? bars->k_empty : bars->v_empty;
        uint8_t* ring = kq ? sK : sV;
        const CUtensorMap* tm = kq ? &tmK : &tmV;
        const int unit = p.unit, page = (int)p.d.page;
        uint32_t it = 0, ii = 0;
        bool ok = true;
        auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
            return __all_sync(0xffffffffu, ptx::mbar_wait_bounded<true>(bar, parity, abort_flag));
        };
        for (int i = 0; item_of(i) < p.items && ok; ++i) {
            PtItem x;
            if (kq) {
                x = pt_item(p, (int)item_of(i), bars->order);
                x.gaps = false;
                const int end = x.kt0 + x.tiles();
                if (x.kt0 < x.n0)
                    for (int e = x.kt0 * PT_KEYS / page + lane; e * page < min(x.len0, end * PT_KEYS); e += 32)
                        x.gaps = x.gaps || (uint32_t)load(x.table0 + e) >= (uint32_t)p.d.pages;
                for (int e = max(0, x.kt0 - x.n0) * PT_KEYS / page + lane; e * page < min(x.len1, (end - x.n0) * PT_KEYS); e += 32)
                    x.gaps = x.gaps || (uint32_t)load(x.table1 + e) >= (uint32_t)p.d.pages;
                x.gaps = __any_sync(0xffffffffu, x.gaps);
                if (!(ok = wait(&bars->x_empty[i & 1], ((i >> 1) & 1) ^ 1))) break;
                if (lane == 0) {
                    shared->items[i & 1] = x;
                    ptx::mbar_arrive(&bars->x_full[i & 1]);
                }
                __syncwarp();
            } else if (!(ok = take(i, x))) {
                break;
            }
            const int n = x.tiles();
            if (n == 0) continue;
            if (kq) {
                const uint32_t qb = ii % QB;
                if (!(ok = wait(&bars->q_empty[qb], ((ii / QB) & 1) ^ 1))) break;
                if (lane == 0) {
                    const CUtensorMap* tq = x.prefix ? &tmQP : &tmQ;
                    const int b = x.at * (x.prefix ? p.qpb : p.qb);
                    ptx::mbar_arrive_expect_tx(&bars->q_full[qb], x.live * NCH * p.G * p.TT * 128);
                    for (int g = 0; g < x.live; ++g)
                        for (int c = 0; c < NCH; ++c)
                            ptx::tma_load_4d(sQ + (qb * QT + g) * L::TILE + c * PT_BOX, tq, &bars->q_full[qb], c * 64, x.h * p.G,
                                             x.t0 + g * p.TT, b);
                }
                __syncwarp();
            }
            ++ii;
            for (int j = 0; j < n; ++j, ++it) {
                const int t = x.kt0 + j;
                const bool ahead = t < x.n0;
                const int key = (ahead ? t : t - x.n0) * PT_KEYS + lane * unit;
                const bool mine = lane * unit < PT_KEYS && key < (ahead ? x.len0 : x.len1);
                int pg = mine ? load((ahead ? x.table0 : x.table1) + key / page) : -1;
                if (pg < 0 || pg >= p.d.pages) pg = -1;   // an absent page: outside the tensor, zeros
                const uint32_t boxes = __popc(__ballot_sync(0xffffffffu, mine));
                const uint32_t st = it % KVS;
                if (!(ok = wait(empty + st, ((it / KVS) & 1) ^ 1))) break;
                if (lane == 0) {
                    ptx::mbar_arrive_expect_tx(full + st, boxes * NCH * unit * 128);
                    // for the group that does not use this tile
                    if (x.shared() || j >= x.count0) ptx::mbar_arrive(empty + st);
                    if (!x.shared() && j >= x.count1) ptx::mbar_arrive(empty + st);
                }
                __syncwarp();
                if (mine)
                    for (int c = 0; c < NCH; ++c)
                        ptx::tma_load_4d(ring + st * L::TILE + c * PT_BOX + lane * unit * 128, tm, full + st, c * 64, x.h, key % page, pg);
                __syncwarp();
            }
        }
        if (lane == 0) {
            if (!ok) {
                pt_error(p.err, ERRBIT_TIMEOUT_ATTENTION);
                *abort_flag = 1;
            }
            // copies in flight land before the CTA can exit
            if (kq)
                for (uint32_t i = 0; i < (uint32_t)QB; ++i)
                    if (ii > i && !ptx::mbar_wait_bounded(&bars->q_full[(ii - 1 - i) % QB], ((ii - 1 - i) / QB) & 1, nullptr))
                        pt_error(p.err, ERRBIT_TIMEOUT_TEARDOWN);
            for (uint32_t i = 0; i < KVS; ++i)
                if (it > i && !ptx::mbar_wait_bounded(full + (it - 1 - i) % KVS, ((it - 1 - i) / KVS) & 1, nullptr))
                    pt_error(p.err, ERRBIT_TIMEOUT_TEARDOWN);
        }
        __syncwarp();
    } else if (warp <= 1) {
        // ---------------------------------------------------- MMA issue, one lane; the others wait
        // alongside and help to clear V rows
        const int g = warp == 1 ? 0 : 1;
        constexpr uint32_t idS = ptx::idesc_bf16_f32(PT_ROWS, PT_SUB, false, false);
        constexpr uint32_t idO = ptx::idesc_bf16_f32(PT_ROWS, DH, false, true);
        const uint32_t tS = tmem + g * 128, tO = tmem + 256 + g * 128;
        uint32_t base = 0, ii = 0, pc = 0, ic = 0;   // key tiles, items with keys, half tiles, own items so far
        bool ok = true;
        auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
            return __all_sync(0xffffffffu, ptx::mbar_wait_bounded(bar, parity, abort_flag));
        };
        for (int i = 0; item_of(i) < p.items && ok; ++i) {
            PtItem x;
            if (!(ok = take(i, x))) break;
            const int n = x.tiles();
            if (n == 0) continue;
            const uint32_t qb = ii % QB;
            ok = wait(&bars->q_full[qb], (ii / QB) & 1);
            ++ii;
            if (!ok) break;
            const int nst = x.halves(p, g), qt = x.shared() ? 0 : g;
            if (nst == 0) {
                if (ptx::elect_one()) ptx::mma_commit(&bars->q_empty[qb]);
                base += n;
                continue;
            }
            // S of half tile j of this item, and what its last user releases
            auto scores = [&](int j) -> bool {
                const uint32_t it = base + x.tile(g, j >> 1), st = it % KS, b = (pc + j) & 1;
                if (!wait(&bars->k_full[st], (it / KS) & 1)) return false;
                ptx::tc_fence_after();
                // descriptors count 16-byte units: those of later steps are sums
                const uint64_t qd = ptx::smem_desc(ptx::smem_addr(sQ + (qb * QT + qt) * L::TILE), 16, 1024, ptx::kLayoutSw128);
                const uint64_t kd = ptx::smem_desc(ptx::smem_addr(sK + st * L::TILE + (j & 1) * (PT_SUB * 128)), 16, 1024,
                                                   ptx::kLayoutSw128);
                const uint32_t tD = tS + b * PT_SUB;
                if (ptx::elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < DH / 16; ++kk) {
                        const uint64_t off = ((kk >> 2) * PT_BOX + (kk & 3) * 32) >> 4;
                        ptx::mma_bf16_ss(tD, qd + off, kd + off, idS, kk > 0);
                    }
                    ptx::mma_commit(&bars->s_full[g][b]);
                    if ((j & 1) || j + 1 == nst) ptx::mma_commit(&bars->k_empty[st]);
                    if (j + 1 == nst) ptx::mma_commit(&bars->q_empty[qb]);
                }
                __syncwarp();
                return true;
            };
            // the first scores overwrite the last item's P: after its last P V has read it
            ok = (pc == 0 || wait(&bars->o_done[g][(pc - 1) & 1], ((pc - 1) >> 1) & 1)) && scores(0) && (nst < 2 || scores(1));
            for (int j = 0; j < nst && ok; ++j) {
                const int tile = x.tile(g, j >> 1);
                const uint32_t it = base + tile, st = it % VS, m = pc + j;
                if (!(ok = wait(&bars->v_full[st], (it / VS) & 1))) break;
                const int valid = x.keys(tile, x.len1) - (j & 1) * PT_SUB;
                uint8_t* v = sV + st * L::TILE + (j & 1) * (PT_SUB * 128);
                if (valid < PT_SUB) {
                    // rows past the last key may hold anything, and 0 * NaN is NaN. Both issuers clear
                    // the same rows: the second finds zeros and writes zeros.
                    for (int e = max(valid, 0) * 8 + lane; e < PT_SUB * 8; e += 32)
#pragma unroll
                        for (int c = 0; c < NCH; ++c)
                            *reinterpret_cast<uint4*>(v + c * PT_BOX + e * 16) = make_uint4(0, 0, 0, 0);
                    ptx::fence_proxy_async_smem();
                    __syncwarp();
                }
                if (!(ok = wait(&bars->p_full[g][m & 1], (m >> 1) & 1))) break;
                if (j == 0 && ic > 0 && !(ok = wait(&bars->o_free[g], (ic - 1) & 1))) break;
                ptx::tc_fence_after();
                const uint64_t vd = ptx::smem_desc(ptx::smem_addr(v), PT_BOX, 1024, ptx::kLayoutSw128);
                const uint32_t tP = tS + (m & 1) * PT_SUB;
                if (ptx::elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < PT_SUB / 16; ++kk)   // 16 keys: 16 rows of V, 8 columns of bf16 pairs of P
                        ptx::mma_bf16_ts(tO, tP + kk * 8, vd + kk * (2048 >> 4), idO, j > 0 || kk > 0);
                    ptx::mma_commit(&bars->o_done[g][m & 1]);
                    if ((j & 1) || j + 1 == nst) ptx::mma_commit(&bars->v_empty[st]);
                }
                __syncwarp();
                if (j + 2 < nst) {
                    // the scores two on overwrite P: after P V has read it; the next ones are there
                    if (!(ok = wait(&bars->o_done[g][m & 1], (m >> 1) & 1))) break;
                    ok = scores(j + 2);
                }
            }
            ++ic;
            pc += nst;
            base += n;
        }
        if (!ok && lane == 0) {
            pt_error(p.err, ERRBIT_TIMEOUT_MMA);
            *abort_flag = 1;
        }
        __syncwarp();
        if (ptx::elect_one()) {
            ptx::mma_commit(&bars->done);
            if (!ptx::mbar_wait_bounded(&bars->done, 0, nullptr)) pt_error(p.err, ERRBIT_TIMEOUT_TEARDOWN);
        }
    } else {
        // ---------------------------------------------------- softmax groups, a thread to a row
        const int g = (warp - 2) >> 2, quarter = warp & 3, r = quarter * 32 + lane;
        const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
        const uint32_t tO = tmem + 256 + g * 128 + lane_off;
        const float sl2 = p.scale_log2;
        const int unit = p.unit < PT_SUB ? p.unit : PT_SUB, page = (int)p.d.page, G = p.G;
        const int tok = r / G;
        uint32_t tt = 0, joins = 0;   // half tiles, shared tiles of this group so far
        bool ok = true;
        auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
            return __all_sync(0xffffffffu, ptx::mbar_wait_bounded(bar, parity, abort_flag));
        };
        for (int i = 0; item_of(i) < p.items && ok; ++i) {
            PtItem x;
            if (!(ok = take(i, x))) break;
            const int nst = x.halves(p, g), qt = x.shared() ? 0 : g;   // query tile that it works on
            const int t = x.t0 + qt * p.TT + tok;
            // a warp whose 32 rows hold no query only keeps the barrier protocol
            const int rows = min(p.TT, x.tokens - (x.t0 + qt * p.TT)) * G;
            const bool live = quarter * 32 < rows;
            const int most = x.limit(p, qt);
            const int lim = t < x.new_ ? x.low + t : most;   // own keys that this row sees
            float m = -INFINITY, l = 0.f;
            const bool gaps = x.gaps;
            bool coarse = false;
            for (int j = 0; j < nst; ++j, ++tt) {
                const int kt = x.kt0 + x.tile(g, j >> 1);
                const bool ahead = kt < x.n0;
                const int key = (ahead ? kt : kt - x.n0) * PT_KEYS + (j & 1) * PT_SUB;
                const int valid = (ahead ? x.len0 : lim) - key;
                // All rows of the warp see the whole half tile and have a maximum: no masks, and mostly none to raise. (At 128,
                // where the products are what takes longest, this way round is slower: 563 us instead of 539 for 4 x 2048
                // queries behind 8200 keys; below it is faster, 55.1 instead of 57.1 for 2 x 1025 over 4100.)
                const bool plain = DH < 128 && !gaps && __all_sync(0xffffffffu, valid >= PT_SUB && m > -INFINITY && !coarse);
                const uint32_t tS = tmem + g * 128 + (tt & 1) * PT_SUB + lane_off;
                if (!(ok = wait(&bars->s_full[g][tt & 1], (tt >> 1) & 1))) break;
                ptx::tc_fence_after();
                if (live) {
                    uint32_t sv[PT_SUB];   // S, then P packed in place; the largest of each half comes with the load
                    uint32_t(&s0)[32] = *reinterpret_cast<uint32_t(*)[32]>(&sv[0]);
                    uint32_t(&s1)[32] = *reinterpret_cast<uint32_t(*)[32]>(&sv[32]);
                    float mrow = ptx::tmem_ld_red_max_32x32b_x32(tS, s0);
                    float mx1 = ptx::tmem_ld_red_max_32x32b_x32(tS + 32, s1);
                    ptx::tmem_ld_wait_for(s0, mrow);
                    ptx::tmem_ld_wait_for(s1, mx1);
                    mrow = fmaxf(mrow, mx1) * sl2;
                    float alpha = 1.f, mul = sl2;
                    if (!plain || __any_sync(0xffffffffu, mrow > m + PT_SLACK)) {
                        if (gaps || __any_sync(0xffffffffu, valid < PT_SUB)) {
                            uint32_t absent = 0;
                            if (__builtin_expect(gaps, 0)) {
                                int pg = 0;   // of this lane's unit of the half tile
                                if (lane * unit < PT_SUB && key + lane * unit < (ahead ? x.len0 : x.len1))
                                    pg = load((ahead ? x.table0 : x.table1) + (key + lane * unit) / page);
                                absent = __ballot_sync(0xffffffffu, pg < 0 || pg >= p.d.pages);
                            }
                            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                            for (int e = 0; e < PT_SUB; e += 16) {
                                const bool away = absent >> (e / unit) & 1;
#pragma unroll
                                for (int y = e; y < e + 16; ++y) {
                                    if (y >= valid || away) sv[y] = __float_as_uint(-INFINITY);
                                    mx[y & 3] = fmaxf(mx[y & 3], __uint_as_float(sv[y]));
                                }
                            }
                            mrow = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sl2;
                        }
                        if (mrow > m + PT_SLACK || m == -INFINITY) {   // raise the maximum
                            const float m_new = fmaxf(m, mrow);
                            if (m_new > -INFINITY) alpha = exp2_approx(m - m_new);
                            m = m_new;
                        }
                        coarse = fabsf(m) > PT_COARSE && m > -INFINITY;
                        if (__any_sync(0xffffffffu, (j > 0 && alpha != 1.f) || coarse)) {
                            if (j > 0) {
                                // P V of the half tile before writes O
                                if (!(ok = wait(&bars->o_done[g][(tt - 1) & 1], ((tt - 1) >> 1) & 1))) break;
                                ptx::tc_fence_after();
#pragma unroll
                                for (int c = 0; c < DH; c += 16) {
                                    uint32_t ov[16];
                                    ptx::tmem_ld_32x32b_x16(tO + c, ov);
                                    ptx::tmem_ld_wait_for(ov);
#pragma unroll
                                    for (int e = 0; e < 16; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
                                    ptx::tmem_st_32x32b_x16(tO + c, ov);
                                }
                            }
                            const float f = coarse ? sl2 : 1.f;
#pragma unroll
                            for (int e = 0; e < PT_SUB; ++e) sv[e] = __float_as_uint(__fmul_rn(__uint_as_float(sv[e]), f));
                        }
                        mul = coarse ? 1.f : sl2;
                    }
                    const float base = m == -INFINITY ? 0.f : m;   // only infinite scores so far: weights of zero
                    const unsigned long long s2 = f2_pack(mul, mul), nm = f2_pack(-base, -base);
                    unsigned long long ls[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
                    for (int e = 0; e < PT_SUB; e += 2) {
                        float x0, x1;
                        f2_unpack(f2_fma(f2_pack(__uint_as_float(sv[e]), __uint_as_float(sv[e + 1])), s2, nm), x0, x1);
                        const float p0 = exp2_approx(x0), p1 = exp2_approx(x1);
                        ls[(e >> 1) & 3] = f2_add(ls[(e >> 1) & 3], f2_pack(p0, p1));
                        sv[e >> 1] = pack_bf16x2(p0, p1);
                    }
                    ptx::tmem_st_32x32b_x32(tS, s0);
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
            if (nst > 0) {
                if (!(ok = wait(&bars->o_done[g][(tt - 1) & 1], ((tt - 1) >> 1) & 1))) break;
                ptx::tc_fence_after();
            }
            // of a shared tile, group 1 hands its part to group 0 and stores what its own tile, which holds no new token, has: zeros
            bool have = nst > 0;
            float f0 = 1.f, f1 = 0.f;   // factors of O_0 and O_1
            const bool both = x.shared() && x.own_tiles(1) > 0;
            if (both) {
                if (g == 1) {
                    sml[r] = m;
                    sml[PT_ROWS + r] = l;
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(&bars->ml_full);
                    have = false;
                } else {
                    if (!(ok = wait(&bars->ml_full, joins & 1))) break;
                    ptx::tc_fence_after();
                    const float m1 = sml[r], l1 = sml[PT_ROWS + r], top = fmaxf(m, m1), base = top == -INFINITY ? 0.f : top;
                    f0 = exp2_approx(m - base);
                    f1 = exp2_approx(m1 - base);
                    l = f0 * l + f1 * l1;
                    m = top;
                }
                ++joins;
            }
            const int out_t0 = x.t0 + g * p.TT;
            if (g == 1 && x.live < 2) {
                have = false;
                m = -INFINITY;
                l = 0.f;
            }
            const int out_rows = min(p.TT, x.tokens - out_t0) * G;   // of this group's own query tile; none if it does not exist
            bool row = r < out_rows && t < x.new_ && !(g == 1 && x.live < 2);
            if (x.prefix && row && p.d.q_lens)   // a token of its sequence
                row = t % (int)p.d.Tq < load(p.d.q_lens + (int64_t)x.at * p.S + t / (int)p.d.Tq);
            if (!row) l = 0.f;
            const bool there = r < out_rows;
            const int64_t at = ((int64_t)x.at * x.tokens + out_t0 + tok) * p.d.H + x.h * G + r % G;   // row of the output
            if (quarter * 32 < out_rows) {
                const int64_t to = (int64_t)(x.prefix ? x.z : p.prefix_parts + x.z) * p.parts.rows + at;
                float* part = static_cast<float*>(p.parts.acc) + to * DH;
                __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.d.o) + at * DH;
                bool none = l == 0.f;
                float inv = none ? 0.f : 1.f / l;
                // A thread stores its row. (Turned round in shared memory, so that neighbouring lanes store one row, an item's
                // end takes as long: 5100 cycles for 128 x 128.)
                auto put = [&](int c, const float (&v)[8]) {
                    if (!there || (p.parts.n && none)) return;
                    if (p.parts.n) {
                        *reinterpret_cast<float4*>(part + c) = make_float4(v[0], v[1], v[2], v[3]);
                        *reinterpret_cast<float4*>(part + c + 4) = make_float4(v[4], v[5], v[6], v[7]);
                    } else {
                        uint32_t w[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) w[e] = none ? 0u : pack_bf16x2(v[2 * e] * inv, v[2 * e + 1] * inv);
                        *reinterpret_cast<uint4*>(out + c) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                };
                float odd = 0.f;
                // A short loop: it runs once an item, and its code has to be fetched (questions 51.7 -> 50.9 us, drafts 41.0 -> 40.6).
                // Items of many keys at 128 lose by what else the compiler then does (4 x 2048 behind 8200: 539 -> 556).
                constexpr int UNROLL = DH == 128 && !NARROW ? DH / 16 : 1;
#pragma unroll UNROLL
                for (int c = 0; c < DH; c += 16) {
                    uint32_t ov[16];
                    if (have) {   // not group 1 behind a shared tile, which has nothing of its own, nor anything beyond its columns
                        ptx::tmem_ld_32x32b_x16(tO + c, ov);
                        ptx::tmem_ld_wait_for(ov);
                        if (both) {
                            uint32_t o1[16];
                            ptx::tmem_ld_32x32b_x16(tO + 128 + c, o1);
                            ptx::tmem_ld_wait_for(o1);
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                ov[e] = __float_as_uint(fmaf(f1, __uint_as_float(o1[e]), f0 * __uint_as_float(ov[e])));
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 16; ++e) ov[e] = 0u;
                    }
#pragma unroll
                    for (int e = 0; e < 16; e += 8) {
                        float v[8];
#pragma unroll
                        for (int y = 0; y < 8; ++y) v[y] = __uint_as_float(ov[e + y]);
#pragma unroll
                        for (int y = 0; y < 8; ++y) odd = fmaf(v[y], 0.f, odd);
                        put(c + e, v);
                    }
                }
                // rows do not all see the same: values that this one does not see can make it a NaN
                if (__builtin_expect(row && x.len1 > 0 && odd != 0.f, 0)) {
                    const PtItem y = x;   // so that x itself keeps to registers
                    float acc[DH + 2];
                    if (pt_row(p, y, t, x.h * G + r % G, lim, acc)) {
                        m = acc[DH];
                        l = acc[DH + 1];
                        none = l == 0.f;
                        inv = none ? 0.f : 1.f / l;
                        for (int c = 0; c < DH; c += 8) put(c, *reinterpret_cast<float(*)[8]>(acc + c));
                    }
                }
                __syncwarp();
                if (p.parts.n && there) static_cast<float2*>(p.parts.ml)[to] = make_float2(none ? -INFINITY : m, l);
            }
            // O has been read: its group's next products may write it, and group 1's where it was read alongside
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (g == 0 ? nst > 0 : (nst > 0 && !both)) ptx::mbar_arrive(&bars->o_free[g]);
                if (g == 0 && both) ptx::mbar_arrive(&bars->o_free[1]);
            }
        }
        if (!ok) {
            if (lane == 0) pt_error(p.err, ERRBIT_TIMEOUT_ATTENTION);
            *abort_flag = 1;
        }
        __syncwarp();
    }

    __syncthreads();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, 512);
    }
}

// Rows of the group's sequences in turn: (groups, S Tq, H, dh). False where their strides do not make one.
bool merged(const PagedDesc& d, int64_t (&st)[3]) {
    const int64_t S = d.B / d.groups;
    if (S > 1 && d.Tq > 1 && d.qs[0] != d.Tq * d.qs[1]) return false;
    st[0] = S * d.qs[0];
    st[1] = d.Tq > 1 ? d.qs[1] : d.qs[0];
    st[2] = d.qs[2];
    return true;
}

template <int DH, bool NARROW> cudaError_t launch_pt(const PtParams& given, const DeviceInfo& dev, cudaStream_t s) {
    using L = PtLayout<DH, NARROW>;
    PtParams p = given;
    const PagedDesc& d = p.d;
    alignas(64) CUtensorMap mq, mqp, mk, mv;
    int64_t qm[3];
    const auto l2 = CU_TENSOR_MAP_L2_PROMOTION_L2_128B;
    if (!ct_map(&mk, d.k, d.ks, d.pages, d.page, d.Hkv, d.dh, 1, p.unit, l2) ||
        !ct_map(&mv, d.v, d.vs, d.pages, d.page, d.Hkv, d.dh, 1, p.unit, l2))
        return cudaErrorInvalidValue;
    // a map that no item uses is a copy of another
    mq = mqp = mk;
    if (p.items > p.prefix_items && !ct_map(&mq, d.q, d.qs, d.B, d.Tq, d.H, d.dh, p.G, p.TT, l2)) return cudaErrorInvalidValue;
    if (p.prefix_items && (!merged(d, qm) || !ct_map(&mqp, d.q, qm, d.groups, p.S * d.Tq, d.H, d.dh, p.G, p.TT, l2)))
        return cudaErrorInvalidValue;
    p.qb = d.qs[0] != 0;
    p.qpb = p.prefix_items && qm[0] != 0;
    static std::atomic<uint64_t> attr{0};
    const cudaError_t e = set_smem_limit_once(paged_tc_kernel<DH, NARROW>, L::SMEM, attr);
    if (e != cudaSuccess) return e;
    const int grid = p.items < dev.num_sms ? p.items : dev.num_sms;
    p.sorted = p.items - p.prefix_items > grid && d.B > 1 && d.B <= PT_SORT;
    return launch_dependent(paged_tc_kernel<DH, NARROW>, dim3(grid), dim3(PT_THREADS), L::SMEM, s, mq, mqp, mk, mv, p);
}

template <int DH> cudaError_t launch_pt(const PtParams& p, const DeviceInfo& dev, cudaStream_t s) {
    const bool one = (p.items == p.prefix_items || p.d.Tq <= p.TT) && (!p.prefix_items || p.S * p.d.Tq <= p.TT);
    return one ? launch_pt<DH, true>(p, dev, s) : launch_pt<DH, false>(p, dev, s);
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace

bool paged_tc_supported(const PagedDesc& d, bool own) {
    if (d.dt != DT_BF16 || (d.dh != 64 && d.dh != 80 && d.dh != 96 && d.dh != 128) || d.page % 16 != 0) return false;
    const int64_t G = d.H / d.Hkv, lim = 0x7fffffff, S = d.B / d.groups;
    // positive scales only: the row maximum is taken before scaling
    if (!((float)(d.scale * 1.4426950408889634) > 0.f) || G > PT_ROWS) return false;
    // the query producer may wait for a whole item: 2^26 keys take half of the wait's limit; own ones have parts, of fewer
    if ((d.table_pages + d.prefix_pages) * d.page > (own ? 32 * PAGED_TC_PART : 1 << 26)) return false;
    if (d.Tq > lim / 2 / S - 1024) return false;
    // items, at two rows each and 64 parts
    if (d.B > lim / 64 / (d.Hkv * (d.Tq * G / 2 + 2))) return false;
    if (d.H > 1 && d.qs[2] == 0) return false;
    int64_t qm[3];
    const int64_t os[3] = {d.Tq * d.H * d.dh, d.H * d.dh, d.dh};
    if (!ct_strides_ok(d.k, d.ks, d.page) || !ct_strides_ok(d.v, d.vs, d.page) || ct_encode_fn() == nullptr) return false;
    if (own) return ct_strides_ok(d.q, d.qs, d.Tq) && ct_strides_ok(d.o, os, d.Tq);
    return merged(d, qm) && ct_strides_ok(d.q, qm, S * d.Tq);
}

int64_t paged_tc_items(const PagedDesc& d, bool own) {
    const int64_t TT = PT_ROWS / (d.H / d.Hkv);
    return own ? d.B * d.Hkv * ceil_div(d.Tq, 2 * TT) : d.groups * d.Hkv * ceil_div(d.B / d.groups * d.Tq, 2 * TT);
}

int64_t paged_tc_rows(const PagedDesc& d) {
    const int64_t G = d.H / d.Hkv;
    return 2 * (PT_ROWS / G) * G;
}

bool paged_tc_apart(const PagedDesc& d) {
    // Rows of one sequence that leave their tiles mostly empty: packed with the others' they take half the tiles or less.
    const int64_t TT = PT_ROWS / (d.H / d.Hkv), S = d.B / d.groups;
    return S * ceil_div(d.Tq, TT) >= 2 * ceil_div(S * d.Tq, TT);
}

cudaError_t launch_paged_tc(const PagedDesc& d, const PagedPlan& plan, const PagedParts& parts, bool own, const DeviceInfo& dev,
                            cudaStream_t s) {
    PtParams p{};
    p.d = d;
    p.parts = parts;
    p.G = (int)(d.H / d.Hkv);
    p.TT = PT_ROWS / p.G;
    p.S = (int)(d.B / d.groups);
    p.unit = 16;
    while (p.unit < PT_KEYS && d.page % (2 * p.unit) == 0) p.unit *= 2;
    p.with_prefix = d.prefix_table && !plan.prefix_parts;
    p.prefix_pairs = (int)ceil_div(p.S * d.Tq, 2 * p.TT);
    p.own_pairs = (int)ceil_div(d.Tq, 2 * p.TT);
    p.prefix_parts = plan.prefix_parts;
    p.own_parts = plan.own_parts;
    p.prefix_items = plan.prefix_parts ? (int)(paged_tc_items(d, false) * plan.prefix_parts) : 0;
    p.items = p.prefix_items + (own ? (int)(paged_tc_items(d, true) * plan.own_parts) : 0);
    p.scale_log2 = (float)(d.scale * 1.4426950408889634);
    p.err = dev.err_word;
    switch (d.dh) {
        case 64: return launch_pt<64>(p, dev, s);
        case 80: return launch_pt<80>(p, dev, s);
        case 96: return launch_pt<96>(p, dev, s);
        case 128: return launch_pt<128>(p, dev, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace vit
