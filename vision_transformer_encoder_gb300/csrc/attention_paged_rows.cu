// attention_paged_rows.cu -- paged attention of few queries (decoding): the mathematics of attention_paged.cu where one key
// head serves at most 16 query rows (Tq * G <= 16), bf16, head width up to 128 in steps of 8, pages of a multiple of
// 16 tokens.
//
// Bound by reading the sequence's own keys and values once. They are dealt out in tiles of 32, two halves that lie in one page
// each, to the warps of one CTA or of a cluster of CTAs; every warp looks its pages up one tile ahead of asking for them, keeps
// its own running maximum, sum and output rows, joined at the end through shared memory and, between the CTAs of a cluster,
// distributed shared memory. 32 sequences of up to 577 keys, 16 heads of 64: 12.2 us (4.6 TB/s), 4 us of it the latency of length,
// page and first tile; 8 of up to 8200, 16 heads of 128 on 2 key heads: 16.6 us (3.0 TB/s), a warp's chain of products.
//
// The rows of the prefix, where there is one, were worked off by the kernel launched before this one: its parts are joined
// here. This kernel starts beside that one and waits for it only then: its own keys, queries and tables were there before that
// one began (it lets this one start behind its own wait).
//
// Rings and products are those of attention_cross_rows.cu: mma.m16n8k16 with the query rows as the n side,
// S^T = K Q^T and O^T = V^T P^T, K and V by TMA into a ring of each warp's own. Weights are rounded to bf16 for the second
// product, whose operands have one type, V's (their sum is not rounded): outputs are off by 2.3e-3 in the 2-norm where their own rounding
// alone leaves 1.7e-3. Weights as two numbers of bf16 would take that back at twice the second product. Exponentials are the
// hardware's, good to 2^-22, where a weight then keeps 2^-8.
//
// A query does not see later tokens, but the product adds their values times weights of zero. Where such a value is
// not finite, the tile is multiplied once per token with what that token does not see cleared.
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

constexpr int PR_ROWS = 16, PR_MAXZ = 8, PR_PARTS = 4, PR_KEYS = 32, PR_HALF = 16;   // a tile is two halves, each within one page
constexpr float PR_SLACK = 8.f;   // log2 of the weights that are carried before a rescale

struct PagedRowsParams {
    PagedDesc d;
    PagedParts parts;    // the prefix's; n 0: none
    float scale_log2;
    int Z;               // CTAs of a cluster
    uint32_t* err;
};

__device__ __forceinline__ bool not_finite(uint32_t pair) {
    return (pair & 0x7f80u) == 0x7f80u || (pair & 0x7f800000u) == 0x7f800000u;
}

// DHT: the head width rounded up to 64 or 128; columns past dh are zeros. NR: eight rows or sixteen.
template <int DHT, int NR, int NW, int STAGES, int MINB>
__global__ void __launch_bounds__(NW * 32, MINB)
paged_rows_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                  const __grid_constant__ PagedRowsParams p) {
    constexpr int NCH = DHT / 64, STAGE = PR_KEYS * NCH * 256;
    constexpr int BOX = PR_KEYS * 128;   // 64 columns of one tile
    constexpr int NT = PR_KEYS / 16;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t bars[NW][STAGES];
    const PagedDesc& d = p.d;
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c4 = lane & 3, r8 = lane >> 2;
    const int Z = p.Z, z = Z > 1 ? (int)ptx::cluster_ctarank() : 0;
    const int bh = blockIdx.x / Z, b = bh / (int)d.Hkv, h = bh % (int)d.Hkv;
    const int Tq = (int)d.Tq, G = (int)(d.H / d.Hkv), R = Tq * G, dh = (int)d.dh;
    uint64_t* bar = bars[warp];
    uint8_t* ring = smem + warp * STAGES * STAGE;
    // once a warp's keys are done, over its ring: O (R x dh), m and l (R each); behind the rings
    // this CTA's joined O, m and l
    constexpr int piece = STAGES * STAGE / 4;
    float* sm = reinterpret_cast<float*>(smem);
    float* wO = sm + warp * piece;
    float* jO = sm + NW * piece;
    static_assert(NR * 8 * (DHT + 2) <= piece, "output rows in a ring");
    if (lane == 0) {
        for (int i = 0; i < STAGES; ++i) ptx::mbar_init(bar + i, 1);
        ptx::fence_mbar_init();
        ptx::prefetch_tensormap(&tmK);
        ptx::prefetch_tensormap(&tmV);
    }
    __syncwarp();
    // tiles of this warp: first, first + stride, ...
    const int first = z * NW + warp, stride = Z * NW;
    if (!p.parts.n) {
        // While the kernel in front ends: what is read first goes to L2, by lengths and pages as they stand, which may
        // still change. They are read again behind the wait.
        if (lane < 2) {
            const int len = __ldcg(d.kv_lens + b), hpp = (int)d.page / PR_HALF;
#pragma unroll
            for (int i = 0; i < STAGES; ++i) {
                const int half = 2 * (first + i * stride) + lane;
                const int pg = half / hpp < d.table_pages && half < len / PR_HALF ? __ldcg(d.table + (int64_t)b * d.table_pages + half / hpp) : -1;
                if (pg < 0 || pg >= d.pages) continue;
#pragma unroll
                for (int c = 0; c < NCH; ++c) {
                    ptx::tma_prefetch_4d(&tmK, c * 64, h, half % hpp * PR_HALF, pg);
                    ptx::tma_prefetch_4d(&tmV, c * 64, h, half % hpp * PR_HALF, pg);
                }
            }
        }
        griddep_wait();
        griddep_launch_dependents();
    }

    const int held = (int)(d.table_pages * d.page), hpp = (int)d.page / PR_HALF;
    const int32_t* table = d.table + (int64_t)b * d.table_pages;
    // Lanes 0 and 1 look the pages of a tile's halves up: entry and half in the page, of the tile that comes next. Entries
    // behind the last key are read with the others, so that the first ones are asked for together with the length.
    int place = (2 * first + (lane & 1)) / hpp, part_of = (2 * first + (lane & 1)) % hpp;
    const int place_step = 2 * stride / hpp, part_step = 2 * stride % hpp;
    struct Page { int pg, half; };
    auto look_up = [&]() -> Page {   // in turn: first, first + stride, ...
        const Page x{place < d.table_pages ? load(table + place) : -1, part_of};
        place += place_step;
        part_of += part_step;
        if (part_of >= hpp) {
            part_of -= hpp;
            ++place;
        }
        return x;
    };
    Page ahead, early[STAGES];
#pragma unroll
    for (int i = 0; i < STAGES; ++i) early[i] = look_up();
    ahead = look_up();
    const int len = min(max(load(d.kv_lens + b), 0), held);
    const int new_ = d.q_lens ? min(max(load(d.q_lens + b), 0), Tq) : Tq;
    const int tiles = new_ > 0 ? (len + PR_KEYS - 1) / PR_KEYS : 0;   // a sequence without new tokens needs none
    uint32_t absent = 0;   // two bits of each stage: its halves' pages are
    auto request = [&](int tile, const Page& x, int st) {   // converged
        if (tile >= tiles) return;
        const bool on = lane < 2 && (tile * 2 + lane) * PR_HALF < len, there = x.pg >= 0 && x.pg < d.pages;
        absent = (absent & ~(3u << (2 * st))) | __ballot_sync(0xffffffffu, on && !there) << (2 * st);
        if (lane == 0) ptx::mbar_arrive_expect_tx(bar + st, (tile * 2 + 1) * PR_HALF < len ? STAGE : STAGE / 2);
        __syncwarp();
        if (on) {
            uint8_t* dst = ring + st * STAGE + lane * (PR_HALF * 128);
            const int token = x.half * PR_HALF, pg = there ? x.pg : -1;   // an absent page: outside the tensor, zeros
#pragma unroll
            for (int c = 0; c < NCH; ++c) ptx::tma_load_4d(dst + c * BOX, &tmK, bar + st, c * 64, h, token, pg);
#pragma unroll
            for (int c = 0; c < NCH; ++c) ptx::tma_load_4d(dst + STAGE / 2 + c * BOX, &tmV, bar + st, c * 64, h, token, pg);
        }
    };
#pragma unroll
    for (int i = 0; i < STAGES; ++i) request(first + i * stride, early[i], i);

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
    // Row 8 i + 2 c4 + e sees the keys before lim; all live rows those before `low`. Rows of no token see what there
    // is: they are zeroed at the end.
    const int low = len - (new_ - 1);
    int lim[NR][2];
#pragma unroll
    for (int i = 0; i < NR; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int t = (8 * i + 2 * c4 + e) / G;
            lim[i][e] = t < new_ ? low + t : len;
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
        const uint32_t st = it % STAGES;
        const int next = tile + STAGES * stride;
        ok = __all_sync(0xffffffffu, ptx::mbar_wait_bounded(bar + st, (it / STAGES) & 1, nullptr));
        if (!ok) break;
        const uint8_t* sk = ring + st * STAGE;
        const uint8_t* sv = sk + STAGE / 2;
        const int u0 = tile * PR_KEYS;
        // s[i][t]: keys 16 t + r8 (0, 1) and 16 t + 8 + r8 (2, 3), rows 8 i + 2 c4 + {0, 1}
        float s[NR][NT][4];
        {
            float sp[NR][NT][2][4] = {};   // even and odd k-steps: shorter chains of dependent products
#pragma unroll
            for (int c = 0; c < 2 * NCH; ++c) {
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    // 16-byte unit i of key u at i ^ (u % 8)
                    const uint8_t* at = sk + (c >> 1) * BOX + (t * 16 + r8) * 128 + (((2 * c4 + (c & 1)) ^ r8) << 4);
                    const uint4 k0 = *reinterpret_cast<const uint4*>(at), k1 = *reinterpret_cast<const uint4*>(at + 1024);
                    const uint32_t a0[4] = {k0.x, k1.x, k0.y, k1.y}, a1[4] = {k0.z, k1.z, k0.w, k1.w};
#pragma unroll
                    for (int i = 0; i < NR; ++i) {
                        mma_16816(sp[i][t][0], a0, q[i][c].x, q[i][c].y);
                        mma_16816(sp[i][t][1], a1, q[i][c].z, q[i][c].w);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < NR; ++i)
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        s[i][t][e] = __fmul_rn(sp[i][t][0][e] + sp[i][t][1][e], p.scale_log2);   // rounded like the maximum
        }
        const bool edge = u0 + PR_KEYS > low;   // some row does not see all of it
        if (edge) {
#pragma unroll
            for (int i = 0; i < NR; ++i)
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (u0 + t * 16 + (e >> 1) * 8 + r8 >= lim[i][e & 1]) s[i][t][e] = -INFINITY;
        }
        const uint32_t gone = absent >> (2 * st) & 3u;
        if (__builtin_expect(gone != 0, 0)) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
                if (gone >> t & 1)
#pragma unroll
                    for (int i = 0; i < NR; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e) s[i][t][e] = -INFINITY;
        }
        // A row's maximum is raised when a score exceeds it by more than PR_SLACK: one vote a tile, and weights of up to
        // 2^PR_SLACK, exactly as good in bf16.
        bool over = false;
        float top[NR][2];
#pragma unroll
        for (int i = 0; i < NR; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                top[i][e] = fmaxf(fmaxf(s[i][0][e], s[i][0][e + 2]), fmaxf(s[i][1][e], s[i][1][e + 2]));
                over = over || top[i][e] > m[i][e] + PR_SLACK;   // from -inf: any score
            }
        if (__any_sync(0xffffffffu, over)) {
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                float alpha[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float mx = fmaxf(m[i][e], top[i][e]);
#pragma unroll
                    for (int w = 4; w < 32; w *= 2) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
                    alpha[e] = mx > m[i][e] ? exp2_approx(m[i][e] - mx) : 1.f;
                    m[i][e] = mx;
                    l[i][e] *= alpha[e];
                }
#pragma unroll
                for (int j = 0; j < NCH * 4; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[i][j][e] *= alpha[e & 1];
            }
        }
        uint32_t pt[NR][NT][2];   // P^T: row 8 i + r8, keys 16 t + 2 c4 + {0, 1} and + 8
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const float base[2] = {m[i][0] == -INFINITY ? 0.f : m[i][0], m[i][1] == -INFINITY ? 0.f : m[i][1]};   // no scores so far: weights of zero
#pragma unroll
            for (int t = 0; t < NT; ++t) {
#pragma unroll
                for (int e = 0; e < 4; ++e) s[i][t][e] = exp2_approx(s[i][t][e] - base[e & 1]);
                pt[i][t][0] = transpose_8x8(pack_bf16x2(s[i][t][0], s[i][t][1]));
                pt[i][t][1] = transpose_8x8(pack_bf16x2(s[i][t][2], s[i][t][3]));
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) l[i][e] += (s[i][0][e] + s[i][0][e + 2]) + (s[i][1][e] + s[i][1][e + 2]);
        }
        // V rows of keys 2 c4, 2 c4 + 1, 2 c4 + 8, 2 c4 + 9 of 16, columns 8 r8 on
        auto key_of = [&](int t, int k) { return t * 16 + 2 * c4 + (k & 1) + 8 * (k >> 1); };
        auto values = [&](int t, int c, int k) {
            const int u = key_of(t, k);
            return *reinterpret_cast<const uint4*>(sv + c * BOX + u * 128 + ((r8 ^ (u & 7)) << 4));
        };
        auto pairs = [&](const uint32_t (&w)[4][4], int e, uint32_t (&a)[4]) {   // m-tile e
            a[0] = __byte_perm(w[0][e], w[1][e], 0x5410);
            a[1] = __byte_perm(w[0][e], w[1][e], 0x7632);
            a[2] = __byte_perm(w[2][e], w[3][e], 0x5410);
            a[3] = __byte_perm(w[2][e], w[3][e], 0x7632);
        };
        if (!edge) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int c = 0; c < NCH; ++c) {
                    uint32_t w[4][4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) *reinterpret_cast<uint4*>(w[k]) = values(t, c, k);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint32_t a[4];
                        pairs(w, e, a);
#pragma unroll
                        for (int i = 0; i < NR; ++i) mma_16816(o[i][c * 4 + e], a, pt[i][t][0], pt[i][t][1]);
                    }
                }
        } else {
#pragma unroll 1
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int c = 0; c < NCH; ++c) {
                    uint32_t w[4][4], p0[NR], p1[NR];
                    bool odd = false;
#pragma unroll
                    for (int i = 0; i < NR; ++i) {
                        p0[i] = t ? pt[i][1][0] : pt[i][0][0];
                        p1[i] = t ? pt[i][1][1] : pt[i][0][1];
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        *reinterpret_cast<uint4*>(w[k]) = values(t, c, k);
                        // past the length there may be anything, and 0 * NaN is NaN
                        if (u0 + key_of(t, k) >= len) w[k][0] = w[k][1] = w[k][2] = w[k][3] = 0u;
                        odd = odd || (u0 + key_of(t, k) >= low &&
                                      (not_finite(w[k][0]) || not_finite(w[k][1]) || not_finite(w[k][2]) || not_finite(w[k][3])));
                    }
                    if (!__any_sync(0xffffffffu, odd)) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            uint32_t a[4];
                            pairs(w, e, a);
#pragma unroll
                            for (int i = 0; i < NR; ++i) mma_16816(o[i][c * 4 + e], a, p0[i], p1[i]);
                        }
                        continue;
                    }
#pragma unroll 1
                    for (int tok = 0; tok < new_; ++tok) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            uint32_t x[4][4], a[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k) x[k][e] = u0 + key_of(t, k) < low + tok ? w[k][e] : 0u;
                            pairs(x, e, a);
#pragma unroll
                            for (int i = 0; i < NR; ++i) {
                                float one[4] = {0.f, 0.f, 0.f, 0.f};
                                mma_16816(one, a, p0[i], p1[i]);
#pragma unroll
                                for (int y = 0; y < 4; ++y)
                                    if ((8 * i + 2 * c4 + (y & 1)) / G == tok) o[i][c * 4 + e][y] += one[y];
                            }
                        }
                    }
                }
        }
        __syncwarp();   // the stage has been read
        request(next, ahead, st);
        ahead = look_up();
    }
    if (!ok) {
        if (lane == 0 && p.err) atomicOr(p.err, ERRBIT_TIMEOUT_ATTENTION);
        // copies in flight land before the CTA can exit
        for (uint32_t i = it; i < it + STAGES; ++i)
            if (first + (int)i * stride < tiles) ptx::mbar_wait_bounded(bar + i % STAGES, (i / STAGES) & 1, nullptr);
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
    if (p.parts.n) {   // the prefix's rows are there
        griddep_wait();
        griddep_launch_dependents();
    }

    // Four columns from col of row r, joined from own keys (x, weights' sum and maximum) and the prefix's parts, stored. Parts are
    // asked for four at a time: one by one, seven of them for 16 rows of 128 took 12 us.
    auto finish = [&](int r, int col, float (&x)[4], float sum, float mx) {
        const int t = r / G;
        const int64_t row = ((int64_t)b * Tq + t) * d.H + h * G + r % G;
        if (p.parts.n) {
            const float2* ml = static_cast<const float2*>(p.parts.ml) + row;
            const float* acc = static_cast<const float*>(p.parts.acc) + row * dh + col;
            for (int i = 0; i < p.parts.n; i += PR_PARTS) {
                float2 w[PR_PARTS];
                float4 v[PR_PARTS];
#pragma unroll
                for (int y = 0; y < PR_PARTS; ++y) {
                    const int64_t at = min(i + y, p.parts.n - 1) * p.parts.rows;
                    w[y] = __ldcg(ml + at);
                    v[y] = __ldcg(reinterpret_cast<const float4*>(acc + at * dh));
                }
                float top = mx;
#pragma unroll
                for (int y = 0; y < PR_PARTS; ++y) {
                    if (i + y >= p.parts.n) w[y] = make_float2(-INFINITY, 0.f);
                    top = fmaxf(top, w[y].x);
                }
                const float base = top == -INFINITY ? 0.f : top, f = exp2_approx(mx - base);
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] *= f;
                sum *= f;
                mx = top;
#pragma unroll
                for (int y = 0; y < PR_PARTS; ++y) {
                    if (w[y].y == 0.f) continue;   // no keys: its row is not there
                    const float g = exp2_approx(w[y].x - base);
                    x[0] = fmaf(g, v[y].x, x[0]);
                    x[1] = fmaf(g, v[y].y, x[1]);
                    x[2] = fmaf(g, v[y].z, x[2]);
                    x[3] = fmaf(g, v[y].w, x[3]);
                    sum = fmaf(g, w[y].y, sum);
                }
            }
        }
        const bool none = sum == 0.f || t >= new_;
        const float inv = 1.f / sum;
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = none ? 0.f : x[e] * inv;
        __nv_bfloat16* at = static_cast<__nv_bfloat16*>(d.o) + row * dh + col;
        if ((reinterpret_cast<uintptr_t>(at) & 7) == 0) {
            *reinterpret_cast<uint2*>(at) = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) at[e] = __float2bfloat16_rn(x[e]);
        }
    };
    // join the warps' rows, four columns per thread and step, every operand asked for at once
    for (int i = threadIdx.x * 4; i < R * dh; i += NW * 128) {
        const int r = i / dh;
        float mw[NW], mx = -INFINITY;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            mw[w] = sm[w * piece + R * dh + r];
            mx = fmaxf(mx, mw[w]);
        }
        const float base = mx == -INFINITY ? 0.f : mx;
        float acc[4] = {};
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const float f = exp2_approx(mw[w] - base);
            const float4 v = *reinterpret_cast<const float4*>(sm + w * piece + i);
            acc[0] = fmaf(f, v.x, acc[0]);
            acc[1] = fmaf(f, v.y, acc[1]);
            acc[2] = fmaf(f, v.z, acc[2]);
            acc[3] = fmaf(f, v.w, acc[3]);
            sum = fmaf(f, sm[w * piece + R * dh + R + r], sum);
        }
        if (Z == 1) {
            finish(r, i - r * dh, acc, sum, mx);
        } else {
            *reinterpret_cast<float4*>(jO + i) = make_float4(acc[0], acc[1], acc[2], acc[3]);
            if (i == r * dh) {
                jO[R * dh + r] = mx;
                jO[R * dh + R + r] = sum;
            }
        }
    }
    if (Z > 1) {
        ptx::cluster_sync();   // every CTA's joined rows are in place
        const uint32_t own = ptx::smem_addr(jO);
        for (int i = (z * NW * 32 + threadIdx.x) * 4; i < R * dh; i += Z * NW * 128) {
            const int r = i / dh;
            float mz[PR_MAXZ], lz[PR_MAXZ], oz[PR_MAXZ][4];
#pragma unroll
            for (int y = 0; y < PR_MAXZ; ++y) {
                const uint32_t at = ptx::mapa_shared(own, y < Z ? y : 0);
                mz[y] = ptx::ld_cluster_f32(at + (R * dh + r) * 4);
                lz[y] = ptx::ld_cluster_f32(at + (R * dh + R + r) * 4);
#pragma unroll
                for (int e = 0; e < 4; ++e) oz[y][e] = ptx::ld_cluster_f32(at + (i + e) * 4);
                if (y >= Z) mz[y] = -INFINITY;
            }
            float mx = -INFINITY;
#pragma unroll
            for (int y = 0; y < PR_MAXZ; ++y) mx = fmaxf(mx, mz[y]);
            const float base = mx == -INFINITY ? 0.f : mx;
            float acc[4] = {}, sum = 0.f;
#pragma unroll
            for (int y = 0; y < PR_MAXZ; ++y) {
                if (y >= Z) break;
                const float f = exp2_approx(mz[y] - base);
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[e] = fmaf(f, oz[y][e], acc[e]);
                sum = fmaf(f, lz[y], sum);
            }
            finish(r, i - r * dh, acc, sum, mx);
        }
        __syncwarp();
        ptx::cluster_sync();   // no CTA leaves while another reads its shared memory
    }
}

// Clusters of Z CTAs, an SM to each, that run at once: asked once, of the first device that calls and of the instance for width 128
// and eight rows, whose shared memory leaves room for one CTA to an SM. The others are given an SM to each CTA as well. Another
// device, or a part of one, may run fewer at once and be slower for it; the results do not depend on it but for their rounding.
int clusters_at_once(int Z) {
    static std::atomic<int> known[PR_MAXZ + 1];   // one more than that
    int n = known[Z].load(std::memory_order_relaxed);
    if (n) return n - 1;
    auto k = paged_rows_kernel<128, 1, 6, 2, 1>;
    constexpr int smem = 6 * 2 * PR_KEYS * 512 + 8 * 130 * 4 + 1024;   // as launch_rows asks for
    static std::atomic<uint64_t> attr{0};
    if (set_smem_limit_once(k, smem, attr) != cudaSuccess) return 0;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = (unsigned)Z;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)Z);
    cfg.blockDim = dim3(6 * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, k, &cfg) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    known[Z].store(n + 1, std::memory_order_relaxed);
    return n;
}

template <int DHT, int NR, int NW, int STAGES, int MINB>
cudaError_t launch_rows(const PagedRowsParams& p, cudaStream_t s) {
    constexpr int STAGE = PR_KEYS * (DHT / 64) * 256;
    auto k = paged_rows_kernel<DHT, NR, NW, STAGES, MINB>;
    static std::atomic<uint64_t> attr{0};
    constexpr int smem = NW * STAGES * STAGE + NR * 8 * (DHT + 2) * 4 + 1024;
    const cudaError_t e = set_smem_limit_once(k, smem, attr);
    if (e != cudaSuccess) return e;
    const PagedDesc& d = p.d;
    alignas(64) CUtensorMap mk, mv;
    if (!ct_map(&mk, d.k, d.ks, d.pages, d.page, d.Hkv, d.dh, 1, PR_HALF, CU_TENSOR_MAP_L2_PROMOTION_L2_256B) ||
        !ct_map(&mv, d.v, d.vs, d.pages, d.page, d.Hkv, d.dh, 1, PR_HALF, CU_TENSOR_MAP_L2_PROMOTION_L2_256B))
        return cudaErrorInvalidValue;
    const dim3 grid((unsigned)(d.B * d.Hkv * p.Z)), block(NW * 32);
    if (p.Z == 1) return launch_dependent(k, grid, block, smem, s, mk, mv, p);
    return launch_dependent_cluster(k, grid, block, p.Z, smem, s, mk, mv, p);
}

}  // namespace

bool paged_rows_supported(const PagedDesc& d) {
    if (d.dt != DT_BF16 || d.dh % 8 != 0 || d.dh > 128 || d.Tq * (d.H / d.Hkv) > PR_ROWS || d.page % PR_HALF != 0) return false;
    if (d.B > 0x7fffffff / 8 / d.Hkv) return false;
    if ((reinterpret_cast<uintptr_t>(d.q) & 15) || d.qs[0] % 8 || d.qs[1] % 8 || d.qs[2] % 8) return false;
    return ct_strides_ok(d.k, d.ks, d.page) && ct_strides_ok(d.v, d.vs, d.page) && ct_encode_fn() != nullptr;
}

cudaError_t launch_paged_rows(const PagedDesc& d, const PagedParts& prefix, const DeviceInfo& dev, cudaStream_t s) {
    // A warp takes 1.1 us for a tile, half of it the matrix instructions' own time, so what counts is to have many of them, each
    // with a tile at least, in one round of CTAs. Few key heads: six warps with an SM of their own, in clusters of as many CTAs as
    // still run at once for all heads (eight for 15 heads, six for 23, five for 28, four for 36: a cluster lies in one of the GPU's
    // SM groups). 16 heads of 128 over 8200 keys, us at 1 / 2 / 4 / 6 / 8 CTAs: 52 / 30 / 18.2 / 15.9 / 27; of 64 at 4 / 6
    // 12.5 / 10.9, three warps and clusters of eight 13.1. Parts joined by another kernel, on all SMs, were no faster.
    // Many: three warps, four CTAs to an SM for widths up to 64 (32 heads x 16, 577 keys: 10.2 us; with four warps, of which
    // three CTAs fit and the rest are a second round, 15.2), two for wider ones; clusters double while every warp has
    // two tiles, wide heads one.
    const int64_t heads = d.B * d.Hkv, sms = dev.num_sms, keys = d.table_pages * d.page;
    const bool narrow = d.dh <= 64, many = d.Tq * (d.H / d.Hkv) > 8;
    int Z = 1;
    if (heads <= sms / 2) {
        const int64_t fill = (keys + 6 * PR_KEYS - 1) / (6 * PR_KEYS);
        Z = (int)(fill < PR_MAXZ ? fill : PR_MAXZ);
        while (Z > 1 && heads > clusters_at_once(Z)) --Z;
        const PagedRowsParams p{d, prefix, (float)(d.scale * 1.4426950408889634), Z, dev.err_word};
        if (narrow) return many ? launch_rows<64, 2, 6, 2, 1>(p, s) : launch_rows<64, 1, 6, 2, 1>(p, s);
        return many ? launch_rows<128, 2, 6, 2, 1>(p, s) : launch_rows<128, 1, 6, 2, 1>(p, s);
    }
    while (Z < PR_MAXZ && heads * Z * 2 <= 2 * sms && keys > Z * 3 * PR_KEYS * (narrow ? 2 : 1)) Z *= 2;
    const PagedRowsParams p{d, prefix, (float)(d.scale * 1.4426950408889634), Z, dev.err_word};
    // Sequences of one tile to a warp, as behind a prefix, need no ring, and more CTAs sit on an SM: 32 sequences of up to 64 keys
    // behind 500, 16 heads of 128, 16.9 -> 12.3 us with two warps (three: 15.1); up to 70 keys and five tokens 20.5 -> 16.4 with three
    // (two: 18.0; sixteen rows then spill 200 bytes, but two CTAs to an SM take 20.9); 100 of up to 40, 8 heads of 64, 7.3 -> 4.2.
    if (keys <= 2 * PR_KEYS) {
        if (narrow) return many ? launch_rows<64, 2, 2, 1, 5>(p, s) : launch_rows<64, 1, 2, 1, 6>(p, s);
        return many ? launch_rows<128, 2, 2, 1, 4>(p, s) : launch_rows<128, 1, 2, 1, 5>(p, s);
    }
    if (keys <= 3 * PR_KEYS) {
        if (narrow) return many ? launch_rows<64, 2, 3, 1, 5>(p, s) : launch_rows<64, 1, 3, 1, 5>(p, s);
        return many ? launch_rows<128, 2, 3, 1, 3>(p, s) : launch_rows<128, 1, 3, 1, 4>(p, s);
    }
    if (narrow) return many ? launch_rows<64, 2, 3, 2, 3>(p, s) : launch_rows<64, 1, 3, 2, 4>(p, s);
    return many ? launch_rows<128, 2, 3, 2, 2>(p, s) : launch_rows<128, 1, 3, 2, 2>(p, s);
}

}  // namespace vit
