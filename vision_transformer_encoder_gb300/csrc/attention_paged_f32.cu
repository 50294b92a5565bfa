// attention_paged_f32.cu -- paged attention in fp32: the mathematics of attention_paged.cu for head widths up to 128 in steps
// of 4 and pages of a multiple of 8 tokens.
//
// Bound by reading keys and values once for every four rows. A warp takes up to four rows (NR) of one key head, of a sequence or for a
// prefix of all its group's, and 8 keys, which lie in one page, at
// a time: its lanes hold VEC columns each, so that a key is one coalesced load, and all 16 loads of a step are in flight
// together; those of the next step, into the same registers, are asked for when its products are done, its pages two steps ahead. The 8 NR products' halves are added across the lanes while they are
// handed out, so that each lane ends up with whole scores of its own: 31 exchanges for 32 scores. fp32 throughout, O in
// registers. The warps of a CTA take every fourth step of its part of the keys and join in shared memory; parts are
// joined as in attention_paged.cu. 8 sequences of up to 577 keys behind 197, 12 heads of 64: 10.9 us, two launches of latencies;
// 2 x 2048 queries of 12 heads of 64 over 2048 keys, bound by the CUDA cores: 991 us (13.0 TFLOP/s).
#include <cuda_runtime.h>

#include "common.cuh"
#include "kernels.h"
#include "launch.cuh"

namespace vit {
namespace {

constexpr int PF_WARPS = 4, PF_KEYS = 8;

struct PagedF32Params {
    PagedDesc d;
    PagedParts parts;                // n 0: rows are stored
    int prefix_parts, own_parts;
    int64_t prefix_blocks;           // CTAs of the prefixes, in front
    int prefix_rb, own_rb;           // blocks of rows of one key head
    float scale_log2;
};

template <int VEC> struct Cols {
    float v[VEC];
    __device__ __forceinline__ void load(const float* p, bool on) {
        if constexpr (VEC == 4) {
            const float4 x = on ? *reinterpret_cast<const float4*>(p) : make_float4(0.f, 0.f, 0.f, 0.f);
            v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
        } else {
            const float2 x = on ? *reinterpret_cast<const float2*>(p) : make_float2(0.f, 0.f);
            v[0] = x.x; v[1] = x.y;
        }
    }
};

// Sums of N values over the lanes, handed out: afterwards lane L holds those of N / 32 values (at least one), the
// bits of its number from 16 down choosing the upper or lower half in turn.
template <int N> __device__ __forceinline__ void hand_out(float (&x)[N], int lane) {
    int n = N;
#pragma unroll
    for (int w = 16; w > 0; w /= 2) {
        if (n > 1) {
            n /= 2;
            const bool up = lane & w;
#pragma unroll
            for (int i = 0; i < N / 2; ++i)
                if (i < n) {
                    const float keep = up ? x[i + n] : x[i], give = up ? x[i] : x[i + n];
                    x[i] = keep + __shfl_xor_sync(0xffffffffu, give, w);
                }
        } else {
            x[0] += __shfl_xor_sync(0xffffffffu, x[0], w);
        }
    }
}

// CTA i of the prefixes, or of the own keys. sO: a row of O for each warp and row, sml: its maximum and sum.
template <int VEC, int NR>
__device__ __forceinline__ void paged_f32_rows_of(const PagedF32Params& p, bool prefix, int i, float* sO, float* sml) {
    constexpr int N = PF_KEYS * NR;   // scores of a step: value key * NR + row
    // lanes that differ in these bits hold the same score; those of one row's keys differ in `across`
    constexpr int ROWBIT = NR == 1 ? 0 : NR == 2 ? 1 : 2;
    const PagedDesc& d = p.d;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, dh = (int)d.dh;
    const int G = (int)(d.H / d.Hkv), Tq = (int)d.Tq, S = (int)(d.B / d.groups);
    const int Z = prefix ? p.prefix_parts : p.own_parts, nrb = prefix ? p.prefix_rb : p.own_rb;
    const int z = i % Z;
    i /= Z;
    const int rb = i % nrb;
    i /= nrb;
    const int hk = i % (int)d.Hkv, at = i / (int)d.Hkv;   // key head; group or sequence
    const int64_t tokens = prefix ? (int64_t)S * Tq : Tq, first = at * tokens;
    const int32_t* table = prefix ? d.prefix_table + at * d.prefix_pages : d.table + at * d.table_pages;
    const int held = (int)((prefix ? d.prefix_pages : d.table_pages) * d.page), page = (int)d.page;
    const int len = min(max(load((prefix ? d.prefix_lens : d.kv_lens) + at), 0), held);
    const int col = lane * VEC;
    const bool on = col < dh;

    Cols<VEC> q[NR];
    int64_t row[NR];
    int lim[NR], most = 0, low = 0x7fffffff;   // low: keys before it all rows see that see any
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        const int64_t n = (int64_t)rb * NR + r, token = first + n / G, h = (int64_t)hk * G + n % G;
        const bool there = n < tokens * G;
        const int64_t b = there ? token / Tq : 0, t = there ? token - b * Tq : 0;
        const int64_t new_ = there ? (d.q_lens ? min(max((int64_t)load(d.q_lens + b), (int64_t)0), (int64_t)Tq) : Tq) : 0;
        row[r] = there ? token * d.H + h : -1;
        lim[r] = t < new_ ? (prefix ? len : max(0, (int)(len - (new_ - 1 - t)))) : 0;
        most = max(most, lim[r]);
        if (lim[r] > 0) low = min(low, lim[r]);
        q[r].load(static_cast<const float*>(d.q) + b * d.qs[0] + t * d.qs[1] + (there ? h : 0) * d.qs[2] + col, there && on);
    }
    const int steps = (most + PF_KEYS - 1) / PF_KEYS, per = (steps + Z - 1) / Z;
    const int s0 = min(steps, z * per), s1 = min(steps, s0 + per);

    float o[NR][VEC], m = -INFINITY, l = 0.f;   // maximum and sum of the row whose scores this lane holds
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int c = 0; c < VEC; ++c) o[r][c] = 0.f;
    // which score this lane ends up with: the upper bits of the lane number choose among the N in order
    constexpr int BITS = N == 8 ? 3 : N == 16 ? 4 : 5;
    const int mine = lane >> (5 - BITS), my_key = mine / NR, my_row = mine % NR;
    int my_lim = lim[0];
#pragma unroll
    for (int r = 1; r < NR; ++r)
        if (my_row == r) my_lim = lim[r];

    const float* kb = static_cast<const float*>(d.k) + hk * d.ks[2] + col;
    const float* vb = static_cast<const float*>(d.v) + hk * d.vs[2] + col;
    auto entry = [&](int s) -> int {
        const int pg = s < s1 ? load(table + s * PF_KEYS / page) : -1;
        return pg < d.pages ? pg : -1;
    };
    Cols<VEC> k[PF_KEYS], v[PF_KEYS];
    auto load = [&](int s, int pg) {
        const int u0 = s * PF_KEYS, slot = u0 % page;
        const float* kr = kb + pg * d.ks[0] + slot * d.ks[1];
        const float* vr = vb + pg * d.vs[0] + slot * d.vs[1];
#pragma unroll
        for (int u = 0; u < PF_KEYS; ++u) {
            const bool there = on && pg >= 0 && u0 + u < most;
            k[u].load(kr + u * d.ks[1], there);
            v[u].load(vr + u * d.vs[1], there);
        }
    };
    int pg = entry(s0 + warp), next = entry(s0 + warp + PF_WARPS);
    if (pg >= 0) load(s0 + warp, pg);
    for (int s = s0 + warp; s < s1; s += PF_WARPS) {
        const int after = entry(s + 2 * PF_WARPS);
        if (pg >= 0) {
            float x[N];
#pragma unroll
            for (int u = 0; u < PF_KEYS; ++u)
#pragma unroll
                for (int r = 0; r < NR; ++r) {
                    float a = 0.f;
#pragma unroll
                    for (int c = 0; c < VEC; ++c) a = fmaf(q[r].v[c], k[u].v[c], a);
                    x[u * NR + r] = a;
                }
            hand_out<N>(x, lane);
            // rounded here: the maximum and what it is taken off are the same numbers
            const float score = s * PF_KEYS + my_key < my_lim ? __fmul_rn(x[0], p.scale_log2) : -INFINITY;
            float mx = fmaxf(score, m);
#pragma unroll
            for (int w = 16; w >= (1 << (5 - BITS + ROWBIT)); w /= 2) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
            const float base = mx == -INFINITY ? 0.f : mx;   // only infinite scores so far: weights of zero
            const float w = exp2f(score - base), alpha = exp2f(m - base);
            l = l * alpha + w;   // of this lane's keys
            m = mx;
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                const float f = __shfl_sync(0xffffffffu, alpha, r << (5 - BITS));   // a lane of key 0 and this row
#pragma unroll
                for (int c = 0; c < VEC; ++c) o[r][c] *= f;
            }
            // A key that the row does not see adds nothing, whatever its value: asked once a step, key by key only where rows end
            // (2 x 2048 queries of 12 heads of 64 over 2048 keys: 1198 -> 991 us; of 128, 2 x 512 of 12 / 3 heads: 759 -> 636).
            if (NR == 1 || (s + 1) * PF_KEYS <= low) {
#pragma unroll
                for (int u = 0; u < PF_KEYS; ++u)
#pragma unroll
                    for (int r = 0; r < NR; ++r) {
                        const float f = __shfl_sync(0xffffffffu, w, (u * NR + r) << (5 - BITS));
#pragma unroll
                        for (int c = 0; c < VEC; ++c) o[r][c] = fmaf(f, v[u].v[c], o[r][c]);
                    }
            } else {
#pragma unroll
                for (int u = 0; u < PF_KEYS; ++u)
#pragma unroll
                    for (int r = 0; r < NR; ++r) {
                        const float f = __shfl_sync(0xffffffffu, w, (u * NR + r) << (5 - BITS));
#pragma unroll
                        for (int c = 0; c < VEC; ++c)
                            if (s * PF_KEYS + u < lim[r]) o[r][c] = fmaf(f, v[u].v[c], o[r][c]);
                    }
            }
        }
        pg = next;
        next = after;
        if (pg >= 0) load(s + PF_WARPS, pg);
    }
    // the sum over the lanes of a row's keys
#pragma unroll
    for (int w = 16; w >= (1 << (5 - BITS + ROWBIT)); w /= 2) l += __shfl_xor_sync(0xffffffffu, l, w);
    if (my_key == 0 && (lane & ((1 << (5 - BITS)) - 1)) == 0) {
        sml[2 * (warp * NR + my_row)] = m;
        sml[2 * (warp * NR + my_row) + 1] = l;
    }
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int c = 0; c < VEC; ++c) sO[(warp * NR + r) * 32 * VEC + col + c] = o[r][c];
    __syncthreads();
    // join the warps, a row to a warp in turn
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        if (r % PF_WARPS != warp) continue;
        int64_t to = row[0];
#pragma unroll
        for (int e = 1; e < NR; ++e)
            if (r == e) to = row[e];
        if (to < 0) continue;
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < PF_WARPS; ++w) top = fmaxf(top, sml[2 * (w * NR + r)]);
        const float base = top == -INFINITY ? 0.f : top;
        float acc[VEC] = {}, sum = 0.f;
#pragma unroll
        for (int w = 0; w < PF_WARPS; ++w) {
            const float f = exp2f(sml[2 * (w * NR + r)] - base);
            sum = fmaf(f, sml[2 * (w * NR + r) + 1], sum);
#pragma unroll
            for (int c = 0; c < VEC; ++c) acc[c] = fmaf(f, sO[(w * NR + r) * 32 * VEC + col + c], acc[c]);
        }
        float* dst;
        if (p.parts.n) {
            const int64_t part = prefix ? z : p.prefix_parts + z, place = part * p.parts.rows + to;
            if (lane == 0) static_cast<float2*>(p.parts.ml)[place] = make_float2(top, sum);
            dst = static_cast<float*>(p.parts.acc) + place * dh;
        } else {
            dst = static_cast<float*>(d.o) + to * dh;
#pragma unroll
            for (int c = 0; c < VEC; ++c) acc[c] = sum == 0.f ? 0.f : acc[c] / sum;
        }
        if (on)
#pragma unroll
            for (int c = 0; c < VEC; ++c) dst[col + c] = acc[c];
    }
}

// NR rows to a warp for own keys, NP for the prefixes, whose rows are those of all sequences of a group.
template <int VEC, int NR, int NP>
__global__ void __launch_bounds__(PF_WARPS * 32) paged_f32_kernel(const __grid_constant__ PagedF32Params p) {
    static_assert(NP >= NR, "a group has a sequence's rows at least");
    __shared__ float sO[PF_WARPS * NP * 32 * VEC], sml[PF_WARPS * NP * 2];
    griddep_wait();
    griddep_launch_dependents();
    const bool prefix = blockIdx.x < p.prefix_blocks;
    const int i = (int)(prefix ? blockIdx.x : blockIdx.x - p.prefix_blocks);
    if constexpr (NR == NP) {
        paged_f32_rows_of<VEC, NR>(p, prefix, i, sO, sml);
    } else {
        if (prefix) paged_f32_rows_of<VEC, NP>(p, true, i, sO, sml);
        else paged_f32_rows_of<VEC, NR>(p, false, i, sO, sml);
    }
}

template <int VEC> cudaError_t launch_f32(const PagedF32Params& p, int NR, int NP, int64_t blocks, cudaStream_t s) {
    const dim3 grid((unsigned)blocks), block(PF_WARPS * 32);
    if (NR == 4) return launch_dependent(paged_f32_kernel<VEC, 4, 4>, grid, block, 0, s, p);
    if (NR == 2)
        return NP == 2 ? launch_dependent(paged_f32_kernel<VEC, 2, 2>, grid, block, 0, s, p)
                       : launch_dependent(paged_f32_kernel<VEC, 2, 4>, grid, block, 0, s, p);
    if (NP == 1) return launch_dependent(paged_f32_kernel<VEC, 1, 1>, grid, block, 0, s, p);
    return NP == 2 ? launch_dependent(paged_f32_kernel<VEC, 1, 2>, grid, block, 0, s, p)
                   : launch_dependent(paged_f32_kernel<VEC, 1, 4>, grid, block, 0, s, p);
}

bool columns_fit(const void* p, const int64_t st[3], int64_t unit) {
    return reinterpret_cast<uintptr_t>(p) % (4 * unit) == 0 && st[0] % unit == 0 && st[1] % unit == 0 && st[2] % unit == 0;
}

}  // namespace

// Rows that share a key's load. A prefix's are those of all sequences of its group: 32 x 1 over 64 keys behind 4100, 12 heads of 64, 88
// us with one row, 47 with four; of 128, 164 -> 65. With few sequences of one row, four rows' registers cost the own keys
// more than their sharing gains: 8 x 1 over 577 keys behind 197, 11.9 us with four, 11.3 with two (one: 11.4).
int paged_f32_rows(const PagedDesc& d, bool own) {
    const int64_t one = d.Tq * (d.H / d.Hkv), R = (own ? 1 : d.B / d.groups) * one;
    return R == 1 ? 1 : R == 2 || (one == 1 && R <= 8) ? 2 : 4;
}

int64_t paged_f32_blocks(const PagedDesc& d, bool own) {
    const int64_t NR = paged_f32_rows(d, own), R = (own ? 1 : d.B / d.groups) * d.Tq * (d.H / d.Hkv);
    return (own ? d.B : d.groups) * d.Hkv * ((R + NR - 1) / NR);
}

bool paged_f32_supported(const PagedDesc& d) {
    if (d.dt != DT_F32 || d.dh % 4 != 0 || d.dh > 128 || d.page % PF_KEYS != 0) return false;
    const int64_t unit = d.dh <= 64 ? 2 : 4;
    // CTAs: rows of a group's sequences and key head, 32 parts, own keys and prefix
    if (d.Tq > 0x7fffffff / 64 / d.H || d.B > 0x7fffffff / 64 / (d.H * d.Tq)) return false;
    return columns_fit(d.q, d.qs, unit) && columns_fit(d.k, d.ks, unit) && columns_fit(d.v, d.vs, unit);
}

cudaError_t launch_paged_f32(const PagedDesc& d, const PagedPlan& plan, const PagedParts& parts, cudaStream_t s) {
    const int NR = paged_f32_rows(d, true), NP = plan.prefix_parts ? paged_f32_rows(d, false) : NR;
    const int64_t G = d.H / d.Hkv;
    PagedF32Params p{};
    p.d = d;
    p.parts = parts;
    p.prefix_parts = plan.prefix_parts;
    p.own_parts = plan.own_parts;
    p.own_rb = (int)((d.Tq * G + NR - 1) / NR);
    p.prefix_rb = (int)((d.B / d.groups * d.Tq * G + NP - 1) / NP);
    p.prefix_blocks = plan.prefix_parts ? paged_f32_blocks(d, false) * plan.prefix_parts : 0;
    p.scale_log2 = (float)(d.scale * 1.4426950408889634);
    const int64_t blocks = p.prefix_blocks + paged_f32_blocks(d, true) * plan.own_parts;
    return d.dh <= 64 ? launch_f32<2>(p, NR, NP, blocks, s) : launch_f32<4>(p, NR, NP, blocks, s);
}

}  // namespace vit
