// attention_paged.cu -- causal attention of a batch's newest tokens over keys and values in pages, behind a prefix that
// the sequences of a group share:
//   o[b, t, h] = sum_u softmax_u(scale q[b, t, h] . k[u, h / G]) v[u, h / G]
// over the prefix of b's group and b's own keys u < lim(b, t) = kv_len - (q_len - 1 - t). G = H / Hkv query heads share a
// key head.
//
// The prefix of a group is worked off for the rows of all its sequences in turn, apart from their own keys, as many rows to a read of
// a key as a kernel's tile has: up to 256 on tensor cores, four in fp32, 4 or 16 in the generic kernel. Either can be
// cut along the keys too. Such a part leaves an unnormalised row, its maximum and its sum of weights in a workspace
// (PagedParts), and what runs last joins them, always in the same order. Without a prefix and with one part, rows are
// stored directly.
//
// Generic kernel: any type, head width up to 512, page size, stride and alignment. A CTA takes up to RT rows of one key
// head and 32 keys at a time: keys to shared memory, scores, the running maximum and sum, values over the keys, sums in
// registers. Bound by the reads of shared memory for its products: 2 x 512 queries of 12 heads of 64 over 512 keys in pages of 20,
// fp32, 209 us; 252 us in bf16 with heads of 72. A prefix has a sequence's RT too: with 16 rows of a group where a sequence has
// one, 32 x 1 behind 4100 keys 190 -> 125 us, but 8 x 1 over 577 behind 197 52 -> 72 and 8 x 1 of fp64 and heads of 512 397 -> 1490.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "launch.cuh"

namespace vit {
namespace {

constexpr int PG_THREADS = 128, PG_KEYS = 32, PG_PARTS = 4;

__device__ __forceinline__ float exp2_of(float x) { return exp2f(x); }
__device__ __forceinline__ double exp2_of(double x) { return exp2(x); }
__device__ __forceinline__ float mul_rn(float a, float b) { return __fmul_rn(a, b); }
__device__ __forceinline__ double mul_rn(double a, double b) { return __dmul_rn(a, b); }
__device__ __forceinline__ float max_of(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ double max_of(double a, double b) { return fmax(a, b); }

struct GenericParams {
    PagedDesc d;
    PagedParts parts;
    int prefix_parts, own_parts;
    int64_t prefix_blocks, blocks;   // CTAs' worth of work: the prefixes', and all
    int64_t prefix_rb, own_rb;       // blocks of rows of one key head
    double scale_log2;
};

template <typename T, typename A, int RT, int DHT>
__global__ void __launch_bounds__(PG_THREADS) paged_generic_kernel(const __grid_constant__ GenericParams p) {
    constexpr int TPR = PG_THREADS / RT, KPT = PG_KEYS / TPR;               // scores: threads of a row, keys of a thread
    constexpr int NC = DHT < 128 ? DHT : 128, NJ = DHT / NC, RPT = RT * NC / PG_THREADS;   // values: columns, rows of a thread
    static_assert(TPR <= 32 && RPT >= 1, "threads");
    extern __shared__ __align__(16) uint8_t smem[];
    const PagedDesc& d = p.d;
    const int dh = (int)d.dh, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    A* sq = reinterpret_cast<A*>(smem);        // RT x dh
    A* skv = sq + RT * dh;                     // 32 x (dh + 1): keys, then values
    __shared__ A sp[RT][PG_KEYS], salpha[RT], sl[RT];
    __shared__ int64_t srow[RT];
    __shared__ int slim[RT], spages[2][PG_KEYS];
    griddep_wait();
    griddep_launch_dependents();
    const int G = (int)(d.H / d.Hkv);
    const int64_t S = d.B / d.groups;
    const A sl2 = (A)p.scale_log2;
    for (int64_t block = blockIdx.x; block < p.blocks; block += gridDim.x) {
        const bool prefix = block < p.prefix_blocks;
        int64_t i = prefix ? block : block - p.prefix_blocks;
        const int Z = prefix ? p.prefix_parts : p.own_parts;
        const int z = (int)(i % Z);
        i /= Z;
        const int64_t nrb = prefix ? p.prefix_rb : p.own_rb, rb = i % nrb;
        i /= nrb;
        const int64_t hk = i % d.Hkv, at = i / d.Hkv;   // key head; group or sequence
        const int64_t tokens = prefix ? S * d.Tq : d.Tq, first = at * tokens;
        const int32_t* table = prefix ? d.prefix_table + at * d.prefix_pages : d.table + at * d.table_pages;
        const int64_t held = (prefix ? d.prefix_pages : d.table_pages) * d.page;
        const int len = (int)min((int64_t)max(load((prefix ? d.prefix_lens : d.kv_lens) + at), 0), held);
        __syncthreads();   // the last block's rows have been stored
        for (int r = warp; r < RT; r += PG_THREADS / 32) {
            const int64_t n = rb * RT + r, token = first + n / G, h = hk * G + n % G;
            const bool there = n < tokens * G;
            const int64_t b = there ? token / d.Tq : 0, t = token - b * d.Tq;
            const int64_t qlen = there ? (d.q_lens ? min((int64_t)max(load(d.q_lens + b), 0), d.Tq) : d.Tq) : 0;
            if (lane == 0) {
                srow[r] = there ? token * d.H + h : -1;
                slim[r] = there && t < qlen ? (prefix ? len : (int)max((int64_t)0, len - (qlen - 1 - t))) : 0;
            }
            const T* q = static_cast<const T*>(d.q) + b * d.qs[0] + t * d.qs[1] + h * d.qs[2];
            for (int c = lane; c < dh; c += 32) sq[r * dh + c] = there ? to_acc<A>(q[c]) : (A)0;
        }
        __syncthreads();
        int most = 0;
        for (int r = 0; r < RT; ++r) most = max(most, slim[r]);
        const int all = (most + PG_KEYS - 1) / PG_KEYS, per = (all + Z - 1) / Z;
        const int t0 = min(all, z * per), t1 = min(all, t0 + per);

        const int r = tid / TPR, k0 = tid % TPR, lim = slim[r];
        A m = -INFINITY, l = 0;
        A acc[RPT][NJ];
#pragma unroll
        for (int e = 0; e < RPT; ++e)
#pragma unroll
            for (int j = 0; j < NJ; ++j) acc[e][j] = 0;
        const int col = tid % NC, r0 = tid / NC * RPT;
        for (int tile = t0; tile < t1; ++tile) {
            const int u0 = tile * PG_KEYS, n = min(PG_KEYS, most - u0);
            int* spage = spages[tile & 1];   // the last tile's may still be read
            if (tid < PG_KEYS) {
                int pg = tid < n ? load(table + (int64_t)(u0 + tid) / d.page) : -1;
                spage[tid] = pg >= 0 && pg < d.pages ? pg : -1;
            }
            // this tile of a pool to shared memory, AT keys of a warp's in flight
            auto fetch = [&](const void* pool, const int64_t(&st)[3]) {
                constexpr int COLS = DHT / 32, AT = DHT <= 128 ? 4 : 1, WARPS = PG_THREADS / 32;
                const T* base = static_cast<const T*>(pool) + hk * st[2];
                for (int u1 = warp; u1 < n; u1 += AT * WARPS) {
                    T x[AT][COLS];
#pragma unroll
                    for (int y = 0; y < AT; ++y) {
                        const int u = u1 + y * WARPS;
                        if (u >= n || spage[u] < 0) continue;
                        const T* row = base + spage[u] * st[0] + (int64_t)(u0 + u) % d.page * st[1];
#pragma unroll
                        for (int c = 0; c < COLS; ++c)
                            if (lane + 32 * c < dh) x[y][c] = row[lane + 32 * c];
                    }
#pragma unroll
                    for (int y = 0; y < AT; ++y) {
                        const int u = u1 + y * WARPS;
                        if (u >= n || spage[u] < 0) continue;
#pragma unroll
                        for (int c = 0; c < COLS; ++c)
                            if (lane + 32 * c < dh) skv[u * (dh + 1) + lane + 32 * c] = to_acc<A>(x[y][c]);
                    }
                }
            };
            __syncthreads();   // the last tile's values have been read
            fetch(d.k, d.ks);
            __syncthreads();
            A x[KPT], mx = m;
#pragma unroll
            for (int j = 0; j < KPT; ++j) x[j] = 0;
            for (int c = 0; c < dh; ++c) {
                const A qc = sq[r * dh + c];
#pragma unroll
                for (int j = 0; j < KPT; ++j) x[j] = qc * skv[(k0 + TPR * j) * (dh + 1) + c] + x[j];
            }
#pragma unroll
            for (int j = 0; j < KPT; ++j) {
                const int u = k0 + TPR * j;
                // rounded here: the maximum and what it is taken off are the same numbers
                x[j] = u0 + u < lim && spage[u] >= 0 ? mul_rn(x[j], sl2) : (A)-INFINITY;
                mx = max_of(mx, x[j]);   // a NaN score is not kept here, but its weight below is NaN
            }
#pragma unroll
            for (int w = TPR / 2; w > 0; w /= 2) mx = max_of(mx, __shfl_xor_sync(0xffffffffu, mx, w));
            const A base = mx == -INFINITY ? (A)0 : mx;   // only infinite scores so far: weights of zero
            const A alpha = exp2_of(m - base);
            A sum = 0;
#pragma unroll
            for (int j = 0; j < KPT; ++j) {
                const A w = exp2_of(x[j] - base);
                sp[r][k0 + TPR * j] = w;
                sum += w;
            }
#pragma unroll
            for (int w = TPR / 2; w > 0; w /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, w);
            l = l * alpha + sum;
            m = mx;
            if (k0 == 0) salpha[r] = alpha;
            __syncthreads();   // scores made, weights there: values over the keys
            fetch(d.v, d.vs);
            __syncthreads();
#pragma unroll
            for (int e = 0; e < RPT; ++e)
#pragma unroll
                for (int j = 0; j < NJ; ++j) acc[e][j] *= salpha[r0 + e];
            for (int u = 0; u < n; ++u) {
                if (spage[u] < 0) continue;
                A v[NJ];
#pragma unroll
                for (int j = 0; j < NJ; ++j) v[j] = col + NC * j < dh ? skv[u * (dh + 1) + col + NC * j] : (A)0;
#pragma unroll
                for (int e = 0; e < RPT; ++e) {
                    // a key that the row does not see adds nothing, whatever its value
                    const bool sees = u0 + u < slim[r0 + e];
#pragma unroll
                    for (int j = 0; j < NJ; ++j) acc[e][j] += sees ? sp[r0 + e][u] * v[j] : (A)0;
                }
            }
        }
        if (k0 == 0) {
            sl[r] = l;
            if (p.parts.n && srow[r] >= 0) {
                const int64_t part = prefix ? z : p.prefix_parts + z;
                A* ml = static_cast<A*>(p.parts.ml) + 2 * (part * p.parts.rows + srow[r]);
                ml[0] = m;
                ml[1] = l;
            }
        }
        __syncthreads();
#pragma unroll
        for (int e = 0; e < RPT; ++e) {
            const int64_t row = srow[r0 + e];
            if (row < 0) continue;
            const A sum = sl[r0 + e];
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                const int c = col + NC * j;
                if (c >= dh) continue;
                if (p.parts.n) {
                    const int64_t part = prefix ? z : p.prefix_parts + z;
                    static_cast<A*>(p.parts.acc)[(part * p.parts.rows + row) * dh + c] = acc[e][j];
                } else {
                    static_cast<T*>(d.o)[row * dh + c] = from_acc<T>(sum == (A)0 ? (A)0 : acc[e][j] / sum);
                }
            }
        }
    }
}

// Joins the parts of rows, V columns per thread.
template <typename T, typename A, int V>
__global__ void __launch_bounds__(256) paged_join_kernel(PagedParts parts, int dh, T* o) {
    griddep_wait();
    griddep_launch_dependents();
    const int64_t per = dh / V, total = parts.rows * per;
    const A* ml = static_cast<const A*>(parts.ml);
    const A* in = static_cast<const A*>(parts.acc);
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t row = i / per, c = i % per * V;
        A acc[V] = {}, sum = 0, mx = -INFINITY;
        for (int q = 0; q < parts.n; q += PG_PARTS) {   // parts asked for together
            A m[PG_PARTS], l[PG_PARTS], x[PG_PARTS][V];
#pragma unroll
            for (int y = 0; y < PG_PARTS; ++y) {
                const int64_t at = min(q + y, parts.n - 1) * parts.rows + row;
                m[y] = ml[2 * at];
                l[y] = ml[2 * at + 1];
                if constexpr (V == 4 && sizeof(A) == 4) {
                    const float4 z = *reinterpret_cast<const float4*>(in + at * dh + c);
                    x[y][0] = z.x;
                    x[y][1] = z.y;
                    x[y][2] = z.z;
                    x[y][3] = z.w;
                } else {
#pragma unroll
                    for (int e = 0; e < V; ++e) x[y][e] = in[at * dh + c + e];
                }
            }
            A top = mx;
#pragma unroll
            for (int y = 0; y < PG_PARTS; ++y) {
                if (q + y >= parts.n) {
                    m[y] = -INFINITY;
                    l[y] = 0;
                }
                top = max_of(top, m[y]);
            }
            const A base = top == -INFINITY ? (A)0 : top, f = exp2_of(mx - base);
#pragma unroll
            for (int e = 0; e < V; ++e) acc[e] *= f;
            sum *= f;
            mx = top;
#pragma unroll
            for (int y = 0; y < PG_PARTS; ++y) {
                if (l[y] == (A)0) continue;   // no keys: its row is not there
                const A g = exp2_of(m[y] - base);
                sum += g * l[y];
#pragma unroll
                for (int e = 0; e < V; ++e) acc[e] += g * x[y][e];
            }
        }
#pragma unroll
        for (int e = 0; e < V; ++e) acc[e] = sum == (A)0 ? (A)0 : acc[e] / sum;
        if constexpr (V == 4 && sizeof(T) == 2) {
            *reinterpret_cast<uint2*>(o + row * dh + c) = make_uint2(pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]));
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e) o[row * dh + c + e] = from_acc<T>(acc[e]);
        }
    }
}

template <typename T, typename A> cudaError_t join(const PagedParts& parts, const PagedDesc& d, const DeviceInfo& dev, cudaStream_t s) {
    const bool four = d.dh % 4 == 0 && reinterpret_cast<uintptr_t>(d.o) % (4 * sizeof(T)) == 0;
    const int64_t want = (parts.rows * (four ? d.dh / 4 : d.dh) + 255) / 256, most = 16 * (int64_t)dev.num_sms;
    const dim3 grid((unsigned)(want < most ? want : most));
    T* o = static_cast<T*>(d.o);
    return four ? launch_dependent(paged_join_kernel<T, A, 4>, grid, dim3(256), 0, s, parts, (int)d.dh, o)
                : launch_dependent(paged_join_kernel<T, A, 1>, grid, dim3(256), 0, s, parts, (int)d.dh, o);
}

template <typename T, typename A, int RT, int DHT>
cudaError_t run_generic(const GenericParams& p, const DeviceInfo& dev, cudaStream_t s) {
    auto k = paged_generic_kernel<T, A, RT, DHT>;
    const int smem = (int)((RT * p.d.dh + PG_KEYS * (p.d.dh + 1)) * sizeof(A));
    static std::atomic<uint64_t> attr{0};
    const cudaError_t e = set_smem_limit_once(k, (int)((RT * DHT + PG_KEYS * (DHT + 1)) * sizeof(A)), attr);
    if (e != cudaSuccess) return e;
    const int64_t most = 32 * (int64_t)dev.num_sms;
    return launch_dependent(k, dim3((unsigned)(p.blocks < most ? p.blocks : most)), dim3(PG_THREADS), (size_t)smem, s, p);
}

template <typename T, typename A, int RT> cudaError_t run_generic_of(const GenericParams& p, const DeviceInfo& dev, cudaStream_t s) {
    if (p.d.dh <= 64) return run_generic<T, A, RT, 64>(p, dev, s);
    if (p.d.dh <= 128) return run_generic<T, A, RT, 128>(p, dev, s);
    if (p.d.dh <= 256) return run_generic<T, A, RT, 256>(p, dev, s);
    return run_generic<T, A, RT, 512>(p, dev, s);
}

// Rows to a CTA: a few where a key head serves few.
int generic_rows(const PagedDesc& d) { return d.Tq * (d.H / d.Hkv) <= 4 ? 4 : 16; }

template <typename T, typename A>
cudaError_t generic(const PagedDesc& d, const PagedPlan& plan, const PagedParts& parts, const DeviceInfo& dev, cudaStream_t s, bool own = true) {
    const int RT = generic_rows(d);
    const int64_t G = d.H / d.Hkv, tokens = d.B / d.groups * d.Tq;
    GenericParams p{};
    p.d = d;
    p.parts = parts;
    p.prefix_parts = plan.prefix_parts;
    p.own_parts = plan.own_parts;
    p.own_rb = (d.Tq * G + RT - 1) / RT;
    p.prefix_rb = (tokens * G + RT - 1) / RT;
    p.prefix_blocks = d.groups * d.Hkv * p.prefix_rb * plan.prefix_parts;
    p.blocks = p.prefix_blocks + (own ? d.B * d.Hkv * p.own_rb * plan.own_parts : 0);
    p.scale_log2 = d.scale * 1.4426950408889634;
    return RT == 4 ? run_generic_of<T, A, 4>(p, dev, s) : run_generic_of<T, A, 16>(p, dev, s);
}

}  // namespace

PagedPlan plan_paged(const PagedDesc& d, const DeviceInfo& dev) {
    PagedPlan plan{};
    const int64_t keys = d.table_pages * d.page, before = d.prefix_pages * d.page, sms = dev.num_sms;
    plan.form = paged_rows_supported(d) ? PAGED_ROWS : paged_tc_supported(d, true) ? PAGED_TC : paged_f32_supported(d) ? PAGED_F32 : PAGED_GENERIC;
    plan.prefix_tc = (plan.form == PAGED_ROWS || plan.form == PAGED_TC) && d.prefix_table && paged_tc_supported(d, false);
    // `blocks` CTAs over n keys, cut into parts of `least` keys or more until there are `want` of them
    auto cut = [](int64_t want, int64_t blocks, int64_t n, int64_t least) {
        int64_t z = want / blocks;
        z = z < n / least ? z : n / least;
        return (int)(z < 1 ? 1 : z > 32 ? 32 : z);
    };
    // The same on tensor cores, a CTA to an SM. Where `blocks` leave SMs idle in the only round, or the last, smaller items can
    // fill more rounds better: an item takes 4 us and 1.5 for each tile of 128 keys, its part of `rows` rows a write and a read.
    auto cut_tc = [&](int64_t blocks, int64_t n, int64_t least, int64_t rows) {
        const int first = cut(sms, blocks, n, least);
        auto us = [&](int64_t z) {
            return (double)((blocks * z + sms - 1) / sms) * (4.0 + 1.5 * (double)((n + 128 * z - 1) / (128 * z))) +
                   (double)z * (0.3 + (double)(rows * d.dh) * 8.0 / 6.8e6);
        };
        int best = first;
        double lowest = 0.9 * us(first);
        for (int z = first + 1; z <= 32 && n >= z * least; ++z) {
            const double t = us(z);
            if (t >= lowest) continue;
            best = z;
            lowest = t;
        }
        return best;
    };
    const int RT = generic_rows(d);
    const int64_t G = d.H / d.Hkv, own_rb = (d.Tq * G + RT - 1) / RT, prefix_rb = (d.B / d.groups * d.Tq * G + RT - 1) / RT;
    if (plan.form == PAGED_TC) {
        // A CTA to an SM. Parts cost a write and a read of fp32 rows: items that fill the SMs once are not cut (2 x 1025
        // queries over 4100 keys, 120 items: 56 us, in two parts 65, in three 58).
        const bool apart = plan.prefix_tc && paged_tc_apart(d);
        if (apart) plan.prefix_parts = cut_tc(paged_tc_items(d, false), before, 512, d.B * d.Tq * d.H);
        plan.own_parts = cut_tc(paged_tc_items(d, true), keys + (apart ? 0 : before), 512, d.B * d.Tq * d.H);
        const int least = (int)((keys + (apart ? 0 : before) + PAGED_TC_PART - 1) / PAGED_TC_PART);
        plan.own_parts = plan.own_parts < least ? least : plan.own_parts;
        plan.partial = plan.prefix_parts + plan.own_parts > 1;
    } else if (plan.form == PAGED_F32) {
        // CTAs of four warps, as many as sit on the SMs at once (three to six to an SM by the registers of own keys' rows or, where they
        // are more, the prefix's), dealt out to own keys and prefix
        // by what there is to read (in turn, each for all SMs, 6 x 2 tokens of 12 / 3 heads of 96 over 300 keys behind 800 took 20.8 us
        // instead of 14.9); parts of three or four steps to each warp at least (two: 16.1)
        const int one = paged_f32_rows(d, true), rows = d.prefix_table ? paged_f32_rows(d, false) : one;
        const int64_t ctas = sms * (d.dh > 64 ? (rows == 4 ? 3 : 4) : rows == 1 ? 6 : rows == 2 && one == 1 ? 5 : 4);
        const int64_t least = one == 1 ? 96 : 128;
        const int64_t own = paged_f32_blocks(d, true), ahead = d.prefix_table ? paged_f32_blocks(d, false) : 0;
        int64_t per = (own * keys + ahead * before + ctas - 1) / ctas;
        per = per < least ? least : per;
        auto parts = [&](int64_t n) { return (int)(n / per < 1 ? 1 : n / per > 32 ? 32 : n / per); };
        plan.own_parts = parts(keys);
        if (ahead) plan.prefix_parts = parts(before);
        plan.partial = plan.prefix_parts + plan.own_parts > 1;
    } else {
        // the prefix of few queries: two key tiles to a part at least, one for each softmax group (32 x 16 heads behind
        // 1025 keys: 10.5 us, with four 11.9, with one 12.2)
        if (d.prefix_table)
            plan.prefix_parts = plan.prefix_tc ? cut_tc(paged_tc_items(d, false), before, 256, d.B * d.Tq * d.H)
                                               : cut(8 * sms, d.groups * d.Hkv * prefix_rb, before, 128);
        // CTAs of four warps, some eight of them to an SM
        if (plan.form == PAGED_GENERIC) plan.own_parts = cut(8 * sms, d.B * d.Hkv * own_rb, keys, 128);
        plan.partial = plan.prefix_parts > 0 || plan.own_parts > 1;
    }
    plan.launches = plan.partial ? 2 : 1;
    if (plan.partial)
        plan.workspace = (size_t)(plan.prefix_parts + plan.own_parts) * (size_t)(d.B * d.Tq * d.H) * (size_t)(d.dh + 2) *
                         (d.dt == DT_F64 ? 8 : 4);
    return plan;
}

int paged_rows_at_once(const PagedDesc& d, const PagedPlan& plan, bool own) {
    const int64_t R = d.Tq * (d.H / d.Hkv);   // of a sequence; apart from the own keys, a prefix's are those of its group
    const int64_t rows = own || (plan.form == PAGED_TC && !plan.prefix_parts) ? R : d.B / d.groups * R;
    int64_t tile;
    if (plan.form == PAGED_F32) tile = paged_f32_rows(d, own);
    else if (plan.form == PAGED_TC || (!own && plan.prefix_tc)) tile = paged_tc_rows(d);
    else if (plan.form == PAGED_ROWS && own) tile = R;
    else tile = generic_rows(d);
    return (int)(tile < rows ? tile : rows);
}

cudaError_t launch_paged_attention(const PagedDesc& d, const PagedPlan& plan, void* workspace, const DeviceInfo& dev,
                                   cudaStream_t s) {
    PagedParts parts{};
    if (plan.partial) {
        parts.n = plan.prefix_parts + plan.own_parts;
        parts.rows = d.B * d.Tq * d.H;
        parts.acc = workspace;
        parts.ml = static_cast<uint8_t*>(workspace) + (size_t)parts.n * parts.rows * d.dh * (d.dt == DT_F64 ? 8 : 4);
    }
    cudaError_t e;
    if (plan.form == PAGED_ROWS) {
        if (plan.prefix_parts) {
            e = plan.prefix_tc ? launch_paged_tc(d, plan, parts, false, dev, s) : generic<__nv_bfloat16, float>(d, plan, parts, dev, s, false);
            if (e != cudaSuccess) return e;
        }
        return launch_paged_rows(d, parts, dev, s);
    }
    if (plan.form == PAGED_F32) e = launch_paged_f32(d, plan, parts, s);
    else if (plan.form == PAGED_TC) e = launch_paged_tc(d, plan, parts, true, dev, s);
    else if (d.dt == DT_F64) e = generic<double, double>(d, plan, parts, dev, s);
    else if (d.dt == DT_F32) e = generic<float, float>(d, plan, parts, dev, s);
    else e = generic<__nv_bfloat16, float>(d, plan, parts, dev, s);
    if (e != cudaSuccess || !plan.partial) return e;
    if (d.dt == DT_F64) return join<double, double>(parts, d, dev, s);
    if (d.dt == DT_F32) return join<float, float>(parts, d, dev, s);
    return join<__nv_bfloat16, float>(parts, d, dev, s);
}

}  // namespace vit
