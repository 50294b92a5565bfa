// rotary.cu -- rotary positions, and appending keys and values to a paged cache on the way.
//   pair i = (u, v) at position p -> scale (u cos a - v sin a, u sin a + v cos a),   a = p f_i
// One kernel turns the heads of the queries into their output and those of the keys into their pages, and copies
// the values into theirs; without keys it is the plain rotation.
//
// The angle: |f_i| / 2 pi as a 64-bit fraction of a turn with the sign put back, once per block and pair (fp64, of which the GPU
// has little). A position times that, modulo 2^64, is the fraction of a turn of p f_i: the modulo is exact, so that there is no
// range reduction, and what is off is p |f_i| 2^-52 for the rounding of f_i / 2 pi and 2 pi p 2^-65 for the fraction's (at
// position 10^6 and f 1, 2.2e-10 in all). That is below what fp32 and bf16 keep; for fp64 f_i / 2 pi is kept in two words, 128 bits of a turn
// (p |f_i| 2^-104; 2 x 8200 tokens of 12 heads of 64: 88 us, with 64 bits 84). Sine and cosine are the hardware's on [-pi, pi] for bf16 (off by 2^-20, where a result is rounded at 2^-9),
// sincospi for fp32 and fp64.
//
// Bound by reading and writing each head once. A block takes a few tokens: it makes their sines and cosines once, in shared
// memory. A thread has one 16-byte unit (both halves of its pairs where they lie apart) of one head and walks over the tokens,
// RO_AHEAD in flight: what depends on the head stays in registers, and a unit costs little more than its load, products and
// store. With few tokens the heads go to blocks of their own.
//
// 2 x 8200 tokens of 12 heads of 64 in fp32: 19.4 us (5.2 TB/s); 4 x 2048 tokens of 16 + 2 + 2 heads of 128 turned and
// appended: 17.3 us (4.6 TB/s). Sines of a thread's own, which then walked over a token's heads: 22.9 and 22.0. Heads and
// tokens in turn, with 105 instructions to a unit: 21.7 and 18.3.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "launch.cuh"

namespace vit {
namespace {

constexpr int RO_THREADS = 256, RO_MAXPAIRS = 256, RO_TOKENS = 32, RO_SINES = 1024, RO_MOST = 512, RO_AHEAD = 4;

// f / 2 pi as a fraction of a turn: in units of 2^-64, and for fp64 of 2^-128.
template <typename A> using TurnOf = typename std::conditional<std::is_same<A, double>::value, unsigned __int128, uint64_t>::type;

template <typename U> __device__ __forceinline__ U turn_of(double f) {
    // of the magnitude: a small negative number's fraction, next to 1, would keep 53 bits behind the point and no more
    const double a = fabs(f), t = a * 0.15915494309189535, r = t - floor(t);
    U turn;
    if constexpr (sizeof(U) == 8) {
        turn = __double2ull_rn(r * 18446744073709551616.0);
    } else {
        // t's rest: of the product, and of 1 / 2 pi behind its first 53 bits
        double low = fma(a, 0.15915494309189535, -t) + a * -9.839338337591243e-18;
        low -= rint(low);
        const double high = r * 0x1p64, units = low * 0x1p64, whole = floor(high), down = floor(units);
        turn = ((U)__double2ull_rz(whole) << 64) + __double2ull_rz((high - whole) * 0x1p64);
        turn += ((U)(uint64_t)__double2ll_rz(down) << 64) + __double2ull_rz((units - down) * 0x1p64);
    }
    return f < 0 ? (U)0 - turn : turn;
}

// `turn` of 2^-64 or 2^-128 in half turns of [-1, 1)
__device__ __forceinline__ double half_turns(uint64_t turn) { return (double)(int64_t)turn * 0x1p-63; }
__device__ __forceinline__ double half_turns(unsigned __int128 turn) {
    const bool below = (int64_t)(uint64_t)(turn >> 64) < 0;
    if (below) turn = 0 - turn;
    const double x = fma((double)(uint64_t)(turn >> 64), 0x1p-63, (double)(uint64_t)turn * 0x1p-127);
    return below ? -x : x;
}

// (cos, sin) of the angle that is `turn` units of a turn
template <typename T, typename A, typename U> __device__ __forceinline__ void cos_sin(U turn, A scale, A& c, A& s) {
    if constexpr (std::is_same<A, double>::value) {
        sincospi(half_turns(turn), &s, &c);
    } else if constexpr (std::is_same<T, float>::value) {
        sincospif((float)(int64_t)turn * 0x1p-63f, &s, &c);
    } else {
        // 32 bits of the turn, 24 in the float: the angle is off by 2 pi 2^-32, pi 2^-25 for the float, pi 2^-25 for pi's own
        // rounding and 2^-23 for the product's
        __sincosf((float)(int32_t)(turn >> 32) * (0x1p-31f * 3.14159265358979f), &s, &c);
    }
    c *= scale;
    s *= scale;
}

// Where token (b, t) stands, and where its key and value go.
struct Token {
    int64_t b, t;
    int64_t pos;
    int64_t page, slot;
    bool live;   // goes into the cache
};

__device__ __forceinline__ Token token_of(const RotaryDesc& d, int64_t tok) {
    Token x;
    if (tok <= 0x7fffffff && d.T <= 0x7fffffff) {
        x.b = (uint32_t)tok / (uint32_t)d.T;
        x.t = (uint32_t)tok % (uint32_t)d.T;
    } else {
        x.b = tok / d.T;
        x.t = tok % d.T;
    }
    const int64_t start = d.starts ? (int64_t)load(d.starts + x.b) : 0;
    const int64_t u = start + x.t;
    x.pos = d.positions ? (int64_t)load(d.positions + tok) : u;
    x.live = false;
    x.page = x.slot = 0;
    if (d.Hkv > 0 && u >= 0 && x.t < (d.lens ? (int64_t)load(d.lens + x.b) : d.T)) {
        const int64_t i = u <= 0x7fffffff && d.page <= 0x7fffffff ? (int64_t)((uint32_t)u / (uint32_t)d.page) : u / d.page;
        if (i < d.table_pages) {
            x.page = load(d.table + x.b * d.table_pages + i);
            x.slot = u - i * d.page;
            x.live = x.page >= 0 && x.page < d.pages;
        }
    }
    return x;
}

// Row of head hh of [queries | keys | values]: false where it goes nowhere.
template <typename T>
__device__ __forceinline__ bool row_of(const RotaryDesc& d, const Token& x, int hh, const T*& src, T*& dst, bool& turned) {
    if (hh < d.H) {
        src = static_cast<const T*>(d.q) + x.b * d.qs[0] + x.t * d.qs[1] + hh * d.qs[2];
        dst = static_cast<T*>(d.q_out) + x.b * d.qo[0] + x.t * d.qo[1] + hh * d.qo[2];
        turned = true;
        return true;
    }
    const int h = hh - (int)d.H;
    if (h < d.Hkv) {
        src = static_cast<const T*>(d.k) + x.b * d.ks[0] + x.t * d.ks[1] + h * d.ks[2];
        dst = static_cast<T*>(d.k_pages) + x.page * d.kp[0] + x.slot * d.kp[1] + h * d.kp[2];
        turned = true;
    } else {
        const int hv = h - (int)d.Hkv;
        src = static_cast<const T*>(d.v) + x.b * d.vs[0] + x.t * d.vs[1] + hv * d.vs[2];
        dst = static_cast<T*>(d.v_pages) + x.page * d.vp[0] + x.slot * d.vp[1] + hv * d.vp[2];
        turned = false;
    }
    return x.live;
}

template <typename T> struct Unit {
    uint4 raw;
    static constexpr int N = 16 / sizeof(T);
    __device__ __forceinline__ void get(float (&x)[N]) const {
        if constexpr (N == 4) {
            x[0] = __uint_as_float(raw.x);
            x[1] = __uint_as_float(raw.y);
            x[2] = __uint_as_float(raw.z);
            x[3] = __uint_as_float(raw.w);
        } else {
            const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = unpack_bf16x2(w[i]);
                x[2 * i] = f.x;
                x[2 * i + 1] = f.y;
            }
        }
    }
    __device__ __forceinline__ void put(const float (&x)[N]) {
        if constexpr (N == 4)
            raw = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
        else
            raw = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
    }
};

// tile: tokens of a block; groups: blocks that share a token's heads, `span` each; every rows-th token of the tile is a
// thread's.
template <typename T, bool HALF>
__global__ void __launch_bounds__(RO_MOST) rotary_units_kernel(const __grid_constant__ RotaryDesc d, int tile, int groups, int span, int rows) {
    constexpr int N = Unit<T>::N, PAIRS = HALF ? N : N / 2;
    __shared__ uint64_t turns[RO_MAXPAIRS];
    __shared__ __align__(16) float sines[2 * RO_SINES];   // token by token: cosines, sines
    // offsets of a token's rows: queries, keys and values, where they come from and go to (-1: nowhere)
    __shared__ int64_t from[RO_TOKENS][3], to[RO_TOKENS][3], place[RO_TOKENS];
    griddep_wait();
    griddep_launch_dependents();
    const int n = (int)d.n, half = HALF ? n / N : 0;   // units whose partner is half units on
    const int items = (int)d.dh / N - half, heads = (int)d.H, Hkv = (int)d.Hkv, HH = heads + 2 * Hkv;
    const int64_t tokens = d.B * d.T, first = (int64_t)(blockIdx.x / groups) * tile;
    const int count = (int)min((int64_t)tile, tokens - first);
    for (int i = threadIdx.x; i < n; i += blockDim.x) turns[i] = turn_of<uint64_t>(d.frequencies[i]);
    for (int i = threadIdx.x; i < count; i += blockDim.x) {
        const Token x = token_of(d, first + i);
        from[i][0] = x.b * d.qs[0] + x.t * d.qs[1];
        from[i][1] = x.b * d.ks[0] + x.t * d.ks[1];
        from[i][2] = x.b * d.vs[0] + x.t * d.vs[1];
        to[i][0] = x.b * d.qo[0] + x.t * d.qo[1];
        to[i][1] = x.live ? x.page * d.kp[0] + x.slot * d.kp[1] : -1;
        to[i][2] = x.live ? x.page * d.vp[0] + x.slot * d.vp[1] : -1;
        place[i] = x.pos;
    }
    __syncthreads();
    const float scale = (float)d.scale;
    for (int i = threadIdx.x; i < count * n; i += blockDim.x) {
        const int t = i / n, j = i - t * n;
        cos_sin<T, float>(turns[j] * (uint64_t)place[t], scale, sines[2 * t * n + j], sines[(2 * t + 1) * n + j]);
    }
    __syncthreads();
    const int item = threadIdx.x % items, r = threadIdx.x / items, hh = (int)(blockIdx.x % groups) * span + r % span;
    int t = r / span;
    if (t >= rows || hh >= HH) return;
    const bool pair = HALF ? item < half : item * N < 2 * n;
    // with a partner: units item and item + half; the others stand behind them
    const int at = (HALF && !pair ? item + half : item) * N, sine = HALF ? at : at / 2;
    const int kind = hh < heads ? 0 : hh < heads + Hkv ? 1 : 2, h = hh - (kind > 0 ? heads : 0) - (kind > 1 ? Hkv : 0);
    const T* src = static_cast<const T*>(kind == 0 ? d.q : kind == 1 ? d.k : d.v) + h * (kind == 0 ? d.qs[2] : kind == 1 ? d.ks[2] : d.vs[2]) + at;
    T* dst = static_cast<T*>(kind == 0 ? d.q_out : kind == 1 ? d.k_pages : d.v_pages) + h * (kind == 0 ? d.qo[2] : kind == 1 ? d.kp[2] : d.vp[2]) + at;
    const bool turned = pair && kind < 2;
    for (; t < count; t += RO_AHEAD * rows) {
        Unit<T> a[RO_AHEAD], b[HALF ? RO_AHEAD : 1];
        int64_t where[RO_AHEAD];
#pragma unroll
        for (int j = 0; j < RO_AHEAD; ++j) {
            const int tt = t + j * rows;
            where[j] = tt < count ? to[tt][kind] : -1;
            if (where[j] < 0) continue;
            const T* row = src + from[tt][kind];
            a[j].raw = *reinterpret_cast<const uint4*>(row);
            if constexpr (HALF)
                if (pair) b[j].raw = *reinterpret_cast<const uint4*>(row + n);
        }
#pragma unroll
        for (int j = 0; j < RO_AHEAD; ++j) {
            if (where[j] < 0) continue;
            if (turned) {
                float c[PAIRS], s[PAIRS], u[N];
                const float* cs = sines + 2 * (t + j * rows) * n + sine;
#pragma unroll
                for (int e = 0; e < PAIRS; ++e) {
                    c[e] = cs[e];
                    s[e] = cs[n + e];
                }
                a[j].get(u);
                if constexpr (HALF) {
                    float v[N];
                    b[j].get(v);
#pragma unroll
                    for (int e = 0; e < N; ++e) {
                        const float x = fmaf(u[e], c[e], -v[e] * s[e]);
                        v[e] = fmaf(u[e], s[e], v[e] * c[e]);
                        u[e] = x;
                    }
                    b[j].put(v);
                } else {
#pragma unroll
                    for (int e = 0; e < N / 2; ++e) {
                        const float x = fmaf(u[2 * e], c[e], -u[2 * e + 1] * s[e]);
                        u[2 * e + 1] = fmaf(u[2 * e], s[e], u[2 * e + 1] * c[e]);
                        u[2 * e] = x;
                    }
                }
                a[j].put(u);
            }
            T* row = dst + where[j];
            *reinterpret_cast<uint4*>(row) = a[j].raw;
            if constexpr (HALF)
                if (pair) *reinterpret_cast<uint4*>(row + n) = b[j].raw;
        }
    }
}

// Any type, width, stride and alignment: a thread owns a pair, or a column behind them.
template <typename T, typename A>
__global__ void __launch_bounds__(RO_THREADS) rotary_generic_kernel(const __grid_constant__ RotaryDesc d, int groups) {
    using U = TurnOf<A>;
    __shared__ U turns[RO_MAXPAIRS];
    griddep_wait();
    griddep_launch_dependents();
    for (int i = threadIdx.x; i < d.n; i += RO_THREADS) turns[i] = turn_of<U>(d.frequencies[i]);
    __syncthreads();
    const int n = (int)d.n, items = (int)d.dh - n, HH = (int)(d.H + 2 * d.Hkv), per = groups * items;
    const int64_t total = d.B * d.T * per;
    for (int64_t i = (int64_t)blockIdx.x * RO_THREADS + threadIdx.x; i < total; i += (int64_t)gridDim.x * RO_THREADS) {
        const int rest = (int)(i % per), group = rest / items, item = rest % items;
        const Token x = token_of(d, i / per);
        const bool pair = item < n;
        const int at = !pair ? item + n : d.layout == VIT_ROTARY_HALF ? item : 2 * item;
        const int to = d.layout == VIT_ROTARY_HALF ? at + n : at + 1;
        A c = 1, s = 0;
        if (pair) cos_sin<T, A>(turns[item] * (U)x.pos, (A)d.scale, c, s);   // modulo a turn, negative positions too
        for (int h = group; h < HH; h += groups) {
            const T* src;
            T* dst;
            bool turned;
            if (!row_of<T>(d, x, h, src, dst, turned)) continue;
            if (!pair) {
                dst[at] = src[at];
            } else if (!turned) {
                const T u = src[at], v = src[to];
                dst[at] = u;
                dst[to] = v;
            } else {
                const A u = to_acc<A>(src[at]), v = to_acc<A>(src[to]);
                dst[at] = from_acc<T>(fma(u, c, -v * s));
                dst[to] = from_acc<T>(fma(u, s, v * c));
            }
        }
    }
}

bool units_fit(const void* p, const int64_t st[3], int64_t N) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && st[0] % N == 0 && st[1] % N == 0 && st[2] % N == 0;
}

}  // namespace

cudaError_t launch_rotary(const RotaryDesc& d, const DeviceInfo& dev, cudaStream_t s) {
    const int64_t HH = d.H + 2 * d.Hkv, N = d.dt == DT_F64 ? 1 : 16 / (int64_t)dt_size(d.dt);
    const bool half = d.layout == VIT_ROTARY_HALF;
    bool units = d.dt != DT_F64 && d.dh % N == 0 && (half ? d.n : 2 * d.n) % N == 0;
    if (d.H) units = units && units_fit(d.q, d.qs, N) && units_fit(d.q_out, d.qo, N);
    if (d.Hkv)
        units = units && units_fit(d.k, d.ks, N) && units_fit(d.v, d.vs, N) && units_fit(d.k_pages, d.kp, N) &&
                units_fit(d.v_pages, d.vp, N);
    if (units) {
        const int64_t items = d.dh / N - (half ? d.n / N : 0), tokens = d.B * d.T, sms = dev.num_sms;
        // Heads to a block: all that fit it; with few tokens they are dealt out, while that gives each SM a block more.
        int64_t span = RO_MOST / items < HH ? RO_MOST / items : HH;
        while (span > 1 && tokens * ((HH + span - 1) / span) * 2 <= sms) span = (span + 1) / 2;
        const int64_t groups = (HH + span - 1) / span;
        const int64_t rows = RO_THREADS / (items * span) > 1 ? RO_THREADS / (items * span) : 1;
        auto launch = [&](auto k, int which) -> cudaError_t {
            // Tokens to a block: whole rounds of blocks, as few as RO_SINES pairs of sines and RO_TOKENS allow, and no rest
            // of one (4 x 2048 tokens of 20 heads of 128 in 586 blocks, of which 608 fit: 17.3 us; in 631: 22).
            static std::atomic<int> fits[4][RO_MOST / 32 + 1];   // blocks of so many warps to an SM, of the first device asked
            const int64_t warps = (items * span * rows + 31) / 32;
            std::atomic<int>& fit = fits[which][warps];
            int resident = fit.load(std::memory_order_relaxed);
            if (!resident) {
                const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&resident, k, (int)warps * 32, 0);
                if (e != cudaSuccess) return e;
                resident = resident < 1 ? 1 : resident;
                fit.store(resident, std::memory_order_relaxed);
            }
            int64_t most = d.n ? RO_SINES / d.n : RO_TOKENS;
            most = most > RO_TOKENS ? RO_TOKENS : most;
            const int64_t room = resident * sms, rounds = (tokens * groups + room * most - 1) / (room * most);
            const int64_t tile = (tokens * groups + room * rounds - 1) / (room * rounds);
            const int64_t blocks = (tokens + tile - 1) / tile * groups, used = rows < tile ? rows : tile;
            if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
            const dim3 grid((unsigned)blocks), block((unsigned)((items * span * used + 31) / 32 * 32));
            return launch_dependent(k, grid, block, 0, s, d, (int)tile, (int)groups, (int)span, (int)used);
        };
        if (d.dt == DT_BF16) return half ? launch(rotary_units_kernel<__nv_bfloat16, true>, 0) : launch(rotary_units_kernel<__nv_bfloat16, false>, 1);
        return half ? launch(rotary_units_kernel<float, true>, 2) : launch(rotary_units_kernel<float, false>, 3);
    }
    const dim3 block(RO_THREADS);
    const int64_t items = d.dh - d.n;
    // heads of a token that one thread walks over: all of them where there are threads enough
    const double threads = (double)d.B * d.T * HH * items;
    int64_t walk = (int64_t)(threads / (1024.0 * dev.num_sms));
    walk = walk < 1 ? 1 : walk > HH ? HH : walk;
    const int groups = (int)((HH + walk - 1) / walk);
    const double want = ((double)d.B * d.T * groups * items + RO_THREADS - 1) / RO_THREADS;
    const dim3 grid((unsigned)(want < 8.0 * dev.num_sms ? want : 8.0 * dev.num_sms));
    if (d.dt == DT_F64) return launch_dependent(rotary_generic_kernel<double, double>, grid, block, 0, s, d, groups);
    if (d.dt == DT_F32) return launch_dependent(rotary_generic_kernel<float, float>, grid, block, 0, s, d, groups);
    return launch_dependent(rotary_generic_kernel<__nv_bfloat16, float>, grid, block, 0, s, d, groups);
}

}  // namespace vit
