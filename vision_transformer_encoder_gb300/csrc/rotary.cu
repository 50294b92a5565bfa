// rotary.cu -- rotary positions, and appending keys and values to a paged cache on the way.
//   pair i = (u, v) at position p -> scale (u cos a - v sin a, u sin a + v cos a),   a = p f_i
// One kernel turns the heads of the queries into their output and those of the keys into their pages, and copies
// the values into theirs; without keys it is the plain rotation.
//
// The angle: f_i / 2 pi as a 64-bit fraction of a turn, once per block and pair (fp64, of which the GPU has little). A
// position times that, modulo 2^64, is the fraction of a turn of p f_i, exact but for p 2^-64 and the rounding of f_i / 2 pi
// (2^-52 of it): no range reduction, and far positions lose nothing. Sine and cosine are the hardware's on [-pi, pi] for
// bf16 (off by 2^-20, where a result is rounded at 2^-9), sincospi for fp32 and fp64.
//
// Bound by reading and writing each head once. A thread owns a 16-byte unit of a head (both halves of its pairs) of
// one token: it makes their sines once and walks over the token's heads, four in flight. With few tokens the heads go to
// threads of their own.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "launch.cuh"

namespace vit {
namespace {

constexpr int RO_THREADS = 256, RO_MAXPAIRS = 256, RO_AHEAD = 4;

// f / 2 pi as a fraction of a turn in units of 2^-64
__device__ __forceinline__ uint64_t turn_of(double f) {
    double t = f * 0.15915494309189533577;
    t -= floor(t);
    return __double2ull_rn(t * 18446744073709551616.0);   // 1 itself saturates
}

// (cos, sin) of the angle that is `turn` 2^-64 of a turn, in half turns of [-1, 1)
template <typename T, typename A> __device__ __forceinline__ void cos_sin(uint64_t turn, A scale, A& c, A& s) {
    if constexpr (std::is_same<A, double>::value) {
        sincospi((double)(int64_t)turn * 0x1p-63, &s, &c);
    } else if constexpr (std::is_same<T, float>::value) {
        sincospif((float)(int64_t)turn * 0x1p-63f, &s, &c);
    } else {
        // 32 bits of the turn: off by pi 2^-32
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
    const int64_t start = d.starts ? (int64_t)__ldg(d.starts + x.b) : 0;
    const int64_t u = start + x.t;
    x.pos = d.positions ? (int64_t)__ldg(d.positions + tok) : u;
    x.live = false;
    x.page = x.slot = 0;
    if (d.Hkv > 0 && u >= 0 && x.t < (d.lens ? (int64_t)__ldg(d.lens + x.b) : d.T)) {
        const int64_t i = u <= 0x7fffffff && d.page <= 0x7fffffff ? (int64_t)((uint32_t)u / (uint32_t)d.page) : u / d.page;
        if (i < d.table_pages) {
            x.page = __ldg(d.table + x.b * d.table_pages + i);
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

// groups: threads that share a token's heads; each takes every groups-th.
template <typename T, bool HALF>
__global__ void __launch_bounds__(RO_THREADS) rotary_units_kernel(const __grid_constant__ RotaryDesc d, int groups) {
    constexpr int N = Unit<T>::N, PAIRS = HALF ? N : N / 2;
    __shared__ uint64_t turns[RO_MAXPAIRS];
    griddep_wait();
    griddep_launch_dependents();
    for (int i = threadIdx.x; i < d.n; i += RO_THREADS) turns[i] = turn_of(d.frequencies[i]);
    __syncthreads();
    const int half = HALF ? (int)d.n / N : 0;   // units whose partner is half units on
    const int items = (int)d.dh / N - half, HH = (int)(d.H + 2 * d.Hkv), per = groups * items;
    const int64_t tokens = d.B * d.T;
    const int64_t total = tokens * per;
    const float scale = (float)d.scale;
    for (int64_t i = (int64_t)blockIdx.x * RO_THREADS + threadIdx.x; i < total; i += (int64_t)gridDim.x * RO_THREADS) {
        int64_t tok;
        int rest;
        if (total <= 0x7fffffff) {
            tok = (uint32_t)i / (uint32_t)per;
            rest = (uint32_t)i % (uint32_t)per;
        } else {
            tok = i / per;
            rest = (int)(i % per);
        }
        const int group = rest / items, item = rest % items;
        const Token x = token_of(d, tok);
        const bool pair = HALF ? item < half : item * N < 2 * d.n;
        // with a partner: units item and item + half; the others stand behind them
        const int at = (HALF && !pair ? item + half : item) * N, to = at + (HALF ? (int)d.n : 0);
        float c[PAIRS], s[PAIRS];
        if (pair) {
            const uint64_t p = (uint64_t)x.pos;
            const int first = HALF ? at : at / 2;
#pragma unroll
            for (int j = 0; j < PAIRS; ++j) cos_sin<T, float>(turns[first + j] * p, scale, c[j], s[j]);
        }
        for (int h0 = group; h0 < HH; h0 += RO_AHEAD * groups) {
            Unit<T> a[RO_AHEAD], b[HALF ? RO_AHEAD : 1];
            T* dst[RO_AHEAD];
            bool on[RO_AHEAD], turned[RO_AHEAD];
#pragma unroll
            for (int j = 0; j < RO_AHEAD; ++j) {
                const T* src;
                on[j] = h0 + j * groups < HH && row_of<T>(d, x, h0 + j * groups, src, dst[j], turned[j]);
                if (!on[j]) continue;
                a[j].raw = *reinterpret_cast<const uint4*>(src + at);
                if constexpr (HALF)
                    if (pair) b[j].raw = *reinterpret_cast<const uint4*>(src + to);
            }
#pragma unroll
            for (int j = 0; j < RO_AHEAD; ++j) {
                if (!on[j]) continue;
                if (pair && turned[j]) {
                    float u[N];
                    a[j].get(u);
                    if constexpr (HALF) {
                        float v[N];
                        b[j].get(v);
#pragma unroll
                        for (int e = 0; e < N; ++e) {
                            const float r = fmaf(u[e], c[e], -v[e] * s[e]);
                            v[e] = fmaf(u[e], s[e], v[e] * c[e]);
                            u[e] = r;
                        }
                        b[j].put(v);
                    } else {
#pragma unroll
                        for (int e = 0; e < N / 2; ++e) {
                            const float r = fmaf(u[2 * e], c[e], -u[2 * e + 1] * s[e]);
                            u[2 * e + 1] = fmaf(u[2 * e], s[e], u[2 * e + 1] * c[e]);
                            u[2 * e] = r;
                        }
                    }
                    a[j].put(u);
                }
                *reinterpret_cast<uint4*>(dst[j] + at) = a[j].raw;
                if constexpr (HALF)
                    if (pair) *reinterpret_cast<uint4*>(dst[j] + to) = b[j].raw;
            }
        }
    }
}

// Any type, width, stride and alignment: a thread owns a pair, or a column behind them.
template <typename T, typename A>
__global__ void __launch_bounds__(RO_THREADS) rotary_generic_kernel(const __grid_constant__ RotaryDesc d, int groups) {
    __shared__ uint64_t turns[RO_MAXPAIRS];
    griddep_wait();
    griddep_launch_dependents();
    for (int i = threadIdx.x; i < d.n; i += RO_THREADS) turns[i] = turn_of(d.frequencies[i]);
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
        if (pair) cos_sin<T, A>(turns[item] * (uint64_t)x.pos, (A)d.scale, c, s);
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
    const int64_t items = units ? d.dh / N - (half ? d.n / N : 0) : d.dh - d.n;
    // heads of a token that one thread walks over: all of them where there are threads enough
    const double threads = (double)d.B * d.T * HH * items;
    int64_t walk = (int64_t)(threads / (1024.0 * dev.num_sms));
    walk = walk < 1 ? 1 : walk > HH ? HH : walk;
    const int groups = (int)((HH + walk - 1) / walk);
    const double want = ((double)d.B * d.T * groups * items + RO_THREADS - 1) / RO_THREADS;
    const dim3 grid((unsigned)(want < 8.0 * dev.num_sms ? want : 8.0 * dev.num_sms)), block(RO_THREADS);
    if (units && d.dt == DT_BF16)
        return half ? launch_dependent(rotary_units_kernel<__nv_bfloat16, true>, grid, block, 0, s, d, groups)
                    : launch_dependent(rotary_units_kernel<__nv_bfloat16, false>, grid, block, 0, s, d, groups);
    if (units)
        return half ? launch_dependent(rotary_units_kernel<float, true>, grid, block, 0, s, d, groups)
                    : launch_dependent(rotary_units_kernel<float, false>, grid, block, 0, s, d, groups);
    if (d.dt == DT_F64) return launch_dependent(rotary_generic_kernel<double, double>, grid, block, 0, s, d, groups);
    if (d.dt == DT_F32) return launch_dependent(rotary_generic_kernel<float, float>, grid, block, 0, s, d, groups);
    return launch_dependent(rotary_generic_kernel<__nv_bfloat16, float>, grid, block, 0, s, d, groups);
}

}  // namespace vit
