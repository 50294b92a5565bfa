// attention_cross_rows.cu -- cross attention of few queries (decoding): the mathematics of
// attention_cross.cu where one key head serves at most 16 query rows (Tq * G <= 16), bf16,
// head width up to 128 in steps of 8.
//
// Bound by reading K and V once. The keys of a (sequence, key head) are dealt out in tiles of 16
// to the warps of one CTA or of a cluster of CTAs; every warp keeps its own running maximum, sum
// and output rows, joined at the end through shared memory and, between the CTAs of a cluster,
// distributed shared memory: no workspace, one launch, the same order of additions every time.
//
// A warp multiplies with mma.m16n8k16 straight from 16-byte global loads, without shared memory:
//  - S = Q K^T: the order of the columns in a dot product is free, so the thread that owns
//    columns 2c, 2c+1, 2c+8, 2c+9 of a k-step takes 8 consecutive columns of a 32-column piece
//    (two k-steps) of its key and of its query rows instead.
//  - O = P V: which output column an n-tile's column means is free too: thread n of a tile loads
//    8 consecutive columns of 4 keys, interleaves key pairs with byte permutes, and column n * 8 + j
//    becomes column n of n-tile j.
// The tensor cores see 16 rows where one may be asked for; they are idle otherwise.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "kernels.h"
#include "launch.cuh"
#include "ptx.cuh"

namespace vit {
namespace {

constexpr int CR_ROWS = 16, CR_KEYS = 16;

__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// Floats of one set of output rows with their maxima and sums, in whole 16-byte units.
__host__ __device__ __forceinline__ int rows_floats(int R, int dh) { return (R * (dh + 2) + 3) & ~3; }

// DHT: the head width rounded up to 64 or 128; columns past dh are zeros.
template <int DHT, int NW>
__global__ void __launch_bounds__(NW * 32)
cross_rows_kernel(const CrossDesc d, float scale_log2, int Z) {
    constexpr int KC = DHT / 32, VC = DHT / 64;   // 32-column pieces of K, 64-column pieces of V
    extern __shared__ __align__(16) float sm[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c4 = lane & 3, r8 = lane >> 2;
    const int z = Z > 1 ? (int)ptx::cluster_ctarank() : 0;
    const int bh = blockIdx.x / Z, b = bh / (int)d.Hkv, h = bh % (int)d.Hkv;
    const int G = (int)(d.H / d.Hkv), R = (int)d.Tq * G, dh = (int)d.dh;
    // shared memory: per warp O (R x dh), m and l (R each); then this CTA's joined O, m, l
    const int piece = rows_floats(R, dh);
    float* wO = sm + warp * piece;
    float* jO = sm + NW * piece;
    griddep_wait();
    griddep_launch_dependents();

    const __nv_bfloat16* k = static_cast<const __nv_bfloat16*>(d.k) + b * d.ks[0] + h * d.ks[2];
    const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(d.v) + b * d.vs[0] + h * d.vs[2];
    int64_t len = d.Tk;
    if (d.kv_lens) len = min((int64_t)max(__ldg(d.kv_lens + b), 0), d.Tk);
    const uint4 zero = make_uint4(0, 0, 0, 0);

    // query rows r8 and r8 + 8; packed row = token * G + head of the group
    uint4 q[2][KC];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = r8 + 8 * i;
        const __nv_bfloat16* qr = static_cast<const __nv_bfloat16*>(d.q) + b * d.qs[0] + (r / G) * d.qs[1] +
                                  (int64_t)(h * G + r % G) * d.qs[2];
#pragma unroll
        for (int c = 0; c < KC; ++c) {
            const int col = c * 32 + c4 * 8;
            q[i][c] = r < R && col < dh ? *reinterpret_cast<const uint4*>(qr + col) : zero;
        }
    }

    float o[VC * 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < VC * 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[j][e] = 0.f;

    uint4 kt[2][KC], vt[4][VC];
    auto load = [&](int64_t u0) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {   // keys r8, r8 + 8: n-tiles 0 and 1 of S
            const int64_t u = u0 + r8 + 8 * i;
            const __nv_bfloat16* kr = k + u * d.ks[1];
#pragma unroll
            for (int c = 0; c < KC; ++c) {
                const int col = c * 32 + c4 * 8;
                kt[i][c] = u < len && col < dh ? __ldg(reinterpret_cast<const uint4*>(kr + col)) : zero;
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {   // keys 2 c4, 2 c4 + 1, 2 c4 + 8, 2 c4 + 9
            const int64_t u = u0 + 2 * c4 + (i & 1) + 8 * (i >> 1);
            const __nv_bfloat16* vr = v + u * d.vs[1];
#pragma unroll
            for (int c = 0; c < VC; ++c) {
                const int col = c * 64 + r8 * 8;
                vt[i][c] = u < len && col < dh ? __ldg(reinterpret_cast<const uint4*>(vr + col)) : zero;
            }
        }
    };

    const int64_t step = (int64_t)Z * NW * CR_KEYS;
    int64_t u0 = (int64_t)(z * NW + warp) * CR_KEYS;
    if (u0 < len) load(u0);
    for (; u0 < len; u0 += step) {
        // S for 16 keys: s[i] are n-tiles of 8 keys
        float s[2][4] = {};
#pragma unroll
        for (int c = 0; c < KC; ++c) {
            const uint32_t a0[4] = {q[0][c].x, q[1][c].x, q[0][c].y, q[1][c].y};
            const uint32_t a1[4] = {q[0][c].z, q[1][c].z, q[0][c].w, q[1][c].w};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                mma_16816(s[i], a0, kt[i][c].x, kt[i][c].y);
                mma_16816(s[i], a1, kt[i][c].z, kt[i][c].w);
            }
        }
        // V of this tile as key pairs, then the next tile's loads go out
        uint32_t vb[VC * 8][2];
#pragma unroll
        for (int c = 0; c < VC; ++c) {
            const uint32_t* w0 = reinterpret_cast<const uint32_t*>(&vt[0][c]);
            const uint32_t* w1 = reinterpret_cast<const uint32_t*>(&vt[1][c]);
            const uint32_t* w2 = reinterpret_cast<const uint32_t*>(&vt[2][c]);
            const uint32_t* w3 = reinterpret_cast<const uint32_t*>(&vt[3][c]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                vb[c * 8 + 2 * e][0] = __byte_perm(w0[e], w1[e], 0x5410);
                vb[c * 8 + 2 * e + 1][0] = __byte_perm(w0[e], w1[e], 0x7632);
                vb[c * 8 + 2 * e][1] = __byte_perm(w2[e], w3[e], 0x5410);
                vb[c * 8 + 2 * e + 1][1] = __byte_perm(w2[e], w3[e], 0x7632);
            }
        }
        const int64_t here = u0;
        if (u0 + step < len) load(u0 + step);

        uint32_t a[4];
        bool grew = false;
        float alpha[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {   // rows r8 + 8 i: s[n][2 i], s[n][2 i + 1]
            float x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int64_t u = here + 8 * (e >> 1) + 2 * c4 + (e & 1);
                x[e] = u < len ? s[e >> 1][2 * i + (e & 1)] * scale_log2 : -INFINITY;
            }
            float mx = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            mx = fmaxf(mx, m[i]);
            alpha[i] = mx > m[i] ? exp2_approx(m[i] - mx) : 1.f;
            grew = grew || mx > m[i];
            m[i] = mx;
            const float base = mx == -INFINITY ? 0.f : mx;
            float p[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) p[e] = exp2_approx(x[e] - base);
            l[i] = l[i] * alpha[i] + ((p[0] + p[1]) + (p[2] + p[3]));   // this thread's keys; joined at the end
            a[i] = pack_bf16x2(p[0], p[1]);
            a[2 + i] = pack_bf16x2(p[2], p[3]);
        }
        if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
            for (int j = 0; j < VC * 8; ++j) {
                o[j][0] *= alpha[0];
                o[j][1] *= alpha[0];
                o[j][2] *= alpha[1];
                o[j][3] *= alpha[1];
            }
        }
#pragma unroll
        for (int j = 0; j < VC * 8; ++j) mma_16816(o[j], a, vb[j][0], vb[j][1]);
    }

    // this warp's rows: column n * 8 + j of piece c is column n of n-tile 8 c + j
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
        const int r = r8 + 8 * i;
        if (r < R) {
#pragma unroll
            for (int c = 0; c < VC; ++c)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int col = c * 64 + (2 * c4 + e) * 8;
                    if (col < dh) {
#pragma unroll
                        for (int j = 0; j < 8; j += 4)
                            *reinterpret_cast<float4*>(wO + r * dh + col + j) =
                                make_float4(o[c * 8 + j][2 * i + e], o[c * 8 + j + 1][2 * i + e],
                                            o[c * 8 + j + 2][2 * i + e], o[c * 8 + j + 3][2 * i + e]);
                    }
                }
            if (c4 == 0) {
                wO[R * dh + r] = m[i];
                wO[R * dh + R + r] = l[i];
            }
        }
    }
    __syncthreads();

    // join the warps' rows: row maxima first, then every output column
    auto out = [&](int r, int col) {
        return static_cast<__nv_bfloat16*>(d.o) + (((int64_t)b * d.Tq + r / G) * d.H + h * G + r % G) * dh + col;
    };
    for (int i = threadIdx.x; i < R * dh; i += NW * 32) {
        const int r = i / dh;
        float mx = -INFINITY;
#pragma unroll
        for (int w = 0; w < NW; ++w) mx = fmaxf(mx, sm[w * piece + R * dh + r]);
        const float base = mx == -INFINITY ? 0.f : mx;
        float acc = 0.f, sum = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const float* p = sm + w * piece;
            const float f = exp2_approx(p[R * dh + r] - base);
            acc = fmaf(f, p[i], acc);
            sum = fmaf(f, p[R * dh + R + r], sum);
        }
        if (Z == 1) {
            *out(r, i - r * dh) = __float2bfloat16_rn(len > 0 ? acc / sum : 0.f);
        } else {
            jO[i] = acc;
            if (i == r * dh) {
                jO[R * dh + r] = mx;
                jO[R * dh + R + r] = sum;
            }
        }
    }
    if (Z > 1) {
        ptx::cluster_sync();   // every CTA's joined rows are in place
        const uint32_t own = ptx::smem_addr(jO);
        for (int i = z * NW * 32 + threadIdx.x; i < R * dh; i += Z * NW * 32) {
            const int r = i / dh;
            float mx = -INFINITY;
            for (int y = 0; y < Z; ++y) mx = fmaxf(mx, ld_cluster_f32(ptx::mapa_shared(own + (R * dh + r) * 4, y)));
            const float base = mx == -INFINITY ? 0.f : mx;
            float acc = 0.f, sum = 0.f;
            for (int y = 0; y < Z; ++y) {
                const float f = exp2_approx(ld_cluster_f32(ptx::mapa_shared(own + (R * dh + r) * 4, y)) - base);
                acc = fmaf(f, ld_cluster_f32(ptx::mapa_shared(own + i * 4, y)), acc);
                sum = fmaf(f, ld_cluster_f32(ptx::mapa_shared(own + (R * dh + R + r) * 4, y)), sum);
            }
            *out(r, i - r * dh) = __float2bfloat16_rn(len > 0 ? acc / sum : 0.f);
        }
        ptx::cluster_sync();   // no CTA leaves while another reads its shared memory
    }
}

template <int DHT, int NW>
cudaError_t launch_rows(const CrossDesc& d, int Z, cudaStream_t s) {
    const int R = (int)(d.Tq * (d.H / d.Hkv));
    const size_t smem = (size_t)(NW + (Z > 1)) * rows_floats(R, (int)d.dh) * 4;
    auto k = cross_rows_kernel<DHT, NW>;
    static std::atomic<uint64_t> attr{0};
    cudaError_t e = set_smem_limit_once(k, (NW + 1) * rows_floats(CR_ROWS, DHT) * 4, attr);
    if (e != cudaSuccess) return e;
    const float sl2 = (float)(d.scale * 1.4426950408889634);
    if (Z == 1) return launch_dependent(k, dim3((unsigned)(d.B * d.Hkv)), dim3(NW * 32), smem, s, d, sl2, 1);
    return launch_dependent_cluster(k, dim3((unsigned)(d.B * d.Hkv * Z)), dim3(NW * 32), Z, smem, s, d, sl2, Z);
}

}  // namespace

bool cross_rows_supported(const CrossDesc& d) {
    if (d.dt != DT_BF16 || d.dh % 8 != 0 || d.dh > 128 || d.Tq * (d.H / d.Hkv) > CR_ROWS) return false;
    if (d.B > 0x7fffffff / 8 / d.Hkv) return false;
    const struct { const void* p; const int64_t* st; } in[] = {{d.q, d.qs}, {d.k, d.ks}, {d.v, d.vs}};
    for (const auto& i : in) {
        if (reinterpret_cast<uintptr_t>(i.p) & 15) return false;
        for (int j = 0; j < 3; ++j)
            if (i.st[j] % 8 != 0) return false;
    }
    return true;
}

cudaError_t launch_cross_rows(const CrossDesc& d, const DeviceInfo& dev, cudaStream_t s) {
    // CTAs of four warps; a key head's keys go to as many CTAs as keep the GPU's warp slots busy
    // (about eight CTAs per SM), each warp having two tiles of 16 keys at least
    const int64_t heads = d.B * d.Hkv, want = 8 * (int64_t)dev.num_sms;
    int Z = 1;
    while (Z < 8 && heads * Z < want && d.Tk >= (int64_t)Z * 2 * 4 * CR_KEYS * 2) Z *= 2;
    return d.dh <= 64 ? launch_rows<64, 4>(d, Z, s) : launch_rows<128, 4>(d, Z, s);
}

}  // namespace vit
