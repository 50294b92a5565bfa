// cross_maps.cuh -- tensor maps over the strided (B, T, heads, dh) operands of cross attention.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>

namespace vit {
namespace {

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn ct_encode_fn() {
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

// (B, T, heads, dh) with element strides st (sequence, token, head); boxes of 64 columns x
// box_heads x box_tokens. A sequence or head stride of 0 becomes an extent of 1.
inline bool ct_map(CUtensorMap* m, const void* base, const int64_t st[3], int64_t B, int64_t T, int64_t heads, int64_t dh,
            uint32_t box_heads, uint32_t box_tokens, CUtensorMapL2promotion l2) {
    const cuuint64_t dims[4] = {(cuuint64_t)dh, (cuuint64_t)(st[2] ? heads : 1), (cuuint64_t)T, (cuuint64_t)(st[0] ? B : 1)};
    const cuuint64_t strides[3] = {(cuuint64_t)((st[2] ? st[2] : dh) * 2), (cuuint64_t)(st[1] * 2),
                                   (cuuint64_t)((st[0] ? st[0] : dh) * 2)};
    const cuuint32_t box[4] = {64, box_heads, box_tokens, 1}, estr[4] = {1, 1, 1, 1};
    return ct_encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, estr,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, l2,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The same in fp32: boxes of 32 columns x one head x box_tokens.
inline bool ct_map_f32(CUtensorMap* m, const void* base, const int64_t st[3], int64_t B, int64_t T, int64_t heads,
                       int64_t dh, uint32_t box_tokens) {
    const cuuint64_t dims[4] = {(cuuint64_t)dh, (cuuint64_t)(st[2] ? heads : 1), (cuuint64_t)T, (cuuint64_t)(st[0] ? B : 1)};
    const cuuint64_t strides[3] = {(cuuint64_t)((st[2] ? st[2] : dh) * 4), (cuuint64_t)(st[1] * 4),
                                   (cuuint64_t)((st[0] ? st[0] : dh) * 4)};
    const cuuint32_t box[4] = {32, 1, box_tokens, 1}, estr[4] = {1, 1, 1, 1};
    return ct_encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, const_cast<void*>(base), dims, strides, box, estr,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 16-byte aligned rows (strides in multiples of `unit` elements), and strides that a tensor map takes.
inline bool ct_strides_ok(const void* base, const int64_t st[3], int64_t T, int unit = 8) {
    if (reinterpret_cast<uintptr_t>(base) & 15) return false;
    for (int i = 0; i < 3; ++i)
        if (st[i] % unit != 0 || st[i] >= ((int64_t)1 << 37)) return false;
    return T == 1 || st[1] > 0;
}

}  // namespace
}  // namespace vit
