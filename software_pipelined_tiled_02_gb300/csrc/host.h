// host.h -- host-side helpers shared by the translation units: tensor-map
// encoding, alignment and the watchdog default.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstdlib>
#include <mutex>

#include "layout.h"

namespace tg {

static const unsigned long long kDefaultWatchdogNs = 2000000000ull;

inline unsigned long long env_watchdog()
{
    const char *e = std::getenv("TGEMM_WATCHDOG_NS");
    if (e && *e) {
        char *end = nullptr;
        unsigned long long v = std::strtoull(e, &end, 10);
        if (end && *end == '\0' && v > 0) return v;
    }
    return kDefaultWatchdogNs;
}

inline int aligned16(const void *ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 15u) == 0; }

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_fn()
{
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q{};
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(ptr);
    });
    return fn;
}

inline CUtensorMapSwizzle swizzle_for(int row_bytes)
{
    return row_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B
           : row_bytes == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                             : CU_TENSOR_MAP_SWIZZLE_32B;
}

// Descriptor swizzle field (bits 61-63): 128 B -> 2, 64 B -> 4, 32 B -> 6.
inline uint32_t desc_layout_for(int row_bytes) { return row_bytes == 128 ? 2u : row_bytes == 64 ? 4u : 6u; }

inline CUtensorMapDataType tmap_dtype(int dt)
{
    return dt == kF32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
           : dt == kBF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                         : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
}

// L2 promotion of the operand loads.  With rows that start on 128-byte
// boundaries, 256-byte promotion helps slightly.  When the row pitch is not a
// multiple of 128 bytes (K = 5000 at 16 bits), every 128-byte box row
// straddles two lines; there 256-byte promotion measured about 5 % slower
// than 128-byte promotion.
inline CUtensorMapL2promotion operand_promotion(uint64_t pitch_bytes)
{
    return pitch_bytes % 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_256B;
}

inline int encode_2d(CUtensorMap *m, int dt, const void *base, uint64_t inner, uint64_t outer, uint64_t pitch_bytes,
                     uint32_t box_inner, uint32_t box_outer, CUtensorMapSwizzle swz, CUtensorMapL2promotion l2)
{
    EncodeTiledFn fn = encode_fn();
    if (!fn) return kErrCuda;
    cuuint64_t dims[2] = {inner, outer};
    cuuint64_t strides[1] = {pitch_bytes};
    cuuint32_t box[2] = {box_inner, box_outer};
    cuuint32_t estr[2] = {1, 1};
    CUresult r = fn(m, tmap_dtype(dt), 2, const_cast<void *>(base), dims, strides, box, estr,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, swz, l2, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? kOk : kErrCuda;
}

}  // namespace tg
