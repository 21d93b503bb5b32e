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

// The current device's properties, queried once per device.
struct Device {
    int ordinal, sms, smem_limit, smem_per_sm;
    bool gb300;  // compute capability 10.3
};

inline int current_device(Device &d)
{
    static std::mutex mu;
    static Device known[64];
    static bool have[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return kErrCuda;
    }
    std::lock_guard<std::mutex> lock(mu);
    if (dev < 64 && have[dev]) {
        d = known[dev];
        return kOk;
    }
    int major = 0, minor = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) ||
        cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev) ||
        cudaDeviceGetAttribute(&d.smem_limit, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) ||
        cudaDeviceGetAttribute(&d.smem_per_sm, cudaDevAttrMaxSharedMemoryPerMultiprocessor, dev)) {
        cudaGetLastError();
        return kErrCuda;
    }
    d.ordinal = dev;
    d.gb300 = major == 10 && minor == 3;
    if (dev < 64) {
        known[dev] = d;
        have[dev] = true;
    }
    return kOk;
}

// Launch as a programmatic dependent of the kernel before it in the stream:
// the launch and set-up overlap that kernel's end, and the kernel waits
// (griddepcontrol.wait) before it touches memory that others may write.
template <class... P, class... A>
inline int launch(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, unsigned cluster,
                  A... args)
{
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[2];
    unsigned na = 0;
    attr[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[na].val.programmaticStreamSerializationAllowed = 1;
    ++na;
    if (cluster > 1) {
        attr[na].id = cudaLaunchAttributeClusterDimension;
        attr[na].val.clusterDim.x = cluster;
        attr[na].val.clusterDim.y = 1;
        attr[na].val.clusterDim.z = 1;
        ++na;
    }
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = na;
    if (cudaLaunchKernelEx(&cfg, kernel, P(args)...) != cudaSuccess) {
        cudaGetLastError();
        return kErrCuda;
    }
    return kOk;
}

}  // namespace tg
