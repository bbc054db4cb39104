// Host-side helpers shared by the C ABI units: the device's limits, alignment checks and the launch.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <cstring>

namespace cvk {

// The device the launch plans size for: SM count (the persistent grids), shared memory per SM
// (residency) and per block (opt-in maximum), queried once per device and cached.  Without a
// usable device (cv_verify_plan on a host without a GPU) the plans are made for a GB300: 152 SMs,
// 228 KB per SM, 227 KB per block.
struct DeviceLimits {
    int sms, smem_per_sm, smem_per_block;
};
inline DeviceLimits device_limits() {
    constexpr DeviceLimits kGB300{152, 232448, 227 * 1024};
    constexpr int kMaxDevices = 64;
    static std::atomic<int> cached[kMaxDevices][3];  // zero until queried
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) {
        cudaGetLastError();  // clear the error the failed query recorded
        return kGB300;
    }
    if (dev < kMaxDevices && cached[dev][0].load(std::memory_order_acquire) > 0)
        return {cached[dev][0].load(std::memory_order_relaxed), cached[dev][1].load(std::memory_order_relaxed),
                cached[dev][2].load(std::memory_order_relaxed)};
    DeviceLimits d{0, 0, 0};
    if (cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&d.smem_per_sm, cudaDevAttrMaxSharedMemoryPerMultiprocessor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&d.smem_per_block, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) != cudaSuccess ||
        d.sms < 1) {
        cudaGetLastError();
        return kGB300;
    }
    if (dev < kMaxDevices) {
        cached[dev][1].store(d.smem_per_sm, std::memory_order_relaxed);
        cached[dev][2].store(d.smem_per_block, std::memory_order_relaxed);
        cached[dev][0].store(d.sms, std::memory_order_release);
    }
    return d;
}

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool stride16(long long stride_elems, int esize) { return ((stride_elems * esize) & 15) == 0; }
inline bool pow2(int v) { return v > 0 && (v & (v - 1)) == 0; }

// Launch with programmatic stream serialization: the kernel may be scheduled while the previous
// grid in the stream finishes; every kernel waits (griddepcontrol.wait) for that grid's completion
// before its first global-memory access, so the order of the stream's work is kept.
template <typename P>
cudaError_t launch_pdl(void (*kernel)(P), dim3 grid, dim3 block, int smem, cudaStream_t stream, const P &p) {
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof cfg);
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    std::memset(attr, 0, sizeof attr);
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

// The same in clusters of `cluster` blocks.
template <typename P>
cudaError_t launch_pdl_cluster(void (*kernel)(P), dim3 grid, dim3 block, int cluster, cudaStream_t stream, const P &p) {
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof cfg);
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    std::memset(attr, 0, sizeof attr);
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

// Opt a kernel into more than 48 KB of dynamic shared memory (once per kernel and device).
inline cudaError_t ensure_smem(const void *kernel, int bytes) {
    if (bytes <= 48 * 1024) return cudaSuccess;
    static std::atomic<unsigned long long> done_cache[64][4];  // tiny open-addressing cache
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long key = reinterpret_cast<uintptr_t>(kernel) ^ ((unsigned long long)dev << 56);
    const unsigned h = (unsigned)((key >> 4) * 0x9E3779B1u) & 63u;
    for (auto &slot : done_cache[h])
        if (slot.load(std::memory_order_relaxed) == key) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, device_limits().smem_per_block);
    if (e != cudaSuccess) return e;
    for (auto &slot : done_cache[h]) {
        unsigned long long z = 0;
        if (slot.compare_exchange_strong(z, key)) break;
    }
    return cudaSuccess;
}

// The driver's encoder of tensor maps, looked up once.
using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                                 const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
inline EncodeTiled encode_tiled() {
    static std::atomic<EncodeTiled> found{nullptr};
    EncodeTiled f = found.load(std::memory_order_relaxed);
    if (f) return f;
    void *fn = nullptr;
    cudaDriverEntryPointQueryResult st;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &st) != cudaSuccess ||
        st != cudaDriverEntryPointSuccess) {
        cudaGetLastError();
        return nullptr;
    }
    f = reinterpret_cast<EncodeTiled>(fn);
    found.store(f, std::memory_order_relaxed);
    return f;
}

}  // namespace cvk
