// qnn_internal.h -- host-side helpers shared by the library's translation units.
#pragma once
#include <atomic>
#include <cstdint>
#include <cuda_runtime.h>
#include "qnn.h"

namespace qnn {

// Device address of the status word that kernels set when a bounded wait
// gives up, for the current device (looked up once per device); nullptr if
// the lookup failed.
uint32_t *status_word();

// Number of SMs of the current device (cached per device).
int sm_count();

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Lets `kern` take `bytes` of dynamic shared memory on the current device, and asks for
// `carveout` percent of the SM's memory as shared memory (-1: the driver's choice);
// `done` keeps the devices on which that was done, so that later calls only look.
template <typename K>
bool opt_in_smem(K kern, int bytes, std::atomic<uint64_t> &done, int carveout = -1)
{
    int d = -1;
    if (cudaGetDevice(&d) != cudaSuccess || d < 0) return false;
    const uint64_t bit = d < 64 ? 1ull << d : 0;
    if (done.load(std::memory_order_relaxed) & bit) return true;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess ||
        cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, carveout) != cudaSuccess) {
        (void)cudaGetLastError();
        return false;
    }
    done.fetch_or(bit, std::memory_order_relaxed);
    return true;
}

// Maps the launch error (if any) of the last kernel launch to a status.
inline qnn_status launch_status()
{
    return cudaGetLastError() == cudaSuccess ? QNN_OK : QNN_ERR_CUDA;
}

// Code range of a quantized type.
inline bool qrange(int dt, int narrow, int32_t *lo, int32_t *hi)
{
    switch (dt) {
    case QNN_S8: *lo = narrow ? -127 : -128; *hi = 127; return true;
    case QNN_U8: *lo = 0; *hi = 255; return true;
    case QNN_S4: *lo = narrow ? -7 : -8; *hi = 7; return true;
    case QNN_U4: *lo = 0; *hi = 15; return true;
    default: return false;
    }
}

}  // namespace qnn
