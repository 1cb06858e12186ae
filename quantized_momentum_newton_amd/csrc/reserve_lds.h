// Dynamic LDS past the default limit (host only).
#pragma once
#include <hip/hip_runtime.h>

#include <atomic>

#include "internal.h"

namespace qm {
namespace {

constexpr int kMaxDevices = 64;

// Raises a kernel's dynamic LDS limit to `bytes` on the current device, once
// per device (done[] indexed by device; devices beyond the table are set on
// every call).
qm_status reserve_lds(const void *kern, size_t bytes, std::atomic<bool> *done) {
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess) return fail(QM_E_HIP, "no current device");
    const bool cached = dev >= 0 && dev < kMaxDevices;
    if (cached && done[dev].load(std::memory_order_acquire)) return QM_OK;
    if (hipFuncSetAttribute(kern, hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) != hipSuccess)
        return fail(QM_E_HIP, "cannot reserve %zu bytes of LDS", bytes);
    if (cached) done[dev].store(true, std::memory_order_release);
    return QM_OK;
}

}  // namespace
}  // namespace qm
