// Host side shared by the entry points that read a tensor list.
#pragma once
#include <hip/hip_runtime.h>

#include "cu_share.h"
#include "internal.h"
#include "list_layout.h"

namespace qm {
namespace {

// Both copies of a list of this kind, checked: where its tables are on the
// device.  h is null on error (st then holds it, message recorded).
struct ListArgs {
    const ListHeader *h = nullptr;
    const ListTensor *tensors = nullptr;
    const int32_t *owner = nullptr;
    qm_status st = QM_OK;
};

ListArgs list_args(const void *host_plan, const void *dev_plan, int kind) {
    ListArgs a;
    const ListHeader *h = list_header(host_plan, kind, &a.st);
    if (!h) return a;
    if (!dev_plan) a.st = fail(QM_E_ARG, "device copy of the list is null");
    else if (!aligned(dev_plan, 64)) a.st = fail(QM_E_ALIGN, "device copy of the list must be 64-byte aligned");
    else {
        const char *dev = static_cast<const char *>(dev_plan);
        a.h = h;
        a.tensors = reinterpret_cast<const ListTensor *>(dev + h->off_tensors);
        a.owner = reinterpret_cast<const int32_t *>(dev + h->off_task_tensor);
    }
    return a;
}

qm_status launched(const char *what) {
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? QM_OK : fail(QM_E_HIP, "%s launch: %s", what, hipGetErrorString(e));
}

}  // namespace
}  // namespace qm
