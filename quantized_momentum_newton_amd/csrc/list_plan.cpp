// Host side of the tensor lists (AdamW, gradient norm): validation and
// encoding, no HIP calls.
#include <math.h>
#include <string.h>

#include <exception>
#include <vector>

#include "internal.h"
#include "list_layout.h"
#include "overlap.h"
#include "plan_layout.h"

namespace qm {

const ListHeader *list_header(const void *host_blob, int kind, qm_status *st) {
    if (!host_blob) {
        *st = fail(QM_E_ARG, "host list is null");
        return nullptr;
    }
    if (!aligned(host_blob, 8)) {
        *st = fail(QM_E_ALIGN, "host list must be 8-byte aligned");
        return nullptr;
    }
    const ListHeader *h = static_cast<const ListHeader *>(host_blob);
    if (h->magic != kListMagic || h->version != kListVersion ||
        (kind ? h->kind != kind : h->kind != kListGrads && h->kind != kListAdamW)) {
        *st = fail(QM_E_PLAN, "not %s blob of version %u",
                   kind == kListGrads ? "a grad list" : kind == kListAdamW ? "an AdamW list" : "a tensor list", kListVersion);
        return nullptr;
    }
    *st = QM_OK;
    return h;
}

namespace {

int64_t dtype_size(int32_t dt) { return dt == QM_F32 ? 4 : dt == QM_BF16 || dt == QM_F16 ? 2 : 0; }

// A contiguous buffer: non-null, aligned to its element, inside the address
// space.  Adds its span.
qm_status check_buffer(int32_t i, const char *what, const void *p, int64_t count, int64_t esz, std::vector<Region> &spans) {
    if (!p) return fail(QM_E_ARG, "tensor %d: %s is null", i, what);
    if (!aligned(p, (uintptr_t)esz)) return fail(QM_E_ALIGN, "tensor %d: %s needs %d-byte alignment", i, what, (int)esz);
    const uintptr_t a = (uintptr_t)p, bytes = (uintptr_t)(count * esz);
    if (a + bytes < a) return fail(QM_E_ARG, "tensor %d: %s runs past the address space", i, what);
    spans.push_back({a, a + bytes, 0, 0});
    return QM_OK;
}

// A gradient, contiguous or a 2-D view.
qm_status check_grad(int32_t i, const void *p, int32_t dtype, int64_t numel, int64_t cols, int64_t ld,
                     std::vector<Region> &spans) {
    const int64_t esz = dtype_size(dtype);
    if (!esz) return fail(QM_E_DTYPE, "tensor %d: unknown grad dtype %d", i, dtype);
    if (cols == 0) return check_buffer(i, "grad", p, numel, esz, spans);
    if (!p) return fail(QM_E_ARG, "tensor %d: grad is null", i);
    if (!aligned(p, (uintptr_t)esz)) return fail(QM_E_ALIGN, "tensor %d: grad needs %d-byte alignment", i, (int)esz);
    if (cols < 0 || numel % cols != 0) return fail(QM_E_SHAPE, "tensor %d: grad columns must be positive and divide numel", i);
    if (ld < cols) return fail(QM_E_SHAPE, "tensor %d: grad pitch below its columns", i);
    if (numel >= (int64_t)1 << 32) return fail(QM_E_UNSUPPORTED, "tensor %d: strided grad too large", i);
    const int64_t rows = numel / cols;
    if (ld > ((int64_t)1 << 56) / (rows * esz)) return fail(QM_E_SHAPE, "tensor %d: grad pitch too large", i);
    const uintptr_t g = (uintptr_t)p, span = (uintptr_t)(((rows - 1) * ld + cols) * esz);
    if (g + span < g) return fail(QM_E_ARG, "tensor %d: grad runs past the address space", i);
    spans.push_back({g, g + span, (uintptr_t)(ld * esz), (uintptr_t)(cols * esz)});
    return QM_OK;
}

qm_status check_numel(int32_t i, int64_t numel) {
    if (numel < 0) return fail(QM_E_ARG, "tensor %d: numel must not be negative", i);
    if (numel > (int64_t)1 << 41) return fail(QM_E_UNSUPPORTED, "tensor %d: too large", i);
    return QM_OK;
}

// Checks one tensor and fills its table entry (addresses, sizes, types).
qm_status take(int32_t i, const qm_grad_tensor &t, ListTensor &e, std::vector<Region> &spans) {
    if (qm_status st = check_numel(i, t.numel)) return st;
    if (t.reserved != 0) return fail(QM_E_ARG, "tensor %d: reserved field must be 0", i);
    if (!dtype_size(t.dtype)) return fail(QM_E_DTYPE, "tensor %d: unknown grad dtype %d", i, t.dtype);
    e.numel = t.numel;
    e.grad_dtype = t.dtype;
    e.state_bits = 32;
    if (t.numel == 0) return QM_OK;
    if (qm_status st = check_grad(i, t.grad, t.dtype, t.numel, t.cols, t.ld, spans)) return st;
    e.grad = (uint64_t)(uintptr_t)t.grad;
    // one row, or rows that follow each other: contiguous
    if (t.cols != 0 && t.cols != t.numel && t.ld != t.cols) {
        e.grad_cols = t.cols;
        e.grad_ld = t.ld;
    }
    return QM_OK;
}

qm_status take(int32_t i, const qm_adamw_tensor &t, ListTensor &e, std::vector<Region> &spans) {
    const int64_t wsz = dtype_size(t.weight_dtype);
    if (!wsz) return fail(QM_E_DTYPE, "tensor %d: unknown weight dtype %d", i, t.weight_dtype);
    if (t.state_bits != 32 && t.state_bits != 8) return fail(QM_E_DTYPE, "tensor %d: states have 32 or 8 bits, not %d", i, t.state_bits);
    if (t.copy && t.copy_dtype != QM_BF16 && t.copy_dtype != QM_F16)
        return fail(QM_E_DTYPE, "tensor %d: a copy is bf16 or f16", i);
    if (!isfinite(t.lr_scale) || !isfinite(t.weight_decay))
        return fail(QM_E_ARG, "tensor %d: lr_scale and weight_decay must be finite", i);
    if (t.state_bits == 32 && (t.m_absmax || t.v_absmax))
        return fail(QM_E_ARG, "tensor %d: 32-bit states have no absmax", i);
    const qm_grad_tensor g = {const_cast<void *>(t.grad), t.numel, t.grad_cols, t.grad_ld, t.grad_dtype, 0};
    if (qm_status st = take(i, g, e, spans)) return st;
    e.weight_dtype = t.weight_dtype;
    e.copy_dtype = t.copy ? t.copy_dtype : 0;
    e.state_bits = t.state_bits;
    e.lr_scale = t.lr_scale;
    e.weight_decay = t.weight_decay;
    if (t.numel == 0) return QM_OK;
    const int64_t ssz = t.state_bits == 32 ? 4 : 1, nb = (t.numel + kBlock - 1) / kBlock;
    if (qm_status st = check_buffer(i, "weight", t.weight, t.numel, wsz, spans)) return st;
    if (qm_status st = check_buffer(i, "m", t.m, t.numel, ssz, spans)) return st;
    if (qm_status st = check_buffer(i, "v", t.v, t.numel, ssz, spans)) return st;
    if (t.state_bits == 8) {
        if (qm_status st = check_buffer(i, "m_absmax", t.m_absmax, nb, 4, spans)) return st;
        if (qm_status st = check_buffer(i, "v_absmax", t.v_absmax, nb, 4, spans)) return st;
    }
    if (t.copy)
        if (qm_status st = check_buffer(i, "copy", t.copy, t.numel, 2, spans)) return st;
    e.weight = (uint64_t)(uintptr_t)t.weight;
    e.m = (uint64_t)(uintptr_t)t.m;
    e.v = (uint64_t)(uintptr_t)t.v;
    e.m_absmax = (uint64_t)(uintptr_t)t.m_absmax;
    e.v_absmax = (uint64_t)(uintptr_t)t.v_absmax;
    e.copy = (uint64_t)(uintptr_t)t.copy;
    return QM_OK;
}

template <typename Tensor>
qm_status encode(const Tensor *tensors, int32_t n, int kind, void *host_blob, size_t *inout_blob_bytes) {
    clear_error();
    if (!tensors || n <= 0) return fail(QM_E_ARG, "no tensors");
    if (!inout_blob_bytes) return fail(QM_E_ARG, "inout_blob_bytes is null");
    try {
        std::vector<Region> spans;
        std::vector<ListTensor> table((size_t)n);
        ListHeader h = {};
        int64_t tasks[2] = {0, 0};   // of 32-bit and of 8-bit states
        for (int32_t i = 0; i < n; i++) {
            ListTensor &e = table[(size_t)i];
            e = ListTensor{};
            if (qm_status st = take(i, tensors[i], e, spans)) return st;
            e.block_offset = h.n_blocks;
            h.n_blocks += (e.numel + kBlock - 1) / kBlock;
            h.total_numel += e.numel;
            int64_t &k = tasks[e.state_bits == 8];
            e.task_offset = k;
            e.full_tasks = e.grad_cols % 8 == 0 ? e.numel / kListTask : 0;
            const int64_t nt = list_tasks(e.numel, e.full_tasks);
            k += nt;
            if (e.grad_dtype == QM_F32) h.n_wide_grad += nt;
            if (e.state_bits == 8 && e.weight_dtype == QM_F32) h.n_wide8 += nt;
        }
        if (any_overlap(spans)) return fail(QM_E_ARG, "buffers of the list overlap");
        h.magic = kListMagic;
        h.version = kListVersion;
        h.kind = kind;
        h.n_tensors = n;
        h.n_tasks32 = tasks[0];
        h.n_tasks = tasks[0] + tasks[1];
        if (h.n_tasks > kListMaxTasks) return fail(QM_E_UNSUPPORTED, "list too large");
        h.off_tensors = align_up(sizeof(ListHeader), 128);
        h.off_task_tensor = h.off_tensors + (int64_t)n * (int64_t)sizeof(ListTensor);
        h.total_bytes = align_up(h.off_task_tensor + h.n_tasks * 4, 64);
        if (!host_blob) {
            *inout_blob_bytes = (size_t)h.total_bytes;
            return QM_OK;
        }
        if (*inout_blob_bytes < (size_t)h.total_bytes)
            return fail(QM_E_ARG, "blob buffer too small: need %lld bytes", (long long)h.total_bytes);
        if (!aligned(host_blob, 8)) return fail(QM_E_ALIGN, "host blob must be 8-byte aligned");
        char *base = static_cast<char *>(host_blob);
        memset(base, 0, (size_t)h.off_tensors);
        memset(base + h.off_task_tensor, 0, (size_t)(h.total_bytes - h.off_task_tensor));
        int32_t *owner = reinterpret_cast<int32_t *>(base + h.off_task_tensor);
        for (int32_t i = 0; i < n; i++) {
            ListTensor &e = table[(size_t)i];
            if (e.state_bits == 8) e.task_offset += tasks[0];
            const int64_t nt = list_tasks(e.numel, e.full_tasks);
            for (int64_t k = 0; k < nt; k++) owner[e.task_offset + k] = i;
        }
        memcpy(base, &h, sizeof h);
        memcpy(base + h.off_tensors, table.data(), table.size() * sizeof(ListTensor));
        *inout_blob_bytes = (size_t)h.total_bytes;
        return QM_OK;
    } catch (const std::exception &) {   // no C++ exception leaves a C entry
        return fail(QM_E_ARG, "out of host memory for a list of %d tensors", n);
    }
}

}  // namespace
}  // namespace qm

using namespace qm;

extern "C" qm_status qm_grad_plan_encode(const qm_grad_tensor *grads, int32_t n_grads, void *host_blob,
                                         size_t *inout_blob_bytes) {
    return encode(grads, n_grads, kListGrads, host_blob, inout_blob_bytes);
}

extern "C" qm_status qm_adamw_plan_encode(const qm_adamw_tensor *tensors, int32_t n_tensors, void *host_blob,
                                          size_t *inout_blob_bytes) {
    return encode(tensors, n_tensors, kListAdamW, host_blob, inout_blob_bytes);
}

extern "C" int64_t qm_list_blocks(const void *host_plan) {
    clear_error();
    qm_status st;
    const ListHeader *h = list_header(host_plan, 0, &st);
    return h ? h->n_blocks : -1;
}
