// Byte layout of a tensor-list blob: what the AdamW step and the gradient
// norm read on the device.  The host encoder (list_plan.cpp) writes it, the
// caller copies it verbatim.
//
// The work is cut into tasks of one tensor's consecutive elements, one wave64
// each: 1024 (four 256-element blocks) with 16-byte accesses throughout, and
// one block a task for what is left at the tensor's end, and for the whole
// tensor where a strided gradient's rows are not multiples of 8 elements and
// cut a lane's group.  No wave goes through several such blocks one after the
// other (a list of small tensors is bound by that latency).
// Tasks of tensors with
// 32-bit states come first, then those with 8-bit states, each in list
// order, so that one launch covers one kind.  A table names every task's
// tensor (4 bytes per 1024 elements, one scalar load instead of a search).
#pragma once
#include <stdint.h>

#include "qmuon.h"

namespace qm {

constexpr uint32_t kListMagic = 0x54534c51u;  // "QLST"
constexpr uint32_t kListVersion = 2;
constexpr int kListTask = 1024;
// A launch takes fewer than 2^32 threads: two workgroups of 256 for every four
// tasks in a state read, the largest of the launches.
constexpr int64_t kListMaxTasks = (((int64_t)1 << 32) / (2 * 256) - 1) * 4;
enum { kListGrads = 1, kListAdamW = 2 };

struct ListHeader {
    uint32_t magic, version;
    int32_t kind, n_tensors;
    int64_t n_blocks, total_numel;
    int64_t n_tasks;          // of all tensors
    int64_t n_tasks32;        // tasks [0, n_tasks32): 32-bit states (grad lists: all)
    int64_t n_wide_grad;      // tasks with an fp32 gradient
    int64_t n_wide8;          // tasks with 8-bit states and an fp32 weight
    int64_t off_tensors;      // ListTensor[n_tensors], list order
    int64_t off_task_tensor;  // int32[n_tasks]
    int64_t total_bytes;
};

struct ListTensor {
    uint64_t weight, grad, m, v, m_absmax, v_absmax, copy;  // device addresses
    int64_t numel;
    int64_t grad_cols, grad_ld;   // 0: contiguous
    int64_t task_offset;          // its first task
    int64_t block_offset;         // its first block, list order
    int32_t grad_dtype, weight_dtype, copy_dtype, state_bits;
    float lr_scale, weight_decay;
    int64_t full_tasks;           // tasks of 1024 elements; the others have at most 256
};

// Tasks of a tensor of n elements, `full` of them whole; task k's first element.
constexpr int64_t list_tasks(int64_t n, int64_t full) { return full + (n - full * kListTask + 255) / 256; }
constexpr int64_t list_task_start(int64_t full, int64_t k) { return k < full ? k * kListTask : full * kListTask + (k - full) * 256; }

// Position, in elements, in a strided gradient's buffer (numel < 2^32) of
// element e, by one division, and, step by step, of the elements after it.
struct GradPos {
    int64_t at = 0, jump = 0;
    uint32_t col = 0, cols = 0;
    constexpr GradPos(const ListTensor &T, uint32_t e) {
        cols = (uint32_t)T.grad_cols;
        const uint32_t row = e / cols;
        col = e - row * cols;
        at = (int64_t)row * T.grad_ld + col;
        jump = T.grad_ld - T.grad_cols;
    }
    constexpr void next() {
        at++;
        if (++col == cols) {
            col = 0;
            at += jump;
        }
    }
    // Whether a whole task's positions are 32-bit byte offsets from its first
    // element's (this one): rows of a task's length or more, so that it meets
    // at most one row end, and a jump there that fits.
    constexpr bool near_all() const { return cols >= kListTask && jump < 1 << 28; }
    // Then: from the first element to element i of the task.
    constexpr uint32_t offset(uint32_t i) const { return i + (col + i >= cols ? (uint32_t)jump : 0u); }
};

static_assert(sizeof(ListHeader) == 88, "list header layout");
static_assert(sizeof(ListTensor) == 128, "list tensor layout");

// Reads and checks a host list blob of this kind (0: either); nullptr on
// error (message recorded).
const ListHeader *list_header(const void *host_blob, int kind, qm_status *st);

}  // namespace qm
