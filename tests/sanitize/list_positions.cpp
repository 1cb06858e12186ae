// Positions of strided gradients, as the list kernels compute them
// (GradPos in list_layout.h), against row * ld + column, element by element:
// random views of every kind (rows of a task's length and more, multiples of 8
// or not, jumps next to the limit of 32-bit offsets), encoded by
// qm_grad_plan_encode and walked group by group as a wave's lanes do.  Built
// with AddressSanitizer and UndefinedBehaviorSanitizer by
// tests/test_list_positions_cpu.py.  Device addresses are fake.
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>

#include <algorithm>
#include <random>
#include <vector>

#include "list_layout.h"
#include "qmuon.h"

using namespace qm;

static long fails = 0;
static long row_ends = 0, far_tasks = 0, cut_groups = 0;

// One group's elements e .. e + n - 1 at positions at, at + 1, ...: inside the
// view, each where its row and column put it.
static void group(const qm_grad_tensor &g, int64_t e, int n, int64_t at) {
    const int64_t span = (g.numel / g.cols - 1) * g.ld + g.cols;
    for (int j = 0; j < n; j++) {
        const int64_t want = (e + j) / g.cols * g.ld + (e + j) % g.cols;
        if (at + j != want || at + j < 0 || at + j >= span) {
            if (fails++ < 10)
                fprintf(stderr, "numel %lld cols %lld ld %lld element %lld: position %lld, not %lld\n", (long long)g.numel,
                        (long long)g.cols, (long long)g.ld, (long long)(e + j), (long long)(at + j), (long long)want);
        }
    }
}

// A whole task, groups of N elements in the lanes (grad_task of list_device.h).
static void whole_task(const qm_grad_tensor &g, const ListTensor &T, int64_t e_task, int N) {
    const GradPos first(T, (uint32_t)e_task);
    const int esz = g.dtype == QM_F32 ? 4 : 2;
    if (first.near_all()) row_ends += first.col + kListTask > first.cols;
    else far_tasks++;
    for (int i = 0; i < kListTask; i += N) {
        const int64_t at = first.near_all() ? first.at + (int64_t)((uint32_t)(first.offset((uint32_t)i) * (uint32_t)esz) / (uint32_t)esz)
                                            : GradPos(T, (uint32_t)e_task + (uint32_t)i).at;
        group(g, e_task + i, N, at);
    }
}

// A block task of n elements, four a lane (load_grad, store_grad).
static void block_task(const qm_grad_tensor &g, const ListTensor &T, int64_t e_task, int n) {
    for (int i = 0; i < n; i += 4) {
        GradPos p(T, (uint32_t)(e_task + i));
        const int k = std::min(4, n - i);
        if (T.grad_cols % 4 == 0) {
            group(g, e_task + i, k, p.at);
            continue;
        }
        cut_groups += (e_task + i) / g.cols != (e_task + i + k - 1) / g.cols;
        for (int j = 0; j < k; j++, p.next()) group(g, e_task + i + j, 1, p.at);
    }
}

int main(int argc, char **argv) {
    const int iters = argc > 1 ? atoi(argv[1]) : 3000;
    std::mt19937_64 rng(2718);
    auto uni = [&](int64_t lo, int64_t hi) { return std::uniform_int_distribution<int64_t>(lo, hi)(rng); };
    long tasks = 0;
    for (int it = 0; it < iters; it++) {
        qm_grad_tensor g = {};
        g.dtype = (int32_t)uni(0, 2);
        const int kind = (int)uni(0, 4);
        g.cols = kind == 0 ? uni(1, 40) : kind == 1 ? 8 * uni(1, 130) : kind == 2 ? 8 * uni(128, 700) : kind == 3 ? uni(200, 3000) : 4 * uni(1, 700);
        const int64_t gap = uni(0, 3) ? uni(1, 2000) : ((int64_t)1 << 28) + uni(-2, 2);
        const int64_t rows = uni(1, std::max<int64_t>(2, 30000 / g.cols));
        g.ld = g.cols + gap;
        g.numel = rows * g.cols;
        g.grad = reinterpret_cast<void *>((uintptr_t)1 << 44);
        size_t size = 0;
        if (qm_grad_plan_encode(&g, 1, nullptr, &size) != QM_OK) { fails++; continue; }
        std::vector<uint64_t> blob((size + 7) / 8);
        if (qm_grad_plan_encode(&g, 1, blob.data(), &size) != QM_OK) { fails++; continue; }
        const char *base = reinterpret_cast<const char *>(blob.data());
        const ListHeader *h = reinterpret_cast<const ListHeader *>(base);
        const ListTensor &T = *reinterpret_cast<const ListTensor *>(base + h->off_tensors);
        if (T.grad_cols == 0) {
            if (rows != 1) fails++;
            continue;
        }
        for (int64_t k = 0; k < h->n_tasks; k++) {
            const int64_t e = list_task_start(T.full_tasks, k);
            tasks++;
            if (k < T.full_tasks) {
                whole_task(g, T, e, 4);
                whole_task(g, T, e, 8);
            } else block_task(g, T, e, (int)std::min<int64_t>(256, T.numel - e));
        }
    }
    // the last rows of a view that ends just below 2^32 elements
    ListTensor T = {};
    qm_grad_tensor g = {};
    for (int64_t cols : {1032, 4096, 65544, 1 << 24, 1000, 8}) {
        g.cols = T.grad_cols = cols;
        g.ld = T.grad_ld = cols + 8;
        g.numel = T.numel = (((int64_t)1 << 32) - 1) / cols * cols;
        T.full_tasks = T.numel / kListTask;
        for (int64_t k = T.full_tasks - 5; k < T.full_tasks; k++) {
            whole_task(g, T, k * kListTask, 4);
            whole_task(g, T, k * kListTask, 8);
        }
        block_task(g, T, T.full_tasks * kListTask, (int)std::min<int64_t>(256, T.numel - T.full_tasks * kListTask));
    }
    printf("%d views, %ld tasks, %ld with a row end, %ld far, %ld cut groups, %ld failed checks\n", iters, tasks, row_ends, far_tasks,
           cut_groups, fails);
    return fails || row_ends < 100 || far_tasks < 100 || cut_groups < 100;
}
