// Randomised driver for the tensor-list encoders (qm_grad_plan_encode,
// qm_adamw_plan_encode, qm_list_blocks, the workspace query's reader), built
// with AddressSanitizer and UndefinedBehaviorSanitizer by
// tests/test_sanitizers_lists_cpu.py.  Device addresses are fake.  For every
// list it accepts, the driver walks the task table as the kernels do and
// checks that the tasks cover each tensor's elements once, in order, inside
// its buffers.
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <algorithm>
#include <random>
#include <vector>

#include "list_layout.h"
#include "qmuon.h"

using namespace qm;

static int fails = 0;
#define CHECK(c)                                                         \
    do {                                                                 \
        if (!(c)) {                                                      \
            fprintf(stderr, "check failed line %d: %s\n", __LINE__, #c); \
            fails++;                                                     \
        }                                                                \
    } while (0)

static void walk(const std::vector<uint64_t> &blob, const std::vector<qm_adamw_tensor> &t, int kind) {
    const char *base = reinterpret_cast<const char *>(blob.data());
    const ListHeader *h = reinterpret_cast<const ListHeader *>(base);
    const ListTensor *T = reinterpret_cast<const ListTensor *>(base + h->off_tensors);
    const int32_t *owner = reinterpret_cast<const int32_t *>(base + h->off_task_tensor);
    CHECK(h->kind == kind && h->n_tensors == (int32_t)t.size());
    CHECK(h->total_bytes <= (int64_t)(blob.size() * 8));
    std::vector<int64_t> at(t.size(), 0);   // elements covered so far
    int64_t blocks = 0;
    for (size_t i = 0; i < t.size(); i++) {
        CHECK(T[i].numel == t[i].numel && T[i].block_offset == blocks);
        blocks += (t[i].numel + 255) / 256;
    }
    CHECK(h->n_blocks == blocks && qm_list_blocks(base) == blocks);
    for (int64_t k = 0; k < h->n_tasks; k++) {
        const int32_t i = owner[k];
        CHECK(i >= 0 && i < h->n_tensors);
        if (i < 0 || i >= h->n_tensors) return;
        CHECK((T[i].state_bits == 32) == (k < h->n_tasks32));
        const int64_t lt = k - T[i].task_offset, e = list_task_start(T[i].full_tasks, lt);
        const int64_t n = lt < T[i].full_tasks ? kListTask : std::min(T[i].numel - e, (int64_t)256);
        CHECK(e == at[i] && n > 0 && e % 256 == 0);
        if (n == kListTask && T[i].grad_cols) CHECK(T[i].grad_cols % 8 == 0);
        at[i] += n;
    }
    for (size_t i = 0; i < t.size(); i++) CHECK(at[i] == t[i].numel);
}

int main(int argc, char **argv) {
    const int iters = argc > 1 ? atoi(argv[1]) : 3000;
    std::mt19937_64 rng(54321);
    auto uni = [&](int64_t lo, int64_t hi) { return std::uniform_int_distribution<int64_t>(lo, hi)(rng); };
    int accepted = 0;
    for (int it = 0; it < iters; it++) {
        const int nt = (int)uni(1, 7);
        const bool grads = uni(0, 2) == 0;
        std::vector<qm_adamw_tensor> t(nt);
        std::vector<qm_grad_tensor> g(nt);
        uintptr_t addr = (uintptr_t)1 << 40;
        auto take = [&](int64_t bytes) {
            const uintptr_t a = addr;
            addr += (uintptr_t)(bytes / 4096 + 2) * 4096;
            return reinterpret_cast<void *>(a + (uni(0, 60) == 0 ? 1 : 4 * (uintptr_t)uni(0, 3)));
        };
        for (int i = 0; i < nt; i++) {
            const int64_t n = uni(0, 12) == 0 ? uni(-1, 3) : uni(1, 9000), nb = (n + 255) / 256;
            memset(&t[i], 0, sizeof t[i]);
            t[i].numel = n;
            t[i].grad_dtype = (int32_t)(uni(0, 40) == 0 ? uni(-2, 5) : uni(0, 2));
            t[i].weight_dtype = (int32_t)(uni(0, 40) == 0 ? uni(-2, 5) : uni(0, 2));
            t[i].state_bits = uni(0, 40) == 0 ? 16 : uni(0, 1) ? 8 : 32;
            t[i].lr_scale = 1.0f;
            t[i].weight = take(4 * n);
            t[i].m = take(4 * n);
            t[i].v = take(4 * n);
            if (t[i].state_bits == 8) {
                t[i].m_absmax = static_cast<float *>(take(4 * nb));
                t[i].v_absmax = static_cast<float *>(take(4 * nb));
            }
            if (uni(0, 2) == 0) {
                t[i].copy = take(2 * n);
                t[i].copy_dtype = (int32_t)uni(0, 10) == 0 ? QM_F32 : QM_BF16;
            }
            if (n > 0 && uni(0, 2) == 0) {
                int64_t cols = uni(1, 40);
                while (n % cols) cols--;
                t[i].grad_cols = uni(0, 20) == 0 ? uni(-4, 60) : cols;
                t[i].grad_ld = cols + uni(-1, 20);
            }
            t[i].grad = take(4 * (n > 0 ? n : 1) * 64);
            if (i > 0 && uni(0, 40) == 0) t[i].grad = t[i - 1].grad;
            g[i] = {const_cast<void *>(t[i].grad), n, t[i].grad_cols, t[i].grad_ld, t[i].grad_dtype, 0};
        }
        size_t size = 0;
        auto enc = [&](void *out) {
            return grads ? qm_grad_plan_encode(g.data(), nt, out, &size) : qm_adamw_plan_encode(t.data(), nt, out, &size);
        };
        if (enc(nullptr) != QM_OK) {
            CHECK(qm_last_error()[0] != 0);
            continue;
        }
        std::vector<uint64_t> blob((size + 7) / 8, ~0ull);
        CHECK(enc(blob.data()) == QM_OK);
        accepted++;
        if (grads) for (auto &x : t) x.state_bits = 32;
        walk(blob, t, grads ? kListGrads : kListAdamW);
        size = size > 64 ? size - 1 : size;
        if (enc(blob.data()) == QM_OK) CHECK(false);
    }
    CHECK(accepted > iters / 10);
    printf("%d lists, %d accepted, %d failed checks\n", iters, accepted, fails);
    return fails ? 1 : 0;
}
