// Argument checks shared by the entry points on activations, gradients of
// products and embeddings (host only).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "internal.h"
#include "overlap.h"
#include "qmuon.h"

namespace qm {
namespace {

constexpr int64_t kMaxSide = (int64_t)1 << 31;     // rows, columns, tokens: indices fit 32 bits
constexpr int64_t kMaxPitch = ((int64_t)1 << 24) - 16;    // 64 rows stay within a 31-bit byte offset

inline int64_t elem_size(int32_t dtype) { return dtype == QM_F32 ? 4 : 2; }
inline bool known_dtype(int32_t dtype) { return dtype == QM_F32 || dtype == QM_BF16 || dtype == QM_F16; }

// A rows x cols matrix of this type with row pitch ld, aligned to its
// elements.  A matrix without elements may be null.
inline qm_status check_matrix(const char *name, const void *p, int32_t dtype, int64_t rows, int64_t cols, int64_t ld) {
    if (!known_dtype(dtype)) return fail(QM_E_DTYPE, "%s: unknown dtype %d", name, dtype);
    if (rows < 0 || cols < 0 || rows >= kMaxSide || cols >= kMaxSide) return fail(QM_E_SHAPE, "%s: bad size", name);
    if (rows == 0 || cols == 0) return QM_OK;
    if (!p) return fail(QM_E_ARG, "%s is null", name);
    if (ld < cols || ld > kMaxPitch) return fail(QM_E_SHAPE, "%s: row pitch below its columns, or above 2^24 - 16", name);
    if (!aligned(p, elem_size(dtype))) return fail(QM_E_ALIGN, "%s must be aligned to its elements", name);
    return QM_OK;
}

inline qm_status check_kept(const char *name, const qm_act8 *k, int64_t rows, int64_t cols) {
    if (!k) return fail(QM_E_ARG, "%s is null", name);
    if (k->rows != rows || k->cols != cols) return fail(QM_E_SHAPE, "%s has another size", name);
    if (rows < 0 || cols < 0 || rows >= kMaxSide || cols >= kMaxSide) return fail(QM_E_SHAPE, "%s: bad size", name);
    if (rows == 0 || cols == 0) return QM_OK;
    if (!k->data || !k->scale) return fail(QM_E_ARG, "%s: null pointer", name);
    if (k->ld < cols || k->ld % 16 || k->ld > kMaxPitch)
        return fail(QM_E_SHAPE, "%s: ld must be a multiple of 16, at least the columns and at most 2^24 - 16", name);
    if (!aligned(k->data, 16) || !aligned(k->scale, 16)) return fail(QM_E_ALIGN, "%s must be 16-byte aligned", name);
    return QM_OK;
}

// Bytes of the buffers of one call: outputs must share none with any other.
class Spans {
  public:
    void matrix(const void *p, int32_t dtype, int64_t rows, int64_t cols, int64_t ld, bool out) {
        if (!p || rows <= 0 || cols <= 0) return;
        const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
        const uintptr_t s = (uintptr_t)elem_size(dtype), row = cols * s, pitch = ld * s;
        add(Region{lo, lo + (rows - 1) * pitch + row, rows > 1 && ld > cols ? pitch : 0, row}, out);
    }
    void bytes(const void *p, int64_t n, bool out) {
        if (!p || n <= 0) return;
        const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
        add(Region{lo, lo + (uintptr_t)n, 0, (uintptr_t)n}, out);
    }
    void kept(const qm_act8 *k, bool out) {
        if (!k) return;
        bytes(k->data, k->rows * k->ld, out);
        bytes(k->scale, (k->rows + 31) / 32 * k->ld, out);
    }
    bool clash() const {
        for (int i = 0; i < n_; i++)
            for (int j = 0; j < i; j++)
                if ((out_[i] || out_[j]) && regions_overlap(at_[i], at_[j])) return true;
        return false;
    }

  private:
    static constexpr int kMost = 12;   // more than any call has
    void add(const Region &r, bool out) {
        at_[n_] = r;
        out_[n_++] = out;
    }
    Region at_[kMost];
    bool out_[kMost];
    int n_ = 0;
};

inline qm_status launch_status(const char *what) {
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? QM_OK : fail(QM_E_HIP, "%s launch: %s", what, hipGetErrorString(e));
}

}  // namespace
}  // namespace qm
