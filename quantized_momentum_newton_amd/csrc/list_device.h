// Device side of the tensor lists: a lane's groups of elements of any type,
// and where a task's elements lie.
#pragma once
#include "device_util.h"
#include "list_layout.h"

namespace qm {
namespace {

// N consecutive elements of one lane, still packed, loaded in 16-byte pieces
// (8 for four 16-bit elements, 4 or 8 for N codes).  The vector types carry no
// alignment: gfx950 takes unaligned vector accesses, so a tensor may start at
// any element of its buffer and aligned ones lose nothing.  Where `base` is
// uniform over the wave and `off` a 32-bit byte offset, an access is one
// scalar base plus one vector register.
template <int BYTES> struct Packed { unsigned w[BYTES / 4]; };
typedef unsigned u32x4_e __attribute__((ext_vector_type(4), aligned(1)));
typedef unsigned u32x2_e __attribute__((ext_vector_type(2), aligned(1)));
typedef unsigned u32_e __attribute__((aligned(1)));

template <int BYTES> __device__ __forceinline__ Packed<BYTES> load_bytes(uint64_t base, uint32_t off) {
    Packed<BYTES> r;
    const char *p = gmem<const char>(base) + off;
    if constexpr (BYTES % 16 == 0) {
#pragma unroll
        for (int k = 0; k < BYTES / 16; k++) {
            const u32x4_e v = __builtin_nontemporal_load(reinterpret_cast<const u32x4_e *>(p + 16 * k));
            r.w[4 * k] = v.x; r.w[4 * k + 1] = v.y; r.w[4 * k + 2] = v.z; r.w[4 * k + 3] = v.w;
        }
    } else if constexpr (BYTES == 8) {
        const u32x2_e v = __builtin_nontemporal_load(reinterpret_cast<const u32x2_e *>(p));
        r.w[0] = v.x; r.w[1] = v.y;
    } else {
        static_assert(BYTES == 4, "piece size");
        r.w[0] = __builtin_nontemporal_load(reinterpret_cast<const u32_e *>(p));
    }
    return r;
}
template <int BYTES> __device__ __forceinline__ void store_bytes(uint64_t base, uint32_t off, const Packed<BYTES> &r) {
    char *p = gmem<char>(base) + off;
    if constexpr (BYTES % 16 == 0) {
#pragma unroll
        for (int k = 0; k < BYTES / 16; k++) {
            const u32x4_e v = {r.w[4 * k], r.w[4 * k + 1], r.w[4 * k + 2], r.w[4 * k + 3]};
            __builtin_nontemporal_store(v, reinterpret_cast<u32x4_e *>(p + 16 * k));
        }
    } else if constexpr (BYTES == 8) {
        const u32x2_e v = {r.w[0], r.w[1]};
        __builtin_nontemporal_store(v, reinterpret_cast<u32x2_e *>(p));
    } else {
        __builtin_nontemporal_store(r.w[0], reinterpret_cast<u32_e *>(p));
    }
}
template <int DT> constexpr int kSizeOf = DT == QM_F32 ? 4 : 2;
template <int DT, int N> using PackedOf = Packed<N * kSizeOf<DT>>;

template <int DT, int BYTES> __device__ __forceinline__ float unpack(const Packed<BYTES> &r, int j) {
    if constexpr (DT == QM_F32) return __uint_as_float(r.w[j]);
    else {
        const uint16_t h = (uint16_t)(r.w[j / 2] >> (16 * (j % 2)));
        return DT == QM_BF16 ? bf16_val(h) : f16_val(h);
    }
}
// x as the fp32 number it is.  The empty asm keeps a conversion to f16 apart
// from the product or sum that made x: fused into one instruction
// (v_fma_mixlo_f16) they round once, and a result next to a border of f16
// depends on whether the compiler fused.
__device__ __forceinline__ float in_fp32(float x) {
    asm("" : "+v"(x));
    return x;
}
template <int DT, int N> __device__ __forceinline__ PackedOf<DT, N> pack(const float *x) {
    PackedOf<DT, N> r;
#pragma unroll
    for (int j = 0; j < N; j++) {
        if constexpr (DT == QM_F32) r.w[j] = __float_as_uint(x[j]);
        else if (j % 2 == 0) {
            if constexpr (DT == QM_BF16) r.w[j / 2] = bf16x2_rne(x[j], x[j + 1]);
            else r.w[j / 2] = (unsigned)f16_rne(x[j]) | ((unsigned)f16_rne(x[j + 1]) << 16);
        }
    }
    return r;
}

// The same of four elements at a tensor's end, of which n are inside
// (0 <= n <= 4; zeros for the others, which are not stored).
template <int DT> __device__ __forceinline__ PackedOf<DT, 4> load_edge(uint64_t base, int64_t e, int n) {
    if (n == 4) return load_bytes<4 * kSizeOf<DT>>(base + (uint64_t)e * kSizeOf<DT>, 0);
    PackedOf<DT, 4> r = {};
#pragma unroll
    for (int j = 0; j < 4; j++) {
        if (j >= n) continue;
        if constexpr (DT == QM_F32) r.w[j] = gmem<const uint32_t>(base)[e + j];
        else r.w[j / 2] |= (unsigned)gmem<const uint16_t>(base)[e + j] << (16 * (j % 2));
    }
    return r;
}
template <int DT> __device__ __forceinline__ void store_one(uint64_t base, int64_t e, float x) {
    if constexpr (DT == QM_F32) gmem<float>(base)[e] = x;
    else gmem<uint16_t>(base)[e] = DT == QM_BF16 ? bf16_rne(x) : f16_rne(x);
}
template <int DT> __device__ __forceinline__ void store_edge(uint64_t base, int64_t e, int n, const float *x) {
    if (n == 4) {
        store_bytes(base + (uint64_t)e * kSizeOf<DT>, 0, pack<DT, 4>(x));
        return;
    }
#pragma unroll
    for (int j = 0; j < 4; j++)
        if (j < n) store_one<DT>(base, e + j, x[j]);
}

// First element of the tensor's task k, and how many it has: 1024, or at most
// 256.
__device__ __forceinline__ int64_t task_start(const ListTensor &T, int64_t k, int &count) {
    const int64_t e = list_task_start(T.full_tasks, k);
    count = k < T.full_tasks ? kListTask : (int)min(T.numel - e, (int64_t)256);
    return e;
}

// Calls access(p, base, off) for a lane's groups of N elements in a whole task
// of the gradient, group p at element p * 64 N + lane * N: base and byte
// offset of its first element (a group lies in one row).  Where a task meets
// at most one row end, one scalar division serves the wave; the last branch
// divides per group.
template <int DT, int N, int PARTS, typename Access>
__device__ __forceinline__ void grad_task(const ListTensor &T, int64_t e_task, int lane, Access access) {
    constexpr int S = kSizeOf<DT>;
    if (T.grad_cols == 0) {
#pragma unroll
        for (int p = 0; p < PARTS; p++) access(p, T.grad + (uint64_t)e_task * S, (uint32_t)(p * 64 + lane) * N * S);
        return;
    }
    const GradPos first(T, (uint32_t)e_task);
    if (first.near_all()) {
#pragma unroll
        for (int p = 0; p < PARTS; p++) access(p, T.grad + (uint64_t)first.at * S, first.offset((p * 64 + lane) * N) * S);
    } else {
#pragma unroll
        for (int p = 0; p < PARTS; p++) access(p, T.grad + (uint64_t)GradPos(T, (uint32_t)e_task + (p * 64 + lane) * N).at * S, 0);
    }
}

template <int DT, int N, int PARTS>
__device__ __forceinline__ void load_grad_task(const ListTensor &T, int64_t e_task, int lane, PackedOf<DT, N> *r) {
    grad_task<DT, N, PARTS>(T, e_task, lane, [&](int p, uint64_t base, uint32_t off) { r[p] = load_bytes<N * kSizeOf<DT>>(base, off); });
}
template <int DT, int N, int PARTS>
__device__ __forceinline__ void store_grad_task(const ListTensor &T, int64_t e_task, int lane, const PackedOf<DT, N> *r) {
    grad_task<DT, N, PARTS>(T, e_task, lane, [&](int p, uint64_t base, uint32_t off) { store_bytes(base, off, r[p]); });
}

// Elements e .. e + n - 1 of the gradient, n <= 4.
template <int DT> __device__ __forceinline__ PackedOf<DT, 4> load_grad(const ListTensor &T, int64_t e, int n) {
    if (T.grad_cols == 0) return load_edge<DT>(T.grad, e, n);
    GradPos p(T, (uint32_t)e);
    if (T.grad_cols % 4 == 0) return load_edge<DT>(T.grad, p.at, n);   // in one row
    PackedOf<DT, 4> r = {};
#pragma unroll
    for (int j = 0; j < 4; j++, p.next()) {
        if (j >= n) continue;
        if constexpr (DT == QM_F32) r.w[j] = gmem<const uint32_t>(T.grad)[p.at];
        else r.w[j / 2] |= (unsigned)gmem<const uint16_t>(T.grad)[p.at] << (16 * (j % 2));
    }
    return r;
}
template <int DT> __device__ __forceinline__ void store_grad(const ListTensor &T, int64_t e, int n, const float *x) {
    if (T.grad_cols == 0) {
        store_edge<DT>(T.grad, e, n, x);
        return;
    }
    GradPos p(T, (uint32_t)e);
    if (T.grad_cols % 4 == 0) {
        store_edge<DT>(T.grad, p.at, n, x);
        return;
    }
#pragma unroll
    for (int j = 0; j < 4; j++, p.next())
        if (j < n) store_one<DT>(T.grad, p.at, x[j]);
}

}  // namespace
}  // namespace qm
