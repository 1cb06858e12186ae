// Device side of the tensor lists: groups of four elements of any type,
// loaded and stored at element alignment.
#pragma once
#include "device_util.h"
#include "list_layout.h"

namespace qm {
namespace {

// Four elements as loaded, still packed: 16 bytes of fp32, 8 of 16-bit
// types, 4 of codes.  The vector types carry the elements' alignment only:
// gfx950 takes unaligned vector accesses, so a tensor may start at any
// element of its buffer and aligned ones lose nothing.
typedef unsigned u32x4_e __attribute__((ext_vector_type(4), aligned(4)));
typedef unsigned u32x2_e __attribute__((ext_vector_type(2), aligned(2)));
typedef unsigned u32_e __attribute__((aligned(1)));

template <int DT> struct Raw4 { unsigned w[DT == QM_F32 ? 4 : 2]; };

template <int DT> __device__ __forceinline__ Raw4<DT> load4(uint64_t base, int64_t e) {
    Raw4<DT> r;
    if constexpr (DT == QM_F32) {
        const u32x4_e v = __builtin_nontemporal_load(gmem<const u32x4_e>(base + (uint64_t)e * 4));
        r.w[0] = v.x; r.w[1] = v.y; r.w[2] = v.z; r.w[3] = v.w;
    } else {
        const u32x2_e v = __builtin_nontemporal_load(gmem<const u32x2_e>(base + (uint64_t)e * 2));
        r.w[0] = v.x; r.w[1] = v.y;
    }
    return r;
}
// The first n of four elements (0 <= n <= 4), zeros for the others.
template <int DT> __device__ __forceinline__ Raw4<DT> load_upto4(uint64_t base, int64_t e, int n) {
    Raw4<DT> r = {};
#pragma unroll
    for (int j = 0; j < 4; j++) {
        if (j >= n) continue;
        if constexpr (DT == QM_F32) r.w[j] = *gmem<const uint32_t>(base + (uint64_t)(e + j) * 4);
        else r.w[j / 2] |= (unsigned)*gmem<const uint16_t>(base + (uint64_t)(e + j) * 2) << (16 * (j % 2));
    }
    return r;
}
template <int DT> __device__ __forceinline__ float elem(const Raw4<DT> &r, int j) {
    if constexpr (DT == QM_F32) return __uint_as_float(r.w[j]);
    else {
        const uint16_t h = (uint16_t)(r.w[j / 2] >> (16 * (j % 2)));
        return DT == QM_BF16 ? bf16_val(h) : f16_val(h);
    }
}

template <int DT> __device__ __forceinline__ void store4(uint64_t base, int64_t e, const float *x) {
    if constexpr (DT == QM_F32) {
        const u32x4_e v = {__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3])};
        __builtin_nontemporal_store(v, gmem<u32x4_e>(base + (uint64_t)e * 4));
    } else {
        u32x2_e v;
        if constexpr (DT == QM_BF16) {
            v.x = bf16x2_rne(x[0], x[1]);
            v.y = bf16x2_rne(x[2], x[3]);
        } else {
            v.x = (unsigned)f16_rne(x[0]) | ((unsigned)f16_rne(x[1]) << 16);
            v.y = (unsigned)f16_rne(x[2]) | ((unsigned)f16_rne(x[3]) << 16);
        }
        __builtin_nontemporal_store(v, gmem<u32x2_e>(base + (uint64_t)e * 2));
    }
}
template <int DT> __device__ __forceinline__ void store1(uint64_t base, int64_t e, float x) {
    if constexpr (DT == QM_F32) *gmem<float>(base + (uint64_t)e * 4) = x;
    else if constexpr (DT == QM_BF16) *gmem<uint16_t>(base + (uint64_t)e * 2) = bf16_rne(x);
    else *gmem<uint16_t>(base + (uint64_t)e * 2) = f16_rne(x);
}
template <int DT> __device__ __forceinline__ void store_upto4(uint64_t base, int64_t e, int n, const float *x) {
    if (n == 4) {
        store4<DT>(base, e, x);
        return;
    }
#pragma unroll
    for (int j = 0; j < 4; j++)
        if (j < n) store1<DT>(base, e + j, x[j]);
}

// Position in its buffer of element e of a strided gradient (numel < 2^32).
__device__ __forceinline__ int64_t grad_pos(const ListTensor &T, int64_t e) {
    const uint32_t c = (uint32_t)T.grad_cols, u = (uint32_t)e, r = u / c;
    return (int64_t)r * T.grad_ld + (int64_t)(u - r * c);
}

// Elements e .. e + n - 1 of the gradient, n <= 4.
template <int DT> __device__ __forceinline__ Raw4<DT> load_grad(const ListTensor &T, int64_t e, int n) {
    if (T.grad_cols == 0 || T.grad_cols % 4 == 0) {   // four elements never straddle two rows
        const int64_t p = T.grad_cols == 0 ? e : grad_pos(T, e);
        return n == 4 ? load4<DT>(T.grad, p) : load_upto4<DT>(T.grad, p, n);
    }
    Raw4<DT> r = {};
#pragma unroll
    for (int j = 0; j < 4; j++) {
        if (j >= n) continue;
        const int64_t p = grad_pos(T, e + j);
        if constexpr (DT == QM_F32) r.w[j] = *gmem<const uint32_t>(T.grad + (uint64_t)p * 4);
        else r.w[j / 2] |= (unsigned)*gmem<const uint16_t>(T.grad + (uint64_t)p * 2) << (16 * (j % 2));
    }
    return r;
}
template <int DT> __device__ __forceinline__ void store_grad(const ListTensor &T, int64_t e, int n, const float *x) {
    if (T.grad_cols == 0 || T.grad_cols % 4 == 0) {
        store_upto4<DT>(T.grad, T.grad_cols == 0 ? e : grad_pos(T, e), n, x);
        return;
    }
#pragma unroll
    for (int j = 0; j < 4; j++)
        if (j < n) store1<DT>(T.grad, grad_pos(T, e + j), x[j]);
}

}  // namespace
}  // namespace qm
