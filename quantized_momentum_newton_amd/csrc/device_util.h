// Device helpers shared by the streaming kernels: global pointers, lane
// exchange, 16-bit conversions, byte packing, the counter-based random
// numbers.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qm {
namespace {

// ------------------------------------------------------------ global pointers

// A device address as a pointer the compiler knows points to global memory.
// The tensor addresses the plan holds, and the pointers inside argument
// structs, are otherwise generic, and their accesses compile to flat
// instructions: a 64-bit address per lane, and both the vector-memory and
// the LDS counters, so each wait for a lane shuffle's result also waits for
// the outstanding loads and stores.
template <typename T> __device__ __forceinline__ T *gmem(uint64_t a) {
    return (T *)(__attribute__((address_space(1))) T *)a;
}
template <typename T> __device__ __forceinline__ T *gmem(T *p) { return gmem<T>((uint64_t)p); }

// ------------------------------------------------------------ lane exchange

// Lane l's value from lane l ^ k.  For k < 32 (inside l's 32-lane half) a
// ds_swizzle in bit-mask mode, which needs no lane-address register, unlike
// the generic shuffle used for k = 32.  Every lane must be active.
__device__ __forceinline__ int xor_lanes(int v, int k) {
    switch (k) {
        case 1: return __builtin_amdgcn_ds_swizzle(v, 0x041f);
        case 2: return __builtin_amdgcn_ds_swizzle(v, 0x081f);
        case 4: return __builtin_amdgcn_ds_swizzle(v, 0x101f);
        case 8: return __builtin_amdgcn_ds_swizzle(v, 0x201f);
        case 16: return __builtin_amdgcn_ds_swizzle(v, 0x401f);
        default: return __shfl_xor(v, k);
    }
}
__device__ __forceinline__ float xor_lanes(float v, int k) { return __int_as_float(xor_lanes(__float_as_int(v), k)); }
__device__ __forceinline__ double xor_lanes(double v, int k) {
    const uint64_t u = (uint64_t)__double_as_longlong(v);
    const uint32_t lo = (uint32_t)xor_lanes((int)(uint32_t)u, k), hi = (uint32_t)xor_lanes((int)(uint32_t)(u >> 32), k);
    return __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
}

// ------------------------------------------------------------ conversions

// Two fp32 values to packed bf16 (a in the low half), round to nearest even,
// a NaN kept quiet with its sign and top payload bits: gfx950's
// v_cvt_pk_bf16_f32, one instruction for the pair.  It gives the same bits as
// the integer form (add 0x7fff plus the kept lsb, shift; NaN: top half | 0x40)
// for every fp32 input, subnormals and NaNs included (checked exhaustively
// on gfx950).
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t bf16x2_rne(float a, float b) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_t){a, b}, bf16x2_t));
}
__device__ __forceinline__ uint16_t bf16_rne(float f) { return (uint16_t)bf16x2_rne(f, 0.0f); }
__device__ __forceinline__ float bf16_val(uint16_t h) { return __uint_as_float((uint32_t)h << 16); }

__device__ __forceinline__ uint16_t f16_rne(float f) {
    _Float16 h = (_Float16)f;  // v_cvt_f16_f32: round to nearest even
    return __builtin_bit_cast(uint16_t, h);
}
__device__ __forceinline__ float f16_val(uint16_t h) {
    return (float)__builtin_bit_cast(_Float16, h);
}

// Vector types of the non-temporal loads and stores (the builtins take plain
// vector types only).
typedef unsigned ntv4 __attribute__((ext_vector_type(4)));
typedef unsigned ntv2 __attribute__((ext_vector_type(2)));
// ------------------------------------------------------------ bytes and random numbers

// Four codes from byte BYTE of a, b, c, d (a's lowest): three byte permutes.
template <int BYTE> __device__ __forceinline__ uint32_t pack_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    const uint32_t ab = __builtin_amdgcn_perm(b, a, 0x0c0c0400u + 0x0101u * BYTE);   // a, b, 0, 0
    const uint32_t cd = __builtin_amdgcn_perm(d, c, 0x0c0c0400u + 0x0101u * BYTE);   // c, d, 0, 0
    return __builtin_amdgcn_perm(cd, ab, 0x05040100u);                               // a, b, c, d
}
__device__ __forceinline__ uint32_t pack_low_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return pack_bytes<0>(a, b, c, d);
}
// Philox4x32-10 ("Parallel random numbers: as easy as 1, 2, 3", Salmon,
// Moraes, Dror and Shaw, SC 2011).
__device__ __forceinline__ void philox4x32_10(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3, uint32_t k0,
                                              uint32_t k1, uint32_t *out) {
    constexpr uint32_t M0 = 0xD2511F53u, M1 = 0xCD9E8D57u, W0 = 0x9E3779B9u, W1 = 0xBB67AE85u;
#pragma unroll
    for (int r = 0; r < 10; r++) {
        if (r > 0) {
            k0 += W0;
            k1 += W1;
        }
        // each 64-bit product as one v_mad_u64_u32 (both halves), not a
        // separate high and low multiply (32-bit integer multiplies issue at
        // a quarter of the VALU rate)
        const uint64_t p0 = (uint64_t)M0 * c0, p1 = (uint64_t)M1 * c2;
        // 0x96: exclusive or of three, one v_bitop3_b32
        const uint32_t n0 = __builtin_amdgcn_bitop3_b32((uint32_t)(p1 >> 32), c1, k0, 0x96);
        const uint32_t n2 = __builtin_amdgcn_bitop3_b32((uint32_t)(p0 >> 32), c3, k1, 0x96);
        c0 = n0;
        c1 = (uint32_t)p1;
        c2 = n2;
        c3 = (uint32_t)p0;
    }
    out[0] = c0;
    out[1] = c1;
    out[2] = c2;
    out[3] = c3;
}

}  // namespace
}  // namespace qm
