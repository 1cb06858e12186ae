// Device side of activations kept in 8 bits: where a wave's elements lie, the
// scale of 32 rows of a column, coding and decoding.
//
// value(r, c) = E4M3(data[r * ld + c]) * 2^(scale[(r / 32) * ld + c] - 127)
//
// Two ways over a matrix.  Wide: a workgroup of four waves takes 32 rows x 512
// columns, a wave eight of the rows, so that an access of a wave is one run of
// up to 1 KiB of a row; the maxima of a column meet in LDS (4096 x 4096 fp32: the
// forward pass 46 us, narrow 53).  Narrow (matrices
// of fewer columns): a wave takes 32 rows x 128 columns, lane l rows l / 16,
// l / 16 + 4, ..., l / 16 + 28, and the maxima meet over lanes 16, 32 and 48
// away.  A lane's eight columns are one run of 16-bit elements and two runs of
// four, far apart, of fp32, so that neighbouring lanes' accesses adjoin.
#pragma once
#include "device_util.h"
#include "list_device.h"

namespace qm {
namespace {

constexpr int kGroupRows = 32;               // rows of a column that share a scale
constexpr int kLaneRows = 8, kPatchWaves = 4;
constexpr int kScaleLow = 32, kScaleHigh = 246;   // scale bytes: exponents -95 .. 119

// A store that leaves its line in the caches to be completed.
template <int BYTES> __device__ __forceinline__ void store_kept(uint64_t base, const Packed<BYTES> &r) {
    char *p = gmem<char>(base);
    if constexpr (BYTES == 16) *reinterpret_cast<u32x4_e *>(p) = u32x4_e{r.w[0], r.w[1], r.w[2], r.w[3]};
    else if constexpr (BYTES == 8) *reinterpret_cast<u32x2_e *>(p) = u32x2_e{r.w[0], r.w[1]};
    else *reinterpret_cast<u32_e *>(p) = r.w[0];
}
// Stores of whole lines (rows that start on one) take the non-temporal hint,
// others do not: the forward pass of 8192 x 14336 in bf16 took 158 us with and
// 168 without it, that of 3001 x 6145 in f16 44 and 37.
template <bool LINES, int BYTES> __device__ __forceinline__ void store_row(uint64_t base, const Packed<BYTES> &r) {
    if constexpr (LINES) store_bytes(base, 0, r);
    else store_kept(base, r);
}

// A patch and a lane's place in it.
template <int TYPE, bool WIDE_> struct Patch {
    static constexpr int DT = TYPE;
    static constexpr bool WIDE = WIDE_;
    static constexpr int W = DT == QM_F32 ? 4 : 8, P = 8 / W;                      // columns of a piece, pieces
    static constexpr int kCols = WIDE ? 512 : 128, kApart = kCols / P, kRowStep = WIDE ? 1 : 4;
    int64_t row, col;    // the lane's first row and column
    bool whole;          // every element of the patch exists (uniform)
    int rows, left;      // rows (of 8, kRowStep apart) the lane has; columns from its first on

    __device__ __forceinline__ Patch(int64_t n_rows, int64_t n_cols, int64_t patch, int64_t patches_across) {
        const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x / 64));
        const int64_t r0 = patch / patches_across * kGroupRows, c0 = patch % patches_across * kCols;
        whole = r0 + kGroupRows <= n_rows && c0 + kCols <= n_cols;
        row = r0 + (WIDE ? wave * kLaneRows : lane / 16);
        col = c0 + (WIDE ? lane : lane % 16) * W;
        rows = row >= n_rows ? 0 : (int)min((int64_t)kLaneRows, (n_rows - row + kRowStep - 1) / kRowStep);
        left = (int)max((int64_t)0, min((int64_t)kCols, n_cols - col));
    }
    // columns of piece q
    __device__ __forceinline__ int n(int q) const { return max(0, min(W, left - q * kApart)); }
    __device__ __forceinline__ uint64_t at(uint64_t base, int64_t ld, int i, int q, int size) const {
        return base + (uint64_t)((row + kRowStep * i) * ld + col + q * kApart) * size;
    }
    __device__ __forceinline__ uint64_t scale_at(uint64_t base, int64_t ld, int q) const {
        return base + (uint64_t)(row / kGroupRows * ld + col + q * kApart);
    }
};

// Eight elements of row i of the lane (zeros where there are none).
template <typename A> __device__ __forceinline__ PackedOf<A::DT, 8> patch_load(uint64_t base, int64_t ld, const A &p, int i) {
    constexpr int DT = A::DT;
    PackedOf<DT, 8> r = {};
#pragma unroll
    for (int q = 0; q < A::P; q++) {
        const uint64_t at = p.at(base, ld, i, q, kSizeOf<DT>);
        if (p.whole || (i < p.rows && p.n(q) == A::W)) {
            const Packed<16> w = load_bytes<16>(at, 0);
#pragma unroll
            for (int j = 0; j < 4; j++) r.w[4 * q + j] = w.w[j];
        } else if (i < p.rows) {
#pragma unroll
            for (int j = 0; j < A::W; j++) {
                if (j >= p.n(q)) continue;
                if constexpr (DT == QM_F32) r.w[4 * q + j] = gmem<const uint32_t>(at)[j];
                else r.w[j / 2] |= (unsigned)gmem<const uint16_t>(at)[j] << (16 * (j % 2));
            }
        }
    }
    return r;
}
template <bool LINES, typename A> __device__ __forceinline__ void patch_store(uint64_t base, int64_t ld, const A &p, int i, const float *x) {
    constexpr int DT = A::DT;
#pragma unroll
    for (int q = 0; q < A::P; q++) {
        const uint64_t at = p.at(base, ld, i, q, kSizeOf<DT>);
        if (p.whole || (i < p.rows && p.n(q) == A::W)) store_row<LINES>(at, qm::pack<DT, A::W>(x + q * A::W));
        else if (i < p.rows) {
#pragma unroll
            for (int j = 0; j < A::W; j++)
                if (j < p.n(q)) store_one<DT>(at, j, x[q * A::W + j]);
        }
    }
}

// The kept bytes and scales: rows of a multiple of 16 bytes, so a piece is there
// (what lies past the last column included) wherever its first column is.
template <typename A> __device__ __forceinline__ bool has_bytes(const A &p, int i, int q) {
    return p.whole || (i < p.rows && p.n(q) > 0);
}
template <bool SCALES, typename A> __device__ __forceinline__ Packed<8> load_kept(const A &p, uint64_t base, int64_t ld, int i) {
    Packed<8> w = {};
#pragma unroll
    for (int q = 0; q < A::P; q++) {
        if (!has_bytes(p, i, q)) continue;
        const uint64_t at = SCALES ? p.scale_at(base, ld, q) : p.at(base, ld, i, q, 1);
        if constexpr (A::P == 1) w = load_bytes<8>(at, 0);
        else w.w[q] = load_bytes<4>(at, 0).w[0];
    }
    return w;
}
template <bool LINES, bool SCALES, typename A>
__device__ __forceinline__ void store_kept8(const A &p, uint64_t base, int64_t ld, int i, const Packed<8> &w) {
#pragma unroll
    for (int q = 0; q < A::P; q++) {
        if (!has_bytes(p, i, q)) continue;
        const uint64_t at = SCALES ? p.scale_at(base, ld, q) : p.at(base, ld, i, q, 1);
        if constexpr (A::P == 1) store_row<LINES>(at, w);
        else store_row<LINES && A::WIDE>(at, Packed<4>{{w.w[q]}});
    }
}

typedef float f32x2_v __attribute__((ext_vector_type(2)));

// Bits of the largest magnitudes of a lane's columns over its rows: as unsigned
// numbers magnitudes of floats order as the floats do, infinities and NaN above
// them.
template <int DT> __device__ __forceinline__ void lane_tops(const PackedOf<DT, 8> (&r)[kLaneRows], uint32_t *top) {
#pragma unroll
    for (int j = 0; j < 8; j++) {
        top[j] = 0;
#pragma unroll
        for (int i = 0; i < kLaneRows; i++) top[j] = max(top[j], __float_as_uint(unpack<DT>(r[i], j)) & 0x7fffffffu);
    }
}
// N matrices' maxima over the 32 rows.
template <typename A, int N> __device__ __forceinline__ void group_tops(uint32_t (&top)[N][8]) {
    if constexpr (A::WIDE) {
        __shared__ __attribute__((aligned(16))) uint32_t all[N][kPatchWaves][8][64];
        const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x / 64));
#pragma unroll
        for (int m = 0; m < N; m++)
#pragma unroll
            for (int j = 0; j < 8; j++) all[m][wave][j][lane] = top[m][j];
        __syncthreads();
#pragma unroll
        for (int m = 0; m < N; m++)
#pragma unroll
            for (int j = 0; j < 8; j++)
#pragma unroll
                for (int w = 0; w < kPatchWaves; w++) top[m][j] = max(top[m][j], all[m][w][j][lane]);
    } else {
#pragma unroll
        for (int m = 0; m < N; m++)
#pragma unroll
            for (int j = 0; j < 8; j++) {
                top[m][j] = max(top[m][j], (uint32_t)xor_lanes((int)top[m][j], 16));
                top[m][j] = max(top[m][j], (uint32_t)xor_lanes((int)top[m][j], 32));
            }
    }
}

// Scale byte of a column whose largest magnitude has these bits: the smallest
// power of two with top <= 448 = 1.75 * 2^8 times it.  Past 1.75 the fraction
// carries into the exponent.
__device__ __forceinline__ uint32_t scale_byte(uint32_t top) {
    const int b = (int)((top + 0x1fffffu) >> 23) - 8;
    return (uint32_t)min(max(b, kScaleLow), kScaleHigh);
}

// Packed elements to be unpacked anew: the compiler otherwise keeps all of them
// unpacked from one use to the next, which takes half of the waves in flight.
template <int BYTES, int N> __device__ __forceinline__ void unpack_anew(Packed<BYTES> (&r)[N]) {
#pragma unroll
    for (int i = 0; i < N; i++)
#pragma unroll
        for (int k = 0; k < BYTES / 4; k++) asm volatile("" : "+v"(r[i].w[k]));
}

// Codes of the lane's eight rows and the scale bytes of its columns, whose
// largest magnitudes are `top`.
template <bool LINES, typename A>
__device__ __forceinline__ void encode(const A &p, const PackedOf<A::DT, 8> (&r)[kLaneRows], const uint32_t *top, uint64_t data,
                                       uint64_t scale, int64_t ld) {
    constexpr int DT = A::DT;
    float inv[8];
    uint32_t sb[8], bad[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; j++) {
        sb[j] = scale_byte(top[j]);
        inv[j] = __uint_as_float((254u - sb[j]) << 23);
        // a column that holds an infinity or a NaN: every code a NaN
        if (top[j] >= 0x7f800000u) bad[j / 4] |= 0x7fu << (8 * (j % 4));
    }
#pragma unroll
    for (int i = 0; i < kLaneRows; i++) {
        float c[8];
        // past 448 only where the exponent met its upper limit
#pragma unroll
        for (int j = 0; j < 8; j++) c[j] = __builtin_amdgcn_fmed3f(unpack<DT>(r[i], j) * inv[j], -448.0f, 448.0f);
        Packed<8> w;
#pragma unroll
        for (int h = 0; h < 2; h++) {
            const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(c[4 * h], c[4 * h + 1], 0, false);
            w.w[h] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c[4 * h + 2], c[4 * h + 3], lo, true) | bad[h];
        }
        store_kept8<LINES, false>(p, data, ld, i, w);
    }
    // the lanes that hold the group's first row
    if (A::WIDE ? threadIdx.x < 64 : threadIdx.x % 64 < 16) {
        Packed<8> w;
        w.w[0] = sb[0] | sb[1] << 8 | sb[2] << 16 | sb[3] << 24;
        w.w[1] = sb[4] | sb[5] << 8 | sb[6] << 16 | sb[7] << 24;
        store_kept8<LINES, true>(p, scale, ld, 0, w);
    }
}

// The lane's eight scales as fp32 numbers, and its codes of row i (zeros where
// there are none).
template <typename A> __device__ __forceinline__ void load_scales(const A &p, uint64_t scale, int64_t ld, float *unit) {
    const Packed<8> w = load_kept<true>(p, scale, ld, 0);
#pragma unroll
    for (int j = 0; j < 8; j++) unit[j] = __uint_as_float((w.w[j / 4] >> (8 * (j % 4)) & 0xffu) << 23);
}
template <typename A> __device__ __forceinline__ Packed<8> load_codes(const A &p, uint64_t data, int64_t ld, int i) {
    return load_kept<false>(p, data, ld, i);
}
__device__ __forceinline__ void decode(const Packed<8> &w, const float *unit, float *x) {
#pragma unroll
    for (int h = 0; h < 2; h++) {
        const f32x2_v a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w.w[h], false);
        const f32x2_v b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w.w[h], true);
        x[4 * h] = a.x * unit[4 * h];
        x[4 * h + 1] = a.y * unit[4 * h + 1];
        x[4 * h + 2] = b.x * unit[4 * h + 2];
        x[4 * h + 3] = b.y * unit[4 * h + 3];
    }
}

}  // namespace
}  // namespace qm
