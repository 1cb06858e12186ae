// AdamW over many tensors for gfx950 (wave64), with 32-bit states or with
// 8-bit states in blocks of 256.  Compiled with -ffp-contract=off: the coding
// of 8-bit states is defined by binary32 operations with one rounding each,
// so the codes match a CPU run of the same operations bit for bit.
//
// "Decoupled Weight Decay Regularization" (Loshchilov and Hutter, ICLR 2019)
// gives the step.  Every byte of gradient, weight and state is touched once,
// and HBM binds: a large copy reaches 6.5 TB/s on this part, and of that
//   32-bit states, fp32 weight, bf16 gradient and copy (28 bytes an element):
//     218M elements in 1.04 ms, 5.9 TB/s;
//   8-bit states, fp32 weight, bf16 gradient and copy (16.1): 206M in 0.53
//     ms, 6.2 TB/s;
//   8-bit states, bf16 weight and gradient (10.1): 218M in 0.35 ms, 6.2 TB/s,
//     with the VALU busy 76 % of the time; with stochastic codes the VALU
//     binds (82 %): 36M in 0.072 ms, 5.0 TB/s (979 instructions a task against
//     669; half of the difference makes the random numbers).
//
// One wave64 owns a task of 1024 consecutive elements of one tensor and issues
// all of its loads before the arithmetic (half the task a wave: 1.09 ms for the
// first line; four waves interleaved by the KiB: 1.09; a grid mapped so that
// each XCD takes one contiguous part: 1.11; loads or stores through the caches
// instead of past them: 1.08 to 1.11; workgroups of 64, 128, 512 and 1024
// threads: 1.07 to 1.12).  One launch covers all tensors of one kind of state,
// whatever their types: a wave's types are uniform, so it takes one branch.
#include <hip/hip_runtime.h>

#include <math.h>
#include <stdint.h>

#include "internal.h"
#include "list_device.h"
#include "list_host.h"
#include "list_layout.h"
#include "plan_layout.h"
#include "qmuon.h"

namespace qm {
namespace {

constexpr int kThreads = 256;
constexpr int kWavesPerWG = kThreads / 64;
constexpr float kTiny = 0x1p-100f;   // blocks with a smaller maximum hold zeros

struct AdamArgs {
    const ListTensor *tensors;
    const int32_t *owner;      // tensor of every task
    const float *grad_scale;   // null: 1
    int32_t task_lo, task_hi;
    float b1, omb1, b2, omb2;  // beta1, 1 - beta1, beta2, 1 - beta2
    float step, lr;            // lr / (1 - beta1^t), lr
    float root, eps;           // 1 / sqrt(1 - beta2^t), eps
    uint64_t seed;
    uint32_t offset;
};

// New weight from the new moments.  The root and the reciprocal are the
// hardware's, within an ulp.  The root takes subnormal numbers for 0: SCALED
// keeps it right there too (v below 2^-96 times 2^64), which a step needs only
// where the root of 2^-126 counts next to eps.  denom >= eps >= 2^-126 has a
// finite reciprocal.
template <bool SCALED>
__device__ __forceinline__ float new_weight(float w, float m, float v, float step, float decay, const AdamArgs &A) {
    const bool tiny = SCALED && v < 0x1p-96f;
    const float r = __builtin_amdgcn_sqrtf(tiny ? v * 0x1p64f : v);
    const float denom = __builtin_fmaf(r, tiny ? A.root * 0x1p-32f : A.root, A.eps);
    return in_fp32(__builtin_fmaf(-step, m * __builtin_amdgcn_rcpf(denom), __builtin_fmaf(-decay, w, w)));
}

template <int DT> __device__ __forceinline__ void store_weight(const ListTensor &T, int64_t e, int n, const float *w) {
    store_edge<DT>(T.weight, e, n, w);
    if (T.copy == 0) return;
    if (T.copy_dtype == QM_BF16) store_edge<QM_BF16>(T.copy, e, n, w);
    else store_edge<QM_F16>(T.copy, e, n, w);
}

// ------------------------------------------------------------ 32-bit states

// At most one block.
template <int GDT, int WDT>
__device__ __forceinline__ void task32(const ListTensor &T, int64_t e_task, int nvalid, int lane, float c, const AdamArgs &A) {
    const float step = A.step * T.lr_scale, decay = A.lr * T.lr_scale * T.weight_decay;
    const int n = min(4, nvalid - lane * 4);
    if (n <= 0) return;
    const int64_t e = e_task + lane * 4;
    const PackedOf<GDT, 4> rg = load_grad<GDT>(T, e, n);
    const PackedOf<WDT, 4> rw = load_edge<WDT>(T.weight, e, n);
    const Packed<16> rm = load_edge<QM_F32>(T.m, e, n), rv = load_edge<QM_F32>(T.v, e, n);
    float m[4], v[4], w[4];
#pragma unroll
    for (int j = 0; j < 4; j++) {
        const float g = unpack<GDT>(rg, j) * c;
        m[j] = A.b1 * unpack<QM_F32>(rm, j) + A.omb1 * g;
        v[j] = A.b2 * unpack<QM_F32>(rv, j) + A.omb2 * (g * g);
        w[j] = new_weight<true>(unpack<WDT>(rw, j), m[j], v[j], step, decay, A);
    }
    store_edge<QM_F32>(T.m, e, n, m);
    store_edge<QM_F32>(T.v, e, n, v);
    store_weight<WDT>(T, e, n, w);
}

// A whole task: 4 elements per lane in each of 4 parts, so that an
// instruction covers one contiguous KiB (fp32) or half of one.
template <int GDT, int WDT>
__device__ __forceinline__ void task32_full(const ListTensor &T, int64_t e_task, int lane, float c, const AdamArgs &A) {
    constexpr int P = kListTask / 256;
    PackedOf<GDT, 4> rg[P];
    PackedOf<WDT, 4> rw[P];
    Packed<16> rm[P], rv[P];
    const uint64_t bw = T.weight + (uint64_t)e_task * kSizeOf<WDT>, bm = T.m + (uint64_t)e_task * 4, bv = T.v + (uint64_t)e_task * 4;
    load_grad_task<GDT, 4, P>(T, e_task, lane, rg);
#pragma unroll
    for (int p = 0; p < P; p++) {
        const uint32_t i = p * 256 + lane * 4;
        rw[p] = load_bytes<4 * kSizeOf<WDT>>(bw, i * kSizeOf<WDT>);
        rm[p] = load_bytes<16>(bm, i * 4);
        rv[p] = load_bytes<16>(bv, i * 4);
    }
    const float step = A.step * T.lr_scale, decay = A.lr * T.lr_scale * T.weight_decay;
#pragma unroll
    for (int p = 0; p < P; p++) {
        const uint32_t i = p * 256 + lane * 4;
        float m[4], v[4], w[4];
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const float g = unpack<GDT>(rg[p], j) * c;
            m[j] = A.b1 * unpack<QM_F32>(rm[p], j) + A.omb1 * g;
            v[j] = A.b2 * unpack<QM_F32>(rv[p], j) + A.omb2 * (g * g);
            w[j] = new_weight<true>(unpack<WDT>(rw[p], j), m[j], v[j], step, decay, A);
        }
        store_bytes(bm, i * 4, pack<QM_F32, 4>(m));
        store_bytes(bv, i * 4, pack<QM_F32, 4>(v));
        store_bytes(bw, i * kSizeOf<WDT>, pack<WDT, 4>(w));
        if (T.copy) {
            const uint64_t bc = T.copy + (uint64_t)e_task * 2;
            if (T.copy_dtype == QM_BF16) store_bytes(bc, i * 2, pack<QM_BF16, 4>(w));
            else store_bytes(bc, i * 2, pack<QM_F16, 4>(w));
        }
    }
}

// ------------------------------------------------------------ 8-bit states

__device__ __forceinline__ uint32_t load_codes(uint64_t base, int64_t e, int n) {
    if (n == 4) return *gmem<const u32_e>(base + (uint64_t)e);
    uint32_t r = 0;
#pragma unroll
    for (int j = 0; j < 4; j++)
        if (j < n) r |= (uint32_t)*gmem<const uint8_t>(base + (uint64_t)(e + j)) << (8 * j);
    return r;
}
__device__ __forceinline__ void store_codes(uint64_t base, int64_t e, int n, uint32_t q) {
    if (n == 4) {
        *gmem<u32_e>(base + (uint64_t)e) = q;
        return;
    }
#pragma unroll
    for (int j = 0; j < 4; j++)
        if (j < n) *gmem<uint8_t>(base + (uint64_t)(e + j)) = (uint8_t)(q >> (8 * j));
}

// x / D for D = 127 or 65025, correctly rounded: quotient by the rounded
// reciprocal, one step of its residual.  Equal to the division for every
// significand (checked exhaustively) and every x that a block maximum can be
// (0, or 2^-100 and above).
template <int D> __device__ __forceinline__ float div_const(float x) {
    constexpr float d = (float)D, r = 1.0f / d;
    const float q = x * r;
    return __builtin_fmaf(__builtin_fmaf(-q, d, x), r, q);
}

// Rows are the 16-lane quarters of a wave.  What is computed once a block
// (scales, quotients) is held by the block's row: row r has block
// (r & 1) * 2 + (r >> 1), which is where the swaps below put it.
__device__ __forceinline__ int row_block(int lane) { return ((lane >> 4) & 1) * 2 + (lane >> 5); }

__device__ __forceinline__ void swap16(uint32_t &a, uint32_t &b) {   // odd rows of a with even rows of b
    const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}
__device__ __forceinline__ void swap32(uint32_t &a, uint32_t &b) {   // upper half of a with lower half of b
    const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}

// The rows' values to each lane's value per part: x[h] is that of the block
// the lane's elements of part h are in.
template <int H> __device__ __forceinline__ void row_spread(float row, float *x) {
    uint32_t a = __float_as_uint(row), b = a;
    swap16(a, b);   // a: rows 0 0 2 2, b: rows 1 1 3 3
    if constexpr (H == 2) {
        x[0] = __uint_as_float(a);
        x[1] = __uint_as_float(b);
    } else {
        uint32_t c = a, d = b;
        swap32(a, c);
        swap32(b, d);
        x[0] = __uint_as_float(a);
        x[1] = __uint_as_float(c);
        x[2] = __uint_as_float(b);
        x[3] = __uint_as_float(d);
    }
}

template <int ROR> __device__ __forceinline__ uint32_t max_ror(uint32_t x) {
    return max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x120 + ROR, 0xf, 0xf, false));
}
// Each lane's maximum per part to the blocks' maxima in their rows: every
// swap merges two registers, so all four blocks take one chain of steps.
template <int H> __device__ __forceinline__ uint32_t row_max(uint32_t *t) {
    if constexpr (H == 4) {
        swap32(t[0], t[1]);
        swap32(t[2], t[3]);
        t[0] = max(t[0], t[1]);
        t[1] = max(t[2], t[3]);
    }
    swap16(t[0], t[1]);
    return max_ror<1>(max_ror<2>(max_ror<4>(max_ror<8>(max(t[0], t[1])))));
}

// Maximum over the wave.
__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
    x = max_ror<1>(max_ror<2>(max_ror<4>(max_ror<8>(x))));
    uint32_t y = x;
    swap16(x, y);
    x = y = max(x, y);
    swap32(x, y);
    return max(x, y);
}

// y = v (65025 / max) lies in [0, 65025 (1 + 2^-23)], x = m (127 / max) in
// +-127 (1 + 2^-23).
//
// k = 0 and v > 0: the code is 1 all the same.
__device__ __forceinline__ bool alone(float k, float v) { return v > k * 0x1.fffffep127f; }

// Code of v by nearest value.  k = floor of the hardware root (within an ulp)
// is floor(sqrt y) or its neighbour next to a perfect square, where both give
// the same code; v > 0 codes at least 1.
__device__ __forceinline__ uint32_t v_code_near(float y, float v) {
    const float k = floorf(__builtin_amdgcn_sqrtf(y));
    const float d = __builtin_fmaf(-k, k, y);
    return (uint32_t)(int)k + (uint32_t)((d > k + 0.5f) | alone(k, v));
}

// The same by a 16-bit and a 15-bit random number (the two halves of the
// element's word).
//
// m: with x' = 2^16 x exact and u a whole number, u < 2^16 frac(x) is
// u < ceil(x') - 2^16 floor(x), so the code is the sum ceil(x') - u + 65535
// without its 16 low bits; x past 127 by its own rounding is held back.
// Returns the code in byte 2.
__device__ __forceinline__ uint32_t m_code_random(float x16, uint32_t word) {
    const int s = (int)ceilf(x16) - (int)(word >> 16) + 65535;
    return (uint32_t)min(s, 127 * 65536 + 65535);
}
// v: k = floor of the hardware root is floor(sqrt y) or, next below a square,
// one above (checked for every y up to 65026); there y - k^2 < 0 keeps k,
// as the exact comparison does by a margin of 2 (it misses 2 k + 1 by less
// than 2^-15 of it).  u (2k + 1) has 24 bits.
__device__ __forceinline__ uint32_t v_code_random(float y, float v, uint32_t word) {
    const float k = floorf(__builtin_amdgcn_sqrtf(y));
    const float d = __builtin_fmaf(-k, k, y), t = __builtin_fmaf(k, 0x1p-14f, 0x1p-15f);   // 2^-15 (2k + 1)
    return min((uint32_t)(int)k + (uint32_t)(((float)(word & 0x7fffu) * t < d) | alone(k, v)), 255u);
}

// Codes of N elements of a block: im = 127 / (max of |m|), iv = 65025 / (max
// of v), 0 for a block of zeros; the elements' group of four number `group`
// (64 bits in two words) is the counter of their random words.
template <bool SR, int N>
__device__ __forceinline__ void code_group(const float *m, const float *v, float im, float iv, uint32_t group_lo, uint32_t group_hi,
                                           uint32_t tensor, const AdamArgs &A, Packed<N> &om, Packed<N> &ov) {
    uint32_t cm[N], cv[N];
    if constexpr (SR) {
        uint32_t word[N];
#pragma unroll
        for (int k = 0; k < N / 4; k++)
            philox4x32_10(group_lo + k, group_hi, A.offset, tensor, (uint32_t)A.seed, (uint32_t)(A.seed >> 32), word + 4 * k);
        const float im16 = im * 0x1p16f;
#pragma unroll
        for (int j = 0; j < N; j++) {
            cm[j] = m_code_random(m[j] * im16, word[j]);
            cv[j] = v_code_random(v[j] * iv, v[j], word[j]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < N; j++) {
            // adding 1.5 * 2^23 rounds to a whole number, ties to even: the sum's low byte is the code
            cm[j] = __float_as_uint(m[j] * im + 12582912.0f);
            cv[j] = v_code_near(v[j] * iv, v[j]);
        }
    }
#pragma unroll
    for (int k = 0; k < N; k += 4) {
        om.w[k / 4] = pack_bytes<SR ? 2 : 0>(cm[k], cm[k + 1], cm[k + 2], cm[k + 3]);
        ov.w[k / 4] = pack_bytes<0>(cv[k], cv[k + 1], cv[k + 2], cv[k + 3]);
    }
}

// New moments of N elements, their largest magnitudes into tm and tv (NaN if
// one is), and the new weights.
template <bool SCALED, int N, typename Grad, typename Weight>
__device__ __forceinline__ void update_group(Grad grad, Weight weight, const Packed<N> &qm, const Packed<N> &qv, float step_m, float step_v,
                                             float c, float step, float decay, const AdamArgs &A, float *m, float *v, float *w,
                                             float &tm, float &tv) {
#pragma unroll
    for (int j = 0; j < N; j++) {
        const float g = grad(j) * c;
        // Signed, one instruction as cv.  (The byte plus 128, with 128 steps taken
        // off in a fused product, is 1 % faster on 218M bf16 elements, 352 us for
        // 357, but 128 steps leave fp32's range next to its end.)
        const float cm = (float)(int8_t)(qm.w[j / 4] >> (8 * (j % 4)));
        const float cv = (float)((qv.w[j / 4] >> (8 * (j % 4))) & 0xffu);
        m[j] = cm * step_m + A.omb1 * g;
        v[j] = (cv * cv) * step_v + A.omb2 * (g * g);
        tm = __builtin_elementwise_maximum(tm, fabsf(m[j]));
        tv = __builtin_elementwise_maximum(tv, fabsf(v[j]));
        w[j] = new_weight<SCALED>(weight(j), m[j], v[j], step, decay, A);
    }
}

// At most one block.  Elements past its end are zeros: they leave the maxima
// alone and are not stored.
template <int GDT, int WDT, bool SR, bool SCALED>
__device__ __forceinline__ void task8(const ListTensor &T, int32_t tensor, int64_t e_task, int nvalid, int lane, float c,
                                      const AdamArgs &A) {
    const float step = A.step * T.lr_scale, decay = A.lr * T.lr_scale * T.weight_decay;
    const int n = max(0, min(4, nvalid - lane * 4));
    const int64_t e = e_task + lane * 4;
    float *pm = gmem<float>(T.m_absmax) + (e_task >> 8), *pv = gmem<float>(T.v_absmax) + (e_task >> 8);
    const float old_m = *pm, old_v = *pv;
    PackedOf<GDT, 4> rg = {};
    PackedOf<WDT, 4> rw = {};
    Packed<4> qm = {}, qv = {};
    if (n > 0) {
        rg = load_grad<GDT>(T, e, n);
        rw = load_edge<WDT>(T.weight, e, n);
        qm.w[0] = load_codes(T.m, e, n);
        qv.w[0] = load_codes(T.v, e, n);
    }
    // past the end no scale either: it may be NaN
    const float step_m = n > 0 ? div_const<127>(old_m) * A.b1 : 0.0f, step_v = n > 0 ? div_const<65025>(old_v) * A.b2 : 0.0f;
    float m[4], v[4], w[4], tm = 0.0f, tv = 0.0f;
    update_group<SCALED, 4>([&](int j) { return unpack<GDT>(rg, j); }, [&](int j) { return unpack<WDT>(rw, j); }, qm, qv, step_m, step_v, c, step, decay,
                    A, m, v, w, tm, tv);
    store_weight<WDT>(T, e, n, w);
    float am = __uint_as_float(wave_max(__float_as_uint(tm))), av = __uint_as_float(wave_max(__float_as_uint(tv)));
    if (am < kTiny) am = 0.0f;
    if (av < kTiny) av = 0.0f;
    if (lane == 0) {
        *pm = am;
        *pv = av;
    }
    Packed<4> om, ov;
    code_group<SR, 4>(m, v, am > 0.0f ? 127.0f / am : 0.0f, av > 0.0f ? 65025.0f / av : 0.0f, (uint32_t)((uint64_t)e_task >> 2) + lane,
                      (uint32_t)((uint64_t)e_task >> 34), (uint32_t)tensor, A, om, ov);
    store_codes(T.m, e, n, am < INFINITY ? om.w[0] : 0u);
    store_codes(T.v, e, n, av < INFINITY && av > 0.0f ? ov.w[0] : 0u);
}

// ---- a whole task: N = 8 elements per lane in each of H = 2 halves, a
// block being 32 lanes of one half, or N = 4 in each of H = 4 parts, a block
// being one part.  Eight make one 16-byte access of a 16-bit weight, four one
// of an fp32 weight, so a weight's accesses cover whole contiguous KiB (206M
// elements with fp32 weights: 0.63 ms by eight, 0.55 by four).

template <int WDT> constexpr int kPer8 = 16 / kSizeOf<WDT>;

template <int GDT, int WDT, bool SR, bool SCALED>
__device__ __forceinline__ void task8_full(const ListTensor &T, int32_t tensor, int64_t e_task, int lane, float c, const AdamArgs &A) {
    constexpr int N = kPer8<WDT>, H = kListTask / (64 * N);
    PackedOf<GDT, N> rg[H];
    PackedOf<WDT, N> rw[H];
    Packed<N> qm[H], qv[H];
    const uint64_t bw = T.weight + (uint64_t)e_task * kSizeOf<WDT>, bm = T.m + (uint64_t)e_task, bv = T.v + (uint64_t)e_task;
    float *pm = gmem<float>(T.m_absmax) + (e_task >> 8) + row_block(lane);
    float *pv = gmem<float>(T.v_absmax) + (e_task >> 8) + row_block(lane);
    const float old_m = *pm, old_v = *pv;
    load_grad_task<GDT, N, H>(T, e_task, lane, rg);
#pragma unroll
    for (int h = 0; h < H; h++) {
        const uint32_t i = h * 64 * N + lane * N;
        qm[h] = load_bytes<N>(bm, i);
        qv[h] = load_bytes<N>(bv, i);
        rw[h] = load_bytes<N * kSizeOf<WDT>>(bw, i * kSizeOf<WDT>);
    }
    const float step = A.step * T.lr_scale, decay = A.lr * T.lr_scale * T.weight_decay;
    float step_m[H], step_v[H], m[H][N], v[H][N];
    row_spread<H>(div_const<127>(old_m) * A.b1, step_m);
    row_spread<H>(div_const<65025>(old_v) * A.b2, step_v);
    uint32_t top_m[H], top_v[H];
#pragma unroll
    for (int h = 0; h < H; h++) {
        const uint32_t i = h * 64 * N + lane * N;
        float w[N], tm = 0.0f, tv = 0.0f;
        update_group<SCALED, N>([&](int j) { return unpack<GDT>(rg[h], j); }, [&](int j) { return unpack<WDT>(rw[h], j); }, qm[h], qv[h], step_m[h],
                        step_v[h], c, step, decay, A, m[h], v[h], w, tm, tv);
        top_m[h] = __float_as_uint(tm);
        top_v[h] = __float_as_uint(tv);
        store_bytes(bw, i * kSizeOf<WDT>, pack<WDT, N>(w));
        if (T.copy) {
            const uint64_t bc = T.copy + (uint64_t)e_task * 2;
            if (T.copy_dtype == QM_BF16) store_bytes(bc, i * 2, pack<QM_BF16, N>(w));
            else store_bytes(bc, i * 2, pack<QM_F16, N>(w));
        }
    }
    float am = __uint_as_float(row_max<H>(top_m)), av = __uint_as_float(row_max<H>(top_v));
    if (am < kTiny) am = 0.0f;
    if (av < kTiny) av = 0.0f;
    if ((lane & 15) == 0) {
        *pm = am;
        *pv = av;
    }
    float im[H], iv[H];
    row_spread<H>(am > 0.0f ? 127.0f / am : 0.0f, im);
    row_spread<H>(av > 0.0f ? 65025.0f / av : 0.0f, iv);
    // blocks whose codes are all 0: a maximum that is not finite, or v's is 0
    float keep_m[H] = {}, keep_v[H] = {};
    const bool odd = __any(!(am < INFINITY) || !(av < INFINITY) || av == 0.0f);
    if (odd) {
        row_spread<H>(am < INFINITY ? 1.0f : 0.0f, keep_m);
        row_spread<H>(av < INFINITY && av > 0.0f ? 1.0f : 0.0f, keep_v);
    }
#pragma unroll
    for (int h = 0; h < H; h++) {
        const uint32_t i = h * 64 * N + lane * N;
        // the counter's upper word, the offset and the tensor are uniform, which
        // leaves the first two rounds one product each per lane
        Packed<N> om, ov;
        code_group<SR, N>(m[h], v[h], im[h], iv[h], (uint32_t)((uint64_t)e_task >> 2) + (i >> 2), (uint32_t)((uint64_t)e_task >> 34),
                          (uint32_t)tensor, A, om, ov);
        if (odd) {
#pragma unroll
            for (int k = 0; k < N / 4; k++) {
                if (keep_m[h] == 0.0f) om.w[k] = 0;
                if (keep_v[h] == 0.0f) ov.w[k] = 0;
            }
        }
        store_bytes(bm, i, om);
        store_bytes(bv, i, ov);
    }
}

// ------------------------------------------------------------ kernels

template <int BITS, bool SR, bool SCALED, int GDT, int WDT>
__device__ __forceinline__ void run_task(const ListTensor &T, int32_t tensor, int64_t lt, int lane, float c, const AdamArgs &A) {
    int nvalid;
    const int64_t e_task = task_start(T, lt, nvalid);
    if constexpr (BITS == 32) {
        if (nvalid == kListTask) task32_full<GDT, WDT>(T, e_task, lane, c, A);
        else task32<GDT, WDT>(T, e_task, nvalid, lane, c, A);
    }
    else {
        if (nvalid == kListTask) task8_full<GDT, WDT, SR, SCALED>(T, tensor, e_task, lane, c, A);
        else task8<GDT, WDT, SR, SCALED>(T, tensor, e_task, nvalid, lane, c, A);
    }
}

template <int BITS, bool SR, bool SCALED> __global__ __launch_bounds__(kThreads, 6) void adamw_kernel(AdamArgs A) {
    const int lane = threadIdx.x & 63;
    const int task = A.task_lo + __builtin_amdgcn_readfirstlane((int)(blockIdx.x * kWavesPerWG + (threadIdx.x >> 6)));
    if (task >= A.task_hi) return;
    float c = 1.0f;
    if (A.grad_scale) {
        c = *gmem<const float>(A.grad_scale);
        if (c != c) return;   // the gradient's norm is not finite: leave everything as it is
    }
    const int32_t ti = __builtin_amdgcn_readfirstlane(gmem<const int32_t>(A.owner)[task]);
    const ListTensor T = gmem<const ListTensor>(A.tensors)[ti];
    const int64_t lt = task - T.task_offset;
    switch (T.grad_dtype * 3 + T.weight_dtype) {
        case QM_F32 * 3 + QM_F32: run_task<BITS, SR, SCALED, QM_F32, QM_F32>(T, ti, lt, lane, c, A); break;
        case QM_F32 * 3 + QM_BF16: run_task<BITS, SR, SCALED, QM_F32, QM_BF16>(T, ti, lt, lane, c, A); break;
        case QM_F32 * 3 + QM_F16: run_task<BITS, SR, SCALED, QM_F32, QM_F16>(T, ti, lt, lane, c, A); break;
        case QM_BF16 * 3 + QM_F32: run_task<BITS, SR, SCALED, QM_BF16, QM_F32>(T, ti, lt, lane, c, A); break;
        case QM_BF16 * 3 + QM_BF16: run_task<BITS, SR, SCALED, QM_BF16, QM_BF16>(T, ti, lt, lane, c, A); break;
        case QM_BF16 * 3 + QM_F16: run_task<BITS, SR, SCALED, QM_BF16, QM_F16>(T, ti, lt, lane, c, A); break;
        case QM_F16 * 3 + QM_F32: run_task<BITS, SR, SCALED, QM_F16, QM_F32>(T, ti, lt, lane, c, A); break;
        case QM_F16 * 3 + QM_BF16: run_task<BITS, SR, SCALED, QM_F16, QM_BF16>(T, ti, lt, lane, c, A); break;
        default: run_task<BITS, SR, SCALED, QM_F16, QM_F16>(T, ti, lt, lane, c, A); break;
    }
}

// The values the states stand for.  Even workgroups read m, odd ones v, of
// the same four tasks: a workgroup with one stream in and one out runs 218M
// elements in 8 bits in 0.34 ms (6.4 TB/s, near the rate of a large copy), one
// with both took 0.40.  Codes are loaded through the caches (what a step has
// just written may still be there), values stored past them.
__global__ __launch_bounds__(kThreads) void adamw_read_kernel(const ListTensor *tensors, const int32_t *owner, int n_tasks,
                                                             float *m_out, float *v_out) {
    const int lane = threadIdx.x & 63;
    const bool is_v = blockIdx.x & 1;
    const int task = __builtin_amdgcn_readfirstlane((int)((blockIdx.x >> 1) * kWavesPerWG + (threadIdx.x >> 6)));
    if (task >= n_tasks) return;
    const int32_t ti = __builtin_amdgcn_readfirstlane(gmem<const int32_t>(owner)[task]);
    const ListTensor T = gmem<const ListTensor>(tensors)[ti];
    int nvalid;
    const int64_t e_task = task_start(T, task - T.task_offset, nvalid);
    const uint64_t from = (is_v ? T.v : T.m) + (uint64_t)e_task * (T.state_bits == 32 ? 4 : 1);
    const uint64_t to = (uint64_t)(is_v ? v_out : m_out) + (uint64_t)(T.block_offset * kBlock + e_task) * 4;
    constexpr int P = kListTask / 256;
    Packed<16> x[P] = {};
    if (T.state_bits == 32) {
#pragma unroll
        for (int p = 0; p < P; p++) {
            const int e0 = p * 256 + lane * 4;
            if (e0 + 4 <= nvalid) x[p] = load_bytes<16>(from, e0 * 4);
            else
#pragma unroll
                for (int j = 0; j < 4; j++)
                    if (e0 + j < nvalid) x[p].w[j] = gmem<const uint32_t>(from)[e0 + j];
        }
    } else {
        const float *absmax = gmem<const float>(is_v ? T.v_absmax : T.m_absmax) + (e_task >> 8);
        uint32_t q[P] = {};
        float top[P];
#pragma unroll
        for (int p = 0; p < P; p++) {
            const int e0 = p * 256 + lane * 4;
            top[p] = p * 256 < nvalid ? absmax[p] : 0.0f;
            if (e0 + 4 <= nvalid) q[p] = *gmem<const u32_e>(from + e0);
            else
#pragma unroll
                for (int j = 0; j < 4; j++)
                    if (e0 + j < nvalid) q[p] |= (uint32_t)gmem<const uint8_t>(from)[e0 + j] << (8 * j);
        }
#pragma unroll
        for (int p = 0; p < P; p++) {
            const float step = top[p] / (is_v ? 65025.0f : 127.0f);
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const float cv = (float)((q[p] >> (8 * j)) & 0xffu);
                const float code = is_v ? cv * cv : (float)(int8_t)(q[p] >> (8 * j));
                x[p].w[j] = p * 256 + lane * 4 + j < nvalid ? __float_as_uint(code * step) : 0u;   // not NaN * 0 past the end
            }
        }
    }
#pragma unroll
    for (int p = 0; p < P; p++)
        if (p * 256 < nvalid) store_bytes(to, (p * 256 + lane * 4) * 4, x[p]);
}

unsigned grid_for(int64_t tasks) { return (unsigned)((tasks + kWavesPerWG - 1) / kWavesPerWG); }

}  // namespace
}  // namespace qm

using namespace qm;

extern "C" qm_status adamw_step(const void *host_plan, const void *dev_plan, const qm_adamw_hparams *hp,
                                const float *grad_scale, qm_stream_t stream) {
    clear_error();
    const ListArgs list = list_args(host_plan, dev_plan, kListAdamW);
    const ListHeader *h = list.h;
    if (!h) return list.st;
    if (!hp) return fail(QM_E_ARG, "hyperparameters are null");
    if (!isfinite(hp->lr)) return fail(QM_E_ARG, "lr must be finite");
    if (!(hp->beta1 >= 0.0 && hp->beta1 < 1.0) || !(hp->beta2 >= 0.0 && hp->beta2 < 1.0))
        return fail(QM_E_ARG, "beta1 and beta2 must lie in [0, 1)");
    if (!(hp->eps >= 0x1p-126) || !isfinite((float)hp->eps))   // a normal fp32 number: the reciprocal of it is finite
        return fail(QM_E_ARG, "eps must be at least 2^-126 and finite");
    if (hp->step < 1) return fail(QM_E_ARG, "step is 1-based");
    if (hp->rounding != QM_ROUND_NEAREST && hp->rounding != QM_ROUND_STOCHASTIC)
        return fail(QM_E_ARG, "unknown rounding mode %d", hp->rounding);
    if (!aligned(grad_scale, 4)) return fail(QM_E_ALIGN, "grad_scale needs 4-byte alignment");
    AdamArgs A = {};
    A.tensors = list.tensors;
    A.owner = list.owner;
    A.grad_scale = grad_scale;
    A.b1 = (float)hp->beta1;
    A.omb1 = (float)(1.0 - hp->beta1);
    A.b2 = (float)hp->beta2;
    A.omb2 = (float)(1.0 - hp->beta2);
    A.step = (float)(hp->lr / (1.0 - pow(hp->beta1, (double)hp->step)));
    A.lr = (float)hp->lr;
    if (!isfinite(A.step) || !isfinite(A.lr)) return fail(QM_E_ARG, "lr, or lr / (1 - beta1^step), is too large for fp32");
    A.root = (float)(1.0 / sqrt(1.0 - pow(hp->beta2, (double)hp->step)));
    A.eps = (float)hp->eps;
    A.seed = hp->seed;
    A.offset = hp->offset;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (h->n_tasks32 > 0) {
        A.task_lo = 0;
        A.task_hi = (int32_t)h->n_tasks32;
        adamw_kernel<32, false, true><<<grid_for(A.task_hi - A.task_lo), kThreads, 0, s>>>(A);
        if (qm_status e = launched("AdamW")) return e;
    }
    if (h->n_tasks > h->n_tasks32) {
        A.task_lo = (int32_t)h->n_tasks32;
        A.task_hi = (int32_t)h->n_tasks;
        const unsigned grid = grid_for(A.task_hi - A.task_lo);
        // The 8-bit kernel is held up by its instructions as much as by memory
        // (VALU busy 76 to 82 %): it keeps the root of subnormal moments only where that
        // root, at most 2^-63, is more than half a step of eps.
        const bool scaled = A.root * 0x1p-63f > 0x1p-24f * A.eps;
        const auto kernel = hp->rounding == QM_ROUND_STOCHASTIC ? (scaled ? adamw_kernel<8, true, true> : adamw_kernel<8, true, false>)
                                                                : (scaled ? adamw_kernel<8, false, true> : adamw_kernel<8, false, false>);
        // Workgroups a CU: as many as fit (7), 4, 2.  Nearest codes, bf16 weight and
        // gradient: 17M elements 30.3, 30.9, 35.1 us, 216M 356, 351, 408; fp32 both:
        // 33M 87.8, 87.9, 88.1, 67M 174, 175, 172, 216M 582, 584, 550; fp32 weight,
        // bf16 gradient: 33M 77.2, 77.7, 78.7, 67M 153, 154, 154, 216M 499, 497, 486;
        // a tenth of it bf16 weights: 108M 239, 241, 241, a quarter: 230, 231, 234.
        // Stochastic codes need their waves (fp32 weight, 216M: 493, 484, 540).
        const int64_t n8 = h->n_tasks - h->n_tasks32;
        const bool two = hp->rounding == QM_ROUND_NEAREST && 10 * h->n_wide8 >= 9 * n8 && n8 >= 1 << 16;
        kernel<<<grid, kThreads, two ? 64u << 10 : wgs_per_cu(4), s>>>(A);
        if (qm_status e = launched("AdamW with 8-bit states")) return e;
    }
    return QM_OK;
}

extern "C" qm_status adamw_read_state(const void *host_plan, const void *dev_plan, float *m_out, float *v_out,
                                      qm_stream_t stream) {
    clear_error();
    const ListArgs list = list_args(host_plan, dev_plan, kListAdamW);
    const ListHeader *h = list.h;
    if (!h) return list.st;
    if (h->n_tasks == 0) return QM_OK;
    if (!m_out || !v_out) return fail(QM_E_ARG, "m_out and v_out must not be null");
    if (!aligned(m_out, 16) || !aligned(v_out, 16)) return fail(QM_E_ALIGN, "m_out and v_out need 16-byte alignment");
    const uintptr_t m_at = (uintptr_t)m_out, v_at = (uintptr_t)v_out, bytes = (uintptr_t)h->n_blocks * kBlock * 4;
    if (m_at < v_at + bytes && v_at < m_at + bytes) return fail(QM_E_ARG, "m_out and v_out overlap");
    // Workgroups a CU: as many as fit (8), 6, 3.  States in 8 bits: 4M elements 8.1,
    // 7.8, 9.5 us, 216M 350, 338, 519; in 32 bits: 4M 12.1, 13.5, 13.2, 6M 18.8,
    // 18.1, 17.7, 108M 279, 281, 264; three quarters of the tasks 32 bits: 4M 10.2,
    // 10.7, 11.7, 6M 17.8, 16.6, 16.7, 108M 250, 250, 239; 55 %: 108M 232, 234, 265.
    const unsigned lds = 4 * h->n_tasks32 < 3 * h->n_tasks ? wgs_per_cu(6) : h->n_tasks < 6 << 10 ? 0u : wgs_per_cu(3);
    adamw_read_kernel<<<2 * grid_for(h->n_tasks), kThreads, lds, static_cast<hipStream_t>(stream)>>>(
        list.tensors, list.owner, (int)h->n_tasks, m_out, v_out);
    return launched("AdamW state read");
}
