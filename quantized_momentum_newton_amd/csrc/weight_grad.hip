// The weight gradient of a linear layer, from the gradient of its output and
// its input, the latter in 16 bits or as kept in 8 (act8.hip):
//
//   out[n][k] (= or +=) sum over rows t of dy[t][n] x[t][k]
//
// Both operands hold the contraction index t along their slow axis, which is
// what a training step has in hand, while a matrix instruction wants a lane's
// eight t of one column.  The transposition is done by the LDS reads
// (ds_read_b64_tr_b16 / _b8), so no transposed copy is made.
//
// A kept operand stays in its bytes up to the registers: a fragment is one
// 8-byte read of eight t of a column, and its group of 32 t shares one scale,
// so four conversions with that scale make the bf16 fragment (exact: an E4M3
// number times a power of two).  That is why groups run along the rows.
//
// Tiles of 256 x 256 (eight waves of 128 x 64, fp32 accumulators) or 128 x 128
// (four waves of 64 x 64 or eight of 64 x 32), 64 rows a step, two LDS buffers;
// the rows of the steps after the next are in flight to registers while this one
// is multiplied.  Rows and columns past the ends read as zeros (buffer descriptors
// with their extents), so the loop has no edge cases.  Tiles that do not fill a
// round of the GPU are split over t; their parts go to the workspace and are added
// in order by a second kernel.
//
// What bounds it: 14336 x 4096 over 8192 rows of kept input, 769 us (1251
// TFLOP/s) written and 791 (1216) added to 235 MB; a bf16 product of 8192 cubed
// by the library reaches 1385 over 100 launches, 1190 to 1270 over 20.  The same
// call on zeros takes 586 us: the rest is the clock, which falls to 1.7 GHz under
// the load of real operands.  There the matrix units are busy 66 % of the cycles,
// with LDS reads and writes dealt out between the products (all of a slice's reads
// ahead of its products: 735 us on zeros).  LDS has no bank conflicts and is
// active in 36 % of the cycles.
// Products that leave a CU one 128 tile (1024 x 4096 over 8192 rows, 81 to 89 us) are
// bound by that tile's one wave a SIMD, which issues one thing at a time; where
// there is more to issue than products and their reads, it has two (launch_kind).
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "act_host.h"
#include "list_device.h"
#include "reserve_lds.h"

namespace qm {
namespace {

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8_t;
typedef __attribute__((ext_vector_type(8))) _Float16 f16x8_t;
typedef __attribute__((ext_vector_type(4))) short s16x4_t;
typedef __attribute__((ext_vector_type(2))) int s32x2_t;
typedef __attribute__((ext_vector_type(16))) float f32x16_t;
typedef __attribute__((ext_vector_type(4))) unsigned int u32x4_t;
typedef __attribute__((ext_vector_type(2))) unsigned int u32x2_t;
typedef __attribute__((ext_vector_type(2))) _Float16 f16x2_t;

constexpr int kStep = 64;         // rows t of a step
constexpr int kCus = 256;         // workgroups of a round are counted in these
template <int B> constexpr int kBufStride = 256 * B;      // both operands of a step in 16 bits

struct ProductArgs {
    uint64_t dy, x, scale;        // x: 16-bit elements, or bytes with their scales
    uint64_t out, part;
    int64_t ld_dy, ld_x, ld_out;
    int rows, n, k;
    int tiles_n, tiles_k;
    int whole, rest, splits, split_steps;   // whole tiles, tiles in parts, parts of each, steps of a part
    int out_dtype, accumulate;
    int early_n, early_k;         // the last tiles of n, of k end with the matrix (kAny)
};

// Workgroup barrier that completes this wave's LDS accesses and leaves its
// global loads in flight (the fence of __syncthreads would wait for them).
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// Tile order: bands of four tile rows, walked column by column; consecutive
// workgroups go to the 8 XCDs in turn, and each XCD's share of a round covers
// neighbouring tiles, whose operand panels its L2 then holds once.
__device__ __forceinline__ void tile_at(int p, int tiles_n, int tiles_k, int &bn, int &bk) {
    const int band = p / (4 * tiles_k), r0 = band * 4, h = min(4, tiles_n - r0), q = p - r0 * tiles_k;
    bn = r0 + q % h;
    bk = q / h;
}
// Position i of `count` workgroups, XCD i % 8 taking a contiguous share.
__device__ __forceinline__ int spread(int i, int count) {
    const int x = i & 7, l = i >> 3;
    return x * (count >> 3) + min(x, count & 7) + l;
}

// Descriptor of `bytes` bytes at p, both uniform over the wave (said to the
// compiler, which otherwise loops over the values that lanes might have).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(uint64_t p, int bytes) {
    const uint64_t u = (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(p >> 32)) << 32 |
                       (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)p);
    return __builtin_amdgcn_make_buffer_rsrc((void *)u, 0, __builtin_amdgcn_readfirstlane(bytes), 0x00027000);
}

template <int DT> __device__ __forceinline__ void mfma(const u32x4_t &a, const u32x4_t &b, f32x16_t &c) {
    if constexpr (DT == QM_BF16)
        c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
    else
        c = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c, 0, 0, 0);
}

// Eight kept bytes times their scale, in the product's type.
template <int DT> __device__ __forceinline__ u32x4_t widen(u32x2_t w, float unit) {
    u32x4_t r;
#pragma unroll
    for (int h = 0; h < 2; h++) {
        if constexpr (DT == QM_BF16) {
            r[2 * h] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[h], unit, false));
            r[2 * h + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[h], unit, true));
        } else {
            r[2 * h] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w[h], unit, false));
            r[2 * h + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w[h], unit, true));
        }
    }
    return r;
}

// How a panel is read.  kAligned: 16-byte pieces at 16-byte addresses, rows of
// a multiple of 8 elements (or kept bytes).  kAny: at any address, from a
// matrix of at least B columns: its last panel ends with the matrix and
// overlaps the one before, so no piece is cut.  kNarrow: any address and
// width; pieces that pass a row's end are moved back and shifted.
enum { kAligned = 0, kAny = 1, kNarrow = 2 };

// One operand's 64 x B panel of a step: PIECES 16-byte pieces a thread, kept
// in registers between their loads and the LDS writes.
//
// LDS row t holds the panel's B elements; its 16-byte pieces lie at
// p ^ swizzle(t), so that what one transposing read takes together (four rows
// of 64 bytes, or eight of 32) comes from all banks.
template <int DT, int B, int NT, bool BYTES, int MODE, int DEPTH> struct Panel {
    static constexpr int kSize = BYTES ? 1 : 2, kRow = B * kSize, kPer = 16 / kSize;
    static constexpr int kAcross = kRow / 16, kRowsPass = NT / kAcross, kPieces = kStep / kRowsPass;
    static_assert(kPieces * kRowsPass == kStep && kRowsPass % 8 == 0, "panel split");
    static constexpr int kBytes = kStep * kRow;
    using Raw = std::conditional_t<BYTES, u32x2_t, u32x4_t>;      // a lane's eight t of a column, as they lie in LDS

    u32x4_t r[DEPTH][kPieces];      // DEPTH steps in flight
    uint64_t base;           // row 0 of the matrix, from the panel's first column on
    int64_t pitch;           // bytes
    int col, cols;           // the panel's first column, the matrix's columns
    uint32_t voff, at;       // this thread's first piece: byte offset in the panel, in LDS
    int row, shift, rows[DEPTH];      // unaligned: elements the piece was moved back by; rows of the loads

    static __device__ __forceinline__ int swizzle(int t) {
        if constexpr (!BYTES) return (t & 3) << 2;
        else return kRow == 256 ? (t & 7) << 1 : (t >> 1 & 3) << 1;
    }
    __device__ __forceinline__ Panel(uint64_t p, int64_t ld, int first, int n) {
        base = p + (uint64_t)first * kSize;
        pitch = ld * kSize;
        col = first;
        cols = n;
        row = threadIdx.x / kAcross;
        const int piece = threadIdx.x % kAcross, limit = cols - col;
        at = row * kRow + ((piece ^ swizzle(row)) << 4);
        if constexpr (MODE == kAligned) voff = piece * kPer < limit ? (uint32_t)(row * pitch + piece * 16) : 0x80000000u;
        else if constexpr (MODE == kAny) voff = piece * 16;
        else {
            // the last eight columns of the row where the piece would pass its
            // end; from 8 on nothing of the piece exists
            shift = min(8, max(0, piece * 8 + 8 - limit));
            voff = (uint32_t)max(0, min(col + piece * 8, cols - 8)) * kSize;
            base = p;
        }
    }
    // rows t .. t + 63 below `end`; past it, and past the last column: zeros
    // (of an unaligned panel made by store)
    __device__ __forceinline__ void load(int d, int t, int end) {
        const int have = rows[d] = max(0, min(kStep, end - t));
        if constexpr (MODE == kAligned) {
            // extent: the rows' bytes from the panel's first column on (kept rows
            // are there up to a multiple of 16).  The whole offset is in the
            // vector operand: the scalar one is not part of the bounds check.
            const uint64_t p = base + (uint64_t)((int64_t)t * pitch);
            const int last = BYTES ? (cols - col + 15) / 16 * 16 : (cols - col) * kSize;
            // none without rows: last <= pitch (no branch, which would cut the
            // loop that this stands in)
            const auto rsrc = buffer(p, max(0, (have - 1) * (int)pitch + last));
#pragma unroll
            for (int i = 0; i < kPieces; i++)
                r[d][i] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                                                       rsrc, (int)(voff + (uint32_t)(i * kRowsPass) * (uint32_t)pitch), 0, 0));
        } else if constexpr (MODE == kAny) {
            // rows past the end: the last one's, cleared by store.  Panels are
            // read by several workgroups: loads that stay in the caches.
            const uint64_t p = base + (uint64_t)((int64_t)min(t, end - 1) * pitch);
#pragma unroll
            for (int i = 0; i < kPieces; i++)
                r[d][i] = *reinterpret_cast<const u32x4_e *>(gmem<const char>(p) + voff +
                                                             (uint32_t)max(0, min(row + i * kRowsPass, have - 1)) * (uint32_t)pitch);
        } else {
            static_assert(!BYTES, "kept bytes are aligned");
            if (have == 0) return;
            const uint64_t p = base + (uint64_t)((int64_t)t * pitch);
#pragma unroll
            for (int i = 0; i < kPieces; i++) {
                const uint32_t off = (uint32_t)min(row + i * kRowsPass, have - 1) * (uint32_t)pitch + voff;
                u32x4_e w = {};
                if (cols >= 8) w = *reinterpret_cast<const u32x4_e *>(gmem<const char>(p) + off);
                else {
#pragma unroll
                    for (int j = 0; j < 8; j++)
                        if (j + shift < 8) w[j / 2] |= (unsigned)gmem<const uint16_t>(p + off)[j] << (16 * (j % 2));
                }
                r[d][i] = w;
            }
        }
    }
    __device__ __forceinline__ void store(int d, char *lds) {
        if constexpr (MODE == kAny) {
#pragma unroll
            for (int i = 0; i < kPieces; i++)
#pragma unroll
                for (int j = 0; j < 4; j++) r[d][i][j] = row + i * kRowsPass < rows[d] ? r[d][i][j] : 0;
        }
        if constexpr (MODE == kNarrow) {
            if (rows[d] < kStep || cols - col < B) {
#pragma unroll
                for (int i = 0; i < kPieces; i++) {
                    u32x4_t &v = r[d][i];
                    const int s = cols >= 8 ? shift : shift & 8;
                    if (s & 1) v = u32x4_t{v.x >> 16 | v.y << 16, v.y >> 16 | v.z << 16, v.z >> 16 | v.w << 16, v.w >> 16};
                    if (s & 2) v = u32x4_t{v.y, v.z, v.w, 0};
                    if (s & 4) v = u32x4_t{v.z, v.w, 0, 0};
                    if ((s & 8) || row + i * kRowsPass >= rows[d]) v = u32x4_t{0, 0, 0, 0};
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kPieces; i++)
            *reinterpret_cast<u32x4_t *>(lds + at + i * kRowsPass * kRow) = r[d][i];
    }

    // A lane's part of a fragment read: 32 columns from c0 on, rows 16 s + 8
    // (lane / 32) .. + 7.  16-bit elements: if lane i of 16 points at four
    // elements, lane i receives element i % 4 of lanes i / 4, + 4, + 8, + 12,
    // so with lane i at row i / 4, column 4 (i % 4) it gets column i of four
    // rows.  Bytes: likewise eight rows by 16 columns, lane i at row i / 2,
    // column 8 (i % 2).
    static __device__ __forceinline__ int lane_at(int lane, int c0) {
        const int i = lane & 15;
        const int t = 8 * (lane >> 5) + (BYTES ? i >> 1 : i >> 2);
        const int b = (c0 + 16 * (lane >> 4 & 1)) * kSize + (BYTES ? 8 * (i & 1) : 8 * (i & 3));
        return t * kRow + (((b >> 4) ^ swizzle(t)) << 4) + (b & 15);
    }
    static __device__ __forceinline__ u32x2_t read_b16(const char *p) {
        return __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4_t *)p));
    }
    static __device__ __forceinline__ void read(const char *p, int s, Raw &f) {
        p += 16 * s * kRow;
        if constexpr (BYTES)
            f = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr8_b64_v2i32((__attribute__((address_space(3))) s32x2_t *)p));
        else {
            const u32x2_t lo = read_b16(p), hi = read_b16(p + 4 * kRow);
            f = u32x4_t{lo.x, lo.y, hi.x, hi.y};
        }
    }
};

template <int DT, bool KEPT, int MODE, int B, int WAVES_N, int WAVES_K>
__global__ __launch_bounds__(WAVES_N *WAVES_K * 64, B / WAVES_K == 32 ? 4 : 2) void weight_grad_kernel(ProductArgs a) {
    constexpr int NT = WAVES_N * WAVES_K * 64;
    constexpr int FN = B / WAVES_N / 32, FK = B / WAVES_K / 32, STEPS = kStep / 16;
    // Steps in flight to registers.  A 128 tile's step takes less than a load,
    // and leaves registers for a second.
    constexpr int DEPTH = B == 256 ? 1 : 2;
    using PanelA = Panel<DT, B, NT, false, MODE, DEPTH>;
    using PanelB = Panel<DT, B, NT, KEPT, KEPT ? kAligned : MODE, DEPTH>;
    constexpr int BUF = kBufStride<B>;      // a power of two: the buffers are told apart by one address bit
    static_assert(PanelA::kBytes + PanelB::kBytes + (KEPT ? 2 * B : 0) <= BUF, "LDS buffers");
    extern __shared__ __attribute__((aligned(16))) char lds[];

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int wn = wave / WAVES_K, wk = wave % WAVES_K;
    int tile, t0 = 0, t1 = a.rows;
    uint64_t part = 0;
    // Half of the parts come first, so that the whole tiles behind them end at
    // different times and one half's results leave while the other multiplies.
    const int parts = a.rest * a.splits, early = a.whole ? parts / 2 & ~7 : parts;
    const int w = (int)blockIdx.x - early;
    if (w >= 0 && w < a.whole) {
        // whole: a multiple of 256
        tile = (w >> 8) * 256 + spread(w & 255, 256);
    } else {
        const int p = spread(w < 0 ? (int)blockIdx.x : (int)blockIdx.x - a.whole, parts);
        const int split = p / a.rest, i = p % a.rest;
        tile = a.whole + i;
        t0 = min(a.rows, split * a.split_steps * kStep);
        t1 = min(a.rows, t0 + a.split_steps * kStep);
        if (a.splits > 1) part = a.part + ((uint64_t)i * a.splits + split) * (B * B * 4);
    }
    int bn, bk;
    tile_at(tile, a.tiles_n, a.tiles_k, bn, bk);

    // the tile's first row and column: panels that end with the matrix start early
    const int row_at = MODE == kAny ? min(bn * B, a.n - B) : bn * B;
    const int col_at = MODE == kAny && !KEPT ? min(bk * B, a.k - B) : bk * B;
    PanelA pa(a.dy, a.ld_dy, row_at, a.n);
    PanelB pb(a.x, a.ld_x, col_at, a.k);
    uint32_t off_a[FN], off_b[FK], off_next = 0;      // of the buffer to be read, of the one to be written
    uint32_t off_s = PanelA::kBytes + PanelB::kBytes + wk * FK * 32 + (lane & 31);
#pragma unroll
    for (int i = 0; i < FN; i++) off_a[i] = PanelA::lane_at(lane, wn * FN * 32 + i * 32);
#pragma unroll
    for (int j = 0; j < FK; j++) off_b[j] = PanelA::kBytes + PanelB::lane_at(lane, wk * FK * 32 + j * 32);

    // Scales of a kept step: two groups of 32 rows, B bytes each, one byte a
    // thread, behind the panels in LDS.
    constexpr int SCALES = PanelA::kBytes + PanelB::kBytes;
    static_assert(2 * B <= NT, "a scale byte for each thread");
    uint32_t sc[DEPTH];
    const int sc_group = threadIdx.x / B % 2, sc_col = threadIdx.x % B;
    auto load_scales = [&](int d, int t) {
        if constexpr (KEPT) {
            const int groups = max(0, min(2, (t1 - t + 31) >> 5)), limit = a.k - bk * B;
            const auto rsrc = buffer(a.scale + (uint64_t)((t >> 5) * a.ld_x + bk * B), max(0, (groups - 1) * (int)a.ld_x + limit));
            sc[d] = __builtin_amdgcn_raw_buffer_load_b8(rsrc, sc_col < limit ? sc_col + sc_group * (int)a.ld_x : (int)0x80000000u, 0, 0);
        }
    };
    auto store_scales = [&](int d, char *buf) {
        if constexpr (KEPT) buf[SCALES + threadIdx.x % (2 * B)] = (char)sc[d];
    };

    f32x16_t acc[FN][FK];
#pragma unroll
    for (int i = 0; i < FN; i++)
#pragma unroll
        for (int j = 0; j < FK; j++)
#pragma unroll
            for (int r = 0; r < 16; r++) acc[i][j][r] = 0.0f;

    const int steps = (t1 - t0 + kStep - 1) / kStep;
    // Slices whose fragments are read ahead.  The slice of a wave that has its
    // SIMD to itself (four products, 128 cycles) is shorter than a read.
    constexpr int AHEAD = FN * FK == 4 ? 2 : 1, SETS = 2 * AHEAD;
    u32x4_t fa[SETS][FN];
    typename PanelB::Raw fb[SETS][FK];
    uint32_t unit[2][FK];      // scale bytes of the lane's columns, of both groups
    auto read = [&](int s, u32x4_t *x, typename PanelB::Raw *y) {
        if constexpr (KEPT) {
            if (s % 2 == 0)
#pragma unroll
                for (int j = 0; j < FK; j++) unit[s / 2][j] = (uint8_t)lds[off_s + s / 2 * B + j * 32];
        }
#pragma unroll
        for (int j = 0; j < FK; j++) PanelB::read(lds + off_b[j], s, y[j]);
#pragma unroll
        for (int i = 0; i < FN; i++) PanelA::read(lds + off_a[i], s, x[i]);
    };
    // A step's four slices of 16 rows.  While a slice is multiplied, the
    // fragments of one after it are read into another register set; the barrier
    // between two steps stands before the last AHEAD slices' products, so that
    // those cover the first reads of the next step.  Left alone the compiler moves each
    // read down to its use; issued in one run ahead of the products they would
    // hold up the wave's matrix instructions, and right after a barrier those
    // of every wave.  So each product is followed by its share of the slice's
    // LDS and global accesses.
    constexpr int kProducts = FN * FK, kReads = 2 * FN + 2 * FK;
    auto interleave = [&](auto writes, auto loads) {
        constexpr int W = decltype(writes)::value, V = decltype(loads)::value;
#pragma unroll
        for (int m = 0; m < kProducts; m++) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);      // a matrix product
            __builtin_amdgcn_sched_group_barrier(0x100, (kReads + kProducts - 1) / kProducts, 0);      // LDS reads
            if constexpr (W > 0) __builtin_amdgcn_sched_group_barrier(0x200, (W + kProducts - 1) / kProducts, 0);
            if constexpr (V > 0) __builtin_amdgcn_sched_group_barrier(0x020, (V + kProducts - 1) / kProducts, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    using std::integral_constant;
    if (steps > 0) {
        pa.load(0, t0, t1);
        pb.load(0, t0, t1);
        load_scales(0, t0);
        pa.store(0, lds);
        pb.store(0, lds + PanelA::kBytes);
        store_scales(0, lds);
        off_next = BUF;
#pragma unroll
        for (int d = 0; d < DEPTH; d++) {
            pa.load(d, t0 + (d + 1) * kStep, t1);
            pb.load(d, t0 + (d + 1) * kStep, t1);
            load_scales(d, t0 + (d + 1) * kStep);
        }
        lds_barrier();
#pragma unroll
        for (int s = 0; s < AHEAD; s++) read(s, fa[s], fb[s]);
    }
    // step `it`, whose successor is in the registers d and goes to LDS in the
    // two slices before the barrier
    constexpr int PUT = STEPS - AHEAD - 2;
    auto step = [&](int it, int d) {
        const int ahead = t0 + (it + 1 + DEPTH) * kStep;
#pragma unroll
        for (int s = 0; s < STEPS; s++) {
            const int now = s % SETS, then = (s + AHEAD) % SETS;
            if (s == STEPS - AHEAD) {
                lds_barrier();
                off_s ^= BUF;
#pragma unroll
                for (int i = 0; i < FN; i++) off_a[i] ^= BUF;
#pragma unroll
                for (int j = 0; j < FK; j++) off_b[j] ^= BUF;
                __builtin_amdgcn_sched_barrier(0);
            }
            read((s + AHEAD) % STEPS, fa[then], fb[then]);
            // the other buffer's last readers passed the previous barrier
            if (s == PUT) {
                pa.store(d, lds + off_next);
                pa.load(d, ahead, t1);
            }
            if (s == PUT + 1) {
                pb.store(d, lds + off_next + PanelA::kBytes);
                store_scales(d, lds + off_next);
                off_next ^= BUF;
                pb.load(d, ahead, t1);
                load_scales(d, ahead);
            }
            u32x4_t b[FK];
#pragma unroll
            for (int j = 0; j < FK; j++) {
                if constexpr (KEPT) b[j] = widen<DT>(fb[now][j], __uint_as_float(unit[s / 2][j] << 23));
                else b[j] = fb[now][j];
            }
#pragma unroll
            for (int i = 0; i < FN; i++)
#pragma unroll
                for (int j = 0; j < FK; j++) mfma<DT>(fa[now][i], b[j], acc[i][j]);
            if (s == PUT) interleave(integral_constant<int, PanelA::kPieces>(), integral_constant<int, PanelA::kPieces>());
            else if (s == PUT + 1)
                interleave(integral_constant<int, PanelB::kPieces + KEPT>(), integral_constant<int, PanelB::kPieces + KEPT>());
            else interleave(integral_constant<int, 0>(), integral_constant<int, 0>());
        }
    };
    for (int it = 0; it < steps; it += DEPTH) {
        step(it, 0);
        if constexpr (DEPTH == 2) {
            if (it + 1 < steps) step(it + 1, 1);
        }
    }

    // Element r of a 32 x 32 block: row 8 (r / 4) + 4 (lane / 32) + r % 4,
    // column lane % 32: each store of a wave is two runs of 32 columns.
    const int row0 = wn * FN * 32 + 4 * (lane >> 5), col0 = wk * FK * 32 + (lane & 31);
    if (part) {
#pragma unroll
        for (int i = 0; i < FN; i++)
#pragma unroll
            for (int j = 0; j < FK; j++)
#pragma unroll
                for (int r = 0; r < 16; r++)
                    gmem<float>(part)[(row0 + i * 32 + 8 * (r / 4) + r % 4) * B + col0 + j * 32] = acc[i][j][r];
        return;
    }
    // What does not exist, or is a neighbouring tile's where this one starts
    // early, lies outside the descriptor (rows before its first: negative, so
    // large) or is sent there.
    auto leave = [&](auto dt) {
        constexpr int OT = decltype(dt)::value, S = kSizeOf<OT>;
        const int pitch = (int)a.ld_out * S;
        const auto rsrc = buffer(a.out + (uint64_t)((int64_t)bn * B * a.ld_out + bk * B) * S,
                                 (min(B, a.n - bn * B) - 1) * pitch + (a.k - bk * B) * S);
#pragma unroll
        for (int i = 0; i < FN; i++)
#pragma unroll
            for (int j = 0; j < FK; j++) {
                const int c = col_at - bk * B + col0 + j * 32, n0 = row_at - bn * B + row0 + i * 32;
                const bool there = c >= 0 && c < min(B, a.k - bk * B);
                int at[16];
                float old[16];
#pragma unroll
                for (int r = 0; r < 16; r++) {
                    at[r] = there ? (n0 + 8 * (r / 4) + r % 4) * pitch + c * S : -16;
                    old[r] = 0.0f;
                }
                if (a.accumulate) {
#pragma unroll
                    for (int r = 0; r < 16; r++) {
                        if constexpr (OT == QM_F32) old[r] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rsrc, at[r], 0, 0));
                        else {
                            const uint16_t h = __builtin_amdgcn_raw_buffer_load_b16(rsrc, at[r], 0, 0);
                            old[r] = OT == QM_BF16 ? bf16_val(h) : f16_val(h);
                        }
                    }
                }
#pragma unroll
                for (int r = 0; r < 16; r++) {
                    const float x = in_fp32(old[r] + acc[i][j][r]);
                    if constexpr (OT == QM_F32) __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(x), rsrc, at[r], 0, 0);
                    else __builtin_amdgcn_raw_buffer_store_b16(OT == QM_BF16 ? bf16_rne(x) : f16_rne(x), rsrc, at[r], 0, 0);
                }
            }
    };
    if (a.out_dtype == QM_F32) leave(std::integral_constant<int, QM_F32>());
    else if (a.out_dtype == QM_BF16) leave(std::integral_constant<int, QM_BF16>());
    else leave(std::integral_constant<int, QM_F16>());
}

// The parts of the split tiles, added in order.  A thread takes eight columns
// of a row of the parts; of a tile that starts early, those that are its own.
template <int OT, int B> __global__ __launch_bounds__(256) void weight_grad_join_kernel(ProductArgs a) {
    constexpr int kPerTile = B * B / 8 / 256;
    const int i = blockIdx.x / kPerTile, e = (blockIdx.x % kPerTile) * 256 + threadIdx.x;
    int bn, bk;
    tile_at(a.whole + i, a.tiles_n, a.tiles_k, bn, bk);
    const int row = e / (B / 8), col = e % (B / 8) * 8;
    const int row_at = a.early_n ? min(bn * B, a.n - B) : bn * B, col_at = a.early_k ? min(bk * B, a.k - B) : bk * B;
    const int64_t n = (int64_t)row_at + row, c = (int64_t)col_at + col;
    // the thread's columns from `from` to `to` are this tile's and exist
    const int from = (int)max((int64_t)0, bk * B - c), to = (int)min((int64_t)8, a.k - c);
    if (n < bn * B || n >= a.n || from >= to) return;
    const bool full = from == 0 && to == 8;
    const uint64_t at = a.out + (uint64_t)(n * a.ld_out + c) * kSizeOf<OT>;
    PackedOf<OT, 8> old = {};
    if (a.accumulate) {
        if (full) old = load_bytes<8 * kSizeOf<OT>>(at, 0);
        else {
#pragma unroll
            for (int j = 0; j < 8; j++) {
                if (j < from || j >= to) continue;
                if constexpr (OT == QM_F32) old.w[j] = gmem<const uint32_t>(at)[j];
                else old.w[j / 2] |= (unsigned)gmem<const uint16_t>(at)[j] << (16 * (j % 2));
            }
        }
    }
    float acc[8] = {};
    const uint64_t p = a.part + (uint64_t)i * a.splits * (B * B * 4) + (uint64_t)(row * B + col) * 4;
#pragma unroll 4
    for (int s = 0; s < a.splits; s++) {
        const Packed<32> w = load_bytes<32>(p + (uint64_t)s * (B * B * 4), 0);
#pragma unroll
        for (int j = 0; j < 8; j++) acc[j] += __uint_as_float(w.w[j]);
    }
    float y[8];
#pragma unroll
    for (int j = 0; j < 8; j++) y[j] = in_fp32(unpack<OT>(old, j) + acc[j]);
    if (full) store_bytes(at, 0, qm::pack<OT, 8>(y));
    else {
#pragma unroll
        for (int j = 0; j < 8; j++)
            if (j >= from && j < to) store_one<OT>(at, j, y[j]);
    }
}

// -------------------------------------------------------------------- host

// How a product is cut.
struct Cut {
    int b;                       // tile side
    int tiles_n, tiles_k, whole, rest, splits, split_steps;
    size_t bytes;                // of the parts
};

Cut cut_for(int b, int splits, int64_t rows, int64_t n, int64_t k) {
    Cut c{};
    c.b = b;
    c.tiles_n = (int)((n + b - 1) / b);
    c.tiles_k = (int)((k + b - 1) / b);
    const int64_t tiles = (int64_t)c.tiles_n * c.tiles_k, slots = b == 256 ? kCus : 2 * kCus;
    const int steps = (int)((rows + kStep - 1) / kStep);
    c.whole = (int)(tiles / slots * slots);
    c.rest = (int)(tiles - c.whole);
    c.split_steps = std::max(1, (steps + splits - 1) / splits);
    c.splits = c.rest ? std::max(1, (steps + c.split_steps - 1) / c.split_steps) : 1;
    if (c.splits == 1) c.split_steps = steps;
    c.bytes = c.splits > 1 ? (size_t)c.rest * c.splits * b * b * 4 : 0;
    return c;
}

// Expected microseconds of a cut, from measured steps: a 256 tile's step takes
// 1.7 (kept input 1.55) with one workgroup a CU; a 128 tile's 0.6 alone on its
// CU, 1.0 with a second one, all on aligned panels.  3 + 3 for the launch and what
// a tile starts and ends with; parts are written and read at 5 TB/s, by a launch
// that costs 4.  Panels at odd addresses take up to 1.4 times as long in tiles of
// 128 and 1.2 times in tiles of 256, which is not in the figure.
double cost(const Cut &c, int steps, bool kept) {
    const double full = c.b == 256 ? (kept ? 1.55 : 1.7) : 1.0;
    const int slots = c.b == 256 ? kCus : 2 * kCus, parts = c.rest * c.splits;
    double us = 6 + c.whole / slots * steps * full + parts / slots * c.split_steps * full;
    const int last = parts % slots;
    if (last) us += c.split_steps * (c.b == 128 && last <= kCus ? 0.6 : full);
    if (c.bytes) us += 4 + 2 * c.bytes / 5e6;
    return us;
}

// The cut that should take least.  Measured, cut by cut, and in brackets expected
// (us added to fp32; tile / parts): 2048 x 1008 over 5001 rows 128/1 48 (53), 128/2
// 40 (41), 128/4 43 (43), 256/6 47 (54); 1024 x 4096 over 8192 128/1 88 (83), 128/2
// 87 (87), 256/4 88 (91), from kept input 84, 90 and 84; 1024 x 2048 over 65536
// 256/8 250 (254), 128/4 306 (279); 256 x 256 over 16384 128/8 24 (30), 128/24 17
// (19), 128/64 24 (19); 1000 x 1000 over 300 128/1 9 (9), 128/2 14 (15).  At odd
// addresses 2047 x 1001 over 5001 128/2 51 (41), 128/4 51 (43), 256/8 51 (54).
// Where it takes the slower one: 6144 x 2048 over 8192 128/1 231 (211), 256/1 204
// (224), from kept input the right one, 237 (211) and 191 (204); at odd addresses
// 4097 x 4351 over 3000 128/2 171 (124), 256/6 145 (124).  Sides below 256 take
// tiles of 128: rows at any address are read in tiles that both sides hold.
Cut choose_cut(int64_t rows, int64_t n, int64_t k, bool kept) {
    const int steps = (int)((rows + kStep - 1) / kStep);
    Cut best{};
    double least = INFINITY;
    for (int b = 128; b <= (n < 256 || k < 256 ? 128 : 256); b += 128)
        for (int splits = 1; splits <= std::max(1, std::min(64, steps / 2)); splits++) {
            const Cut c = cut_for(b, splits, rows, n, k);
            const double us = cost(c, steps, kept);
            if (us < least) {
                least = us;
                best = c;
            }
            if (c.rest == 0 || c.rest * (splits + 1) > 8 * kCus) break;
        }
    return best;
}

uint64_t addr(const void *p) { return (uint64_t)(uintptr_t)p; }

template <int DT, bool KEPT, int MODE, int B, int WAVES_N, int WAVES_K>
qm_status launch_product(const ProductArgs &a, hipStream_t q) {
    constexpr size_t lds = kBufStride<B> + kStep * B * (KEPT ? 3 : 4) + (KEPT ? 2 * B : 0);
    auto kern = weight_grad_kernel<DT, KEPT, MODE, B, WAVES_N, WAVES_K>;
    static std::atomic<bool> set[kMaxDevices] = {};
    if (qm_status e = reserve_lds(reinterpret_cast<const void *>(kern), lds, set)) return e;
    kern<<<(unsigned)(a.whole + a.rest * a.splits), WAVES_N * WAVES_K * 64, lds, q>>>(a);
    return launch_status("weight_grad");
}
template <int DT, bool KEPT> qm_status launch_kind(const ProductArgs &a, int mode, int b, hipStream_t q) {
    // Waves of a 128 tile.  Eight, two a SIMD, where pieces are cleared or bytes
    // converted between the products: 2047 x 1001 over 5001 rows 46 us, with four
    // 49; 1024 x 4096 over 8192 kept rows 88 and 93.  Plain aligned panels: four,
    // which read each panel's fragments fewer times: 1024 x 4096 over 8192 rows
    // 92 us, with eight 96; 2560 x 2048 over 2048 43 and 46.
    constexpr int kAlignedWaves = KEPT ? 4 : 2;      // along k, two along n
    if (mode == kNarrow) return launch_product<DT, KEPT, kNarrow, 128, 2, 4>(a, q);
    if (mode == kAligned)
        return b == 256 ? launch_product<DT, KEPT, kAligned, 256, 2, 4>(a, q) : launch_product<DT, KEPT, kAligned, 128, 2, kAlignedWaves>(a, q);
    return b == 256 ? launch_product<DT, KEPT, kAny, 256, 2, 4>(a, q) : launch_product<DT, KEPT, kAny, 128, 2, 4>(a, q);
}
template <int OT> void launch_join(const ProductArgs &a, int b, hipStream_t q) {
    if (b == 256) weight_grad_join_kernel<OT, 256><<<(unsigned)a.rest * 32, 256, 0, q>>>(a);
    else weight_grad_join_kernel<OT, 128><<<(unsigned)a.rest * 8, 256, 0, q>>>(a);
}

bool bad_side(int64_t v) { return v < 0 || v >= (int64_t)1 << 30; }

}  // namespace
}  // namespace qm

using namespace qm;

extern "C" size_t weight_grad_workspace_bytes(int64_t rows, int64_t n, int64_t k) {
    if (bad_side(rows) || bad_side(n) || bad_side(k) || ((n + 127) / 128) * ((k + 127) / 128) >= (int64_t)1 << 22) return 0;
    return std::max(choose_cut(rows, n, k, false).bytes, choose_cut(rows, n, k, true).bytes);
}

extern "C" qm_status weight_grad(const void *dy, int32_t dtype, int64_t ld_dy, const void *x, int64_t ld_x,
                                 const qm_act8 *kept, int64_t rows, int64_t n, int64_t k, void *out, int32_t out_dtype,
                                 int64_t ld_out, int32_t accumulate, void *ws, size_t ws_bytes, qm_stream_t stream) {
    clear_error();
    if (dtype != QM_BF16 && dtype != QM_F16) return fail(QM_E_DTYPE, "dy must be bf16 or f16");
    if (accumulate != 0 && accumulate != 1) return fail(QM_E_ARG, "accumulate must be 0 or 1");
    if (bad_side(rows) || bad_side(n) || bad_side(k)) return fail(QM_E_SHAPE, "rows, n and k are 0 to 2^30 - 1");
    if (!x == !kept && rows && k) return fail(QM_E_ARG, "either x or kept");
    if (qm_status e = check_matrix("dy", dy, dtype, rows, n, ld_dy)) return e;
    if (kept) {
        if (qm_status e = check_kept("kept", kept, rows, k)) return e;
    } else if (qm_status e = check_matrix("x", x, dtype, rows, k, ld_x)) return e;
    if (qm_status e = check_matrix("out", out, out_dtype, n, k, ld_out)) return e;
    if (n == 0 || k == 0 || (rows == 0 && accumulate)) return QM_OK;
    // 256 rows within a 31-bit byte offset
    if (ld_out >= (int64_t)1 << 21) return fail(QM_E_SHAPE, "out: row pitch above 2^21 - 1");
    if (((n + 127) / 128) * ((k + 127) / 128) >= (int64_t)1 << 22) return fail(QM_E_UNSUPPORTED, "more than 2^22 tiles of 128 x 128");
    const Cut c = choose_cut(rows, n, k, kept != nullptr);
    if (c.bytes) {
        if (!ws || ws_bytes < c.bytes) return fail(QM_E_WORKSPACE, "workspace: need %zu bytes", c.bytes);
        if (!aligned(ws, 16)) return fail(QM_E_ALIGN, "workspace needs 16-byte alignment");
    }
    Spans s;
    s.matrix(dy, dtype, rows, n, ld_dy, false);
    if (kept) s.kept(kept, false);
    else s.matrix(x, dtype, rows, k, ld_x, false);
    s.matrix(out, out_dtype, n, k, ld_out, true);
    if (c.bytes) s.bytes(ws, (int64_t)c.bytes, true);
    if (s.clash()) return fail(QM_E_ARG, "out or workspace overlaps another buffer");
    ProductArgs a{};
    a.dy = addr(dy), a.ld_dy = ld_dy;
    a.x = kept ? addr(kept->data) : addr(x), a.ld_x = kept ? kept->ld : ld_x;
    a.scale = kept ? addr(kept->scale) : 0;
    a.out = addr(out), a.ld_out = ld_out, a.part = addr(ws);
    a.rows = (int)rows, a.n = (int)n, a.k = (int)k;
    a.tiles_n = c.tiles_n, a.tiles_k = c.tiles_k, a.whole = c.whole, a.rest = c.rest;
    a.splits = c.splits, a.split_steps = c.split_steps;
    a.out_dtype = out_dtype, a.accumulate = accumulate;
    auto wide = [](const void *p, int64_t ld, int64_t cols) { return aligned(p, 16) && ld % 8 == 0 && cols % 8 == 0; };
    int mode = kAligned;
    if (!wide(dy, ld_dy, n) || !(kept || wide(x, ld_x, k))) mode = n >= c.b && (kept || k >= c.b) ? kAny : kNarrow;
    a.early_n = mode == kAny, a.early_k = mode == kAny && !kept;
    const hipStream_t q = static_cast<hipStream_t>(stream);
    const bool bf = dtype == QM_BF16;
    qm_status e;
    if (kept) e = bf ? launch_kind<QM_BF16, true>(a, mode, c.b, q) : launch_kind<QM_F16, true>(a, mode, c.b, q);
    else e = bf ? launch_kind<QM_BF16, false>(a, mode, c.b, q) : launch_kind<QM_F16, false>(a, mode, c.b, q);
    if (e) return e;
    if (c.splits == 1) return QM_OK;
    if (out_dtype == QM_F32) launch_join<QM_F32>(a, c.b, q);
    else if (out_dtype == QM_BF16) launch_join<QM_BF16>(a, c.b, q);
    else launch_join<QM_F16>(a, c.b, q);
    return launch_status("weight_grad");
}
