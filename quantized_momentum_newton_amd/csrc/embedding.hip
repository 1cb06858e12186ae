// Embedding lookup with a scale, and its gradient.
//
//   out[i, :]  = scale * table[tok_i, :]                  (zeros for tok_i outside the table)
//   grad[v, :] (= or +=) scale * sum of dy[i, :] over tok_i = v
//
// The sum has a fixed order, so a gradient repeats bit for bit: the tokens are
// sorted by value, equal ones by position, and a row of the table is the sum
// of its tokens in that order.  Three launches:
//
//   sort   Each workgroup owns a range of the vocabulary (at most 1024
//          values) and reads every token twice, which 256 workgroups do from
//          their caches as fast as one does.  What lies below its range tells
//          it where its own part of the order starts, so no workgroup waits
//          for another.  Counts are per wave and value: a wave owns a
//          contiguous part of the tokens, so (value, wave, position) is the
//          order, and the place of equal values among a wave's 64 comes from
//          one ballot per bit of the value.
//   sum    A row of at most 64 tokens is summed by one wave (per 512 columns)
//          and stored.  Longer rows are cut where multiples of 64 positions
//          of the order lie: a cut part is summed by one wave into the
//          workspace.  A gradient that is written whole also gets its zeros
//          here, one that is added to is touched in rows that have tokens.
//   join   The parts of a long row are added, in order, by one workgroup.
#include <algorithm>
#include <type_traits>

#include "act_host.h"
#include "list_device.h"

namespace qm {
namespace {

constexpr int kChunk = 64;        // positions of a part, and the longest row without parts
constexpr int kSortWaves = 16, kSortValues = 1024;
constexpr int kSumWaves = 4, kJoinWaves = 8;
constexpr int64_t kMaxTokens = (int64_t)1 << 30;     // tokens, and values: their counts stay 32-bit numbers

// A lane's n <= 8 elements at `at` as fp32.
template <int DT> __device__ __forceinline__ void load_cols(uint64_t at, int n, float *x) {
    PackedOf<DT, 8> r = {};
    if (n == 8) r = load_bytes<8 * kSizeOf<DT>>(at, 0);
    else {
#pragma unroll
        for (int j = 0; j < 8; j++) {
            if (j >= n) continue;
            if constexpr (DT == QM_F32) r.w[j] = gmem<const uint32_t>(at)[j];
            else r.w[j / 2] |= (unsigned)gmem<const uint16_t>(at)[j] << (16 * (j % 2));
        }
    }
#pragma unroll
    for (int j = 0; j < 8; j++) x[j] = unpack<DT>(r, j);
}
template <int DT> __device__ __forceinline__ void store_cols(uint64_t at, int n, const float *x) {
    if (n == 8) {
        store_bytes(at, 0, qm::pack<DT, 8>(x));
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; j++)
        if (j < n) store_one<DT>(at, j, x[j]);
}

__device__ __forceinline__ int64_t token_at(uint64_t tokens, int bits, int64_t i) {
    return bits == 64 ? gmem<const int64_t>(tokens)[i] : (int64_t)gmem<const int32_t>(tokens)[i];
}

// ------------------------------------------------------------------ lookup

struct LookupArgs {
    uint64_t tokens, table, out;
    int64_t n_tokens, ld_table, ld_out;
    int vocab, cols, pieces, token_bits;     // pieces: of 8 columns, in a row
    float scale;
};

constexpr int kLookupThreads = 256, kLookupEach = 4;

template <int DT, int OUT> __global__ __launch_bounds__(kLookupThreads) void embedding_lookup_kernel(LookupArgs a) {
    // the workgroup's pieces follow one another through rows and columns
    const int64_t first = (int64_t)blockIdx.x * (kLookupThreads * kLookupEach);
    const int64_t row0 = first / a.pieces;
    const uint32_t at0 = (uint32_t)(first - row0 * a.pieces);
    int64_t row[kLookupEach], tok[kLookupEach];
    int col[kLookupEach];
#pragma unroll
    for (int k = 0; k < kLookupEach; k++) {
        const uint32_t at = at0 + k * kLookupThreads + threadIdx.x;
        row[k] = row0 + at / (uint32_t)a.pieces;
        col[k] = (int)(at % (uint32_t)a.pieces) * 8;
        tok[k] = row[k] < a.n_tokens ? token_at(a.tokens, a.token_bits, row[k]) : -1;
    }
    float x[kLookupEach][8];
#pragma unroll
    for (int k = 0; k < kLookupEach; k++) {
        const bool inside = (uint64_t)tok[k] < (uint64_t)a.vocab;
        const int n = inside ? min(8, a.cols - col[k]) : 0;
        load_cols<DT>(a.table + (uint64_t)(tok[k] * a.ld_table + col[k]) * kSizeOf<DT>, n, x[k]);
    }
#pragma unroll
    for (int k = 0; k < kLookupEach; k++) {
        if (row[k] >= a.n_tokens) continue;
#pragma unroll
        for (int j = 0; j < 8; j++) x[k][j] = in_fp32(x[k][j] * a.scale);
        store_cols<OUT>(a.out + (uint64_t)(row[k] * a.ld_out + col[k]) * kSizeOf<OUT>, min(8, a.cols - col[k]), x[k]);
    }
}

// -------------------------------------------------------------------- sort

struct Sorted {
    int32_t token, position;
};

struct SortArgs {
    uint64_t tokens, sorted, start;      // sorted: Sorted [n], start: int32 [vocab + 1]
    int n, vocab, token_bits;
    int values, value_bits;              // of a workgroup
};

__global__ __launch_bounds__(kSortWaves * 64) void embedding_sort_kernel(SortArgs a) {
    __shared__ int32_t count[kSortWaves * kSortValues];      // per wave and value: how many, then where the next goes
    __shared__ int32_t wave_total[kSortWaves], wave_less[kSortWaves];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int lo = blockIdx.x * a.values, values = min(a.values, a.vocab - lo);
    for (int i = threadIdx.x; i < kSortWaves * a.values; i += kSortWaves * 64) count[i] = 0;
    __syncthreads();
    const int share = (a.n + kSortWaves * 64 - 1) / (kSortWaves * 64) * 64;
    const int begin = min(wave * share, a.n), end = min(begin + share, a.n);
    int32_t *mine = count + wave * a.values;

    constexpr int kAhead = 4;    // tokens of a lane in flight
    int less = 0;
    for (int c = begin; c < end; c += 64 * kAhead) {
        int64_t t[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; k++) {
            const int i = c + k * 64 + lane;
            t[k] = i < end ? token_at(a.tokens, a.token_bits, i) : -1;
        }
#pragma unroll
        for (int k = 0; k < kAhead; k++) {
            less += t[k] >= 0 && t[k] < lo;
            if (t[k] >= lo && t[k] < lo + values) atomicAdd(&mine[t[k] - lo], 1);
        }
    }
    for (int k = 1; k < 64; k *= 2) less += __shfl_xor(less, k);
    if (lane == 0) wave_less[wave] = less;
    __syncthreads();

    // where each value's and each wave's share of it start
    const int v = threadIdx.x;
    int total = 0;
    if (v < values)
        for (int w = 0; w < kSortWaves; w++) total += count[w * a.values + v];
    int upto = total;
    for (int k = 1; k < 64; k *= 2) {
        const int o = __shfl_up(upto, k);
        if (lane >= k) upto += o;
    }
    if (lane == 63) wave_total[wave] = upto;
    __syncthreads();
    int at = upto - total, all = 0;
    for (int w = 0; w < kSortWaves; w++) {
        at += wave_less[w] + (w < wave ? wave_total[w] : 0);
        all += wave_less[w] + wave_total[w];
    }
    if (v < values) {
        gmem<int32_t>(a.start)[lo + v] = at;
        for (int w = 0; w < kSortWaves; w++) {
            const int c = count[w * a.values + v];
            count[w * a.values + v] = at;
            at += c;
        }
    }
    if (threadIdx.x == 0 && lo + values == a.vocab) gmem<int32_t>(a.start)[a.vocab] = all;
    __syncthreads();

    for (int c = begin; c < end; c += 64 * kAhead) {
        int64_t t[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; k++) {
            const int i = c + k * 64 + lane;
            t[k] = i < end ? token_at(a.tokens, a.token_bits, i) : -1;
        }
#pragma unroll
        for (int k = 0; k < kAhead; k++) {
            const bool in = t[k] >= lo && t[k] < lo + values;
            uint64_t same = __ballot(in);
            if (same == 0) continue;
            const int value = in ? (int)(t[k] - lo) : 0;
            for (int b = 0; b < a.value_bits; b++) {
                const uint64_t set = __ballot(value >> b & 1);
                same &= value >> b & 1 ? set : ~set;
            }
            if (in) {
                const int before = __popcll(same & ((1ull << lane) - 1)), next = mine[value];
                if (before == 0) mine[value] = next + __popcll(same);
                gmem<Sorted>(a.sorted)[next + before] = Sorted{(int32_t)t[k], c + k * 64 + lane};
            }
        }
    }
}

// --------------------------------------------------------------------- sum

struct SumArgs {
    uint64_t sorted, start, head, part, dy, grad;
    int64_t ld_dy, ld_grad;
    int vocab, cols, n_tokens;
    int slabs, part_ld;      // slabs: of 8 * lanes columns; part_ld: columns rounded up to 8
    int chunks, rows;        // units of the launch: chunks * slabs, then rows * slabs
    int accumulate;
    float scale;
};

__device__ __forceinline__ Sorted sorted_at(uint64_t sorted, int i) { return gmem<const Sorted>(sorted)[i]; }
__device__ __forceinline__ int start_of(uint64_t start, int v) { return gmem<const int32_t>(start)[v]; }

// acc = the dy rows of positions first .. first + n - 1 of the order, in that
// order; n >= 1.
template <int DT> __device__ __forceinline__ void sum_positions(const SumArgs &a, int first, int n, int col, int cols, float *acc) {
    constexpr int kAhead = 4;     // rows in flight
    const uint64_t base = a.dy + (uint64_t)col * kSizeOf<DT>;
    load_cols<DT>(base + (uint64_t)(sorted_at(a.sorted, first).position * a.ld_dy) * kSizeOf<DT>, cols, acc);
    for (int k = 1; k < n; k += kAhead) {
        float x[kAhead][8];
        int at[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; u++) at[u] = sorted_at(a.sorted, first + min(k + u, n - 1)).position;
#pragma unroll
        for (int u = 0; u < kAhead; u++) load_cols<DT>(base + (uint64_t)(at[u] * a.ld_dy) * kSizeOf<DT>, cols, x[u]);
#pragma unroll
        for (int u = 0; u < kAhead; u++)
#pragma unroll
            for (int j = 0; j < 8; j++) acc[j] += k + u < n ? x[u][j] : 0.0f;
    }
}

template <int GT> __device__ __forceinline__ void finish_row(const SumArgs &a, int token, int col, int cols, const float *acc) {
    const uint64_t at = a.grad + (uint64_t)(token * a.ld_grad + col) * kSizeOf<GT>;
    float y[8] = {};
    if (a.accumulate) load_cols<GT>(at, cols, y);
#pragma unroll
    for (int j = 0; j < 8; j++) y[j] = in_fp32(y[j] + a.scale * acc[j]);
    store_cols<GT>(at, cols, y);
}

template <int DT, int GT, int LANES> __global__ __launch_bounds__(kSumWaves * 64) void embedding_sum_kernel(SumArgs a) {
    const int lane = threadIdx.x % LANES;
    const int64_t unit = (int64_t)blockIdx.x * (kSumWaves * 64 / LANES) + threadIdx.x / LANES;
    const int64_t chunk_units = (int64_t)a.chunks * a.slabs;
    const int slab = (int)(unit % a.slabs), col = slab * LANES * 8 + lane * 8;
    const int cols = max(0, min(8, a.cols - col));
    float acc[8];
    if (unit < chunk_units) {
        // the parts of long rows that end, pass through or start in this chunk
        const int chunk = (int)(unit / a.slabs), n_sorted = start_of(a.start, a.vocab);
        const int first = chunk * kChunk, last = min(first + kChunk, n_sorted) - 1;
        int head = -1;
        if (first <= last) {
            const int t0 = sorted_at(a.sorted, first).token, t1 = sorted_at(a.sorted, last).token;
            const uint64_t part = a.part + ((uint64_t)chunk * 2 * a.part_ld + col) * 4;
            const int s0 = start_of(a.start, t0), e0 = start_of(a.start, t0 + 1);
            if (e0 - s0 > kChunk) {
                if (s0 == first) head = t0;
                if (cols) {
                    sum_positions<DT>(a, first, min(e0 - 1, last) - first + 1, col, cols, acc);
                    store_cols<QM_F32>(part, cols, acc);
                }
            }
            const int s1 = start_of(a.start, t1), e1 = start_of(a.start, t1 + 1);
            if (t1 != t0 && e1 - s1 > kChunk) {
                head = t1;
                if (cols) {
                    sum_positions<DT>(a, s1, last - s1 + 1, col, cols, acc);
                    store_cols<QM_F32>(part + (uint64_t)a.part_ld * 4, cols, acc);
                }
            }
        }
        if (slab == 0 && lane == 0) gmem<int32_t>(a.head)[chunk] = head;
        return;
    }
    const int64_t row = (unit - chunk_units) / a.slabs;
    if (row >= a.rows) return;
    int token, first, n;
    if (a.accumulate) {      // one unit a position: the first of each row is taken
        first = (int)row;
        if (first >= start_of(a.start, a.vocab)) return;
        token = sorted_at(a.sorted, first).token;
        if (first > 0 && sorted_at(a.sorted, first - 1).token == token) return;
        n = start_of(a.start, token + 1) - first;
    } else {
        token = (int)row;
        first = start_of(a.start, token);
        n = start_of(a.start, token + 1) - first;
    }
    if (n > kChunk || !cols) return;
    if (n > 0) sum_positions<DT>(a, first, n, col, cols, acc);
    else
#pragma unroll
        for (int j = 0; j < 8; j++) acc[j] = 0.0f;
    finish_row<GT>(a, token, col, cols, acc);
}

// One workgroup per chunk and 512 columns; those in whose chunk no long row
// starts have nothing to do.
template <int GT> __global__ __launch_bounds__(kJoinWaves * 64) void embedding_join_kernel(SumArgs a) {
    __shared__ float sums[kJoinWaves][512];
    const int slabs = (a.cols + 511) / 512;
    const int chunk = blockIdx.x / slabs, slab = blockIdx.x % slabs;
    const int token = gmem<const int32_t>(a.head)[chunk];
    if (token < 0) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int col = slab * 512 + lane * 8, cols = max(0, min(8, a.cols - col));
    const int s = start_of(a.start, token), last = (start_of(a.start, token + 1) - 1) / kChunk;
    // wave w adds an eighth of the parts, contiguous, so that the order stays
    const int parts = last - chunk + 1, each = (parts + kJoinWaves - 1) / kJoinWaves;
    const int p0 = min(wave * each, parts), p1 = min(p0 + each, parts);
    float acc[8] = {};
    constexpr int kAhead = 4;
    for (int p = p0; p < p1; p += kAhead) {
        float x[kAhead][8];
#pragma unroll
        for (int u = 0; u < kAhead; u++) {
            const int c = chunk + min(p + u, p1 - 1);
            const int slot = c == chunk && s % kChunk != 0 ? 1 : 0;
            load_cols<QM_F32>(a.part + (((uint64_t)c * 2 + slot) * a.part_ld + col) * 4, cols, x[u]);
        }
#pragma unroll
        for (int u = 0; u < kAhead; u++)
#pragma unroll
            for (int j = 0; j < 8; j++) acc[j] += p + u < p1 ? x[u][j] : 0.0f;
    }
#pragma unroll
    for (int j = 0; j < 8; j++) sums[wave][lane * 8 + j] = acc[j];
    __syncthreads();
    if (wave != 0 || !cols) return;
    for (int w = 1; w < kJoinWaves; w++)
#pragma unroll
        for (int j = 0; j < 8; j++) acc[j] += sums[w][lane * 8 + j];
    finish_row<GT>(a, token, col, cols, acc);
}

// -------------------------------------------------------------------- host

uint64_t addr(const void *p) { return (uint64_t)(uintptr_t)p; }

template <typename F> void with_dtype(int32_t dtype, F f) {
    if (dtype == QM_F32) f(std::integral_constant<int, QM_F32>());
    else if (dtype == QM_BF16) f(std::integral_constant<int, QM_BF16>());
    else f(std::integral_constant<int, QM_F16>());
}

qm_status check_tokens(const void *tokens, int32_t token_bits, int64_t n_tokens, int64_t vocab) {
    if (token_bits != 32 && token_bits != 64) return fail(QM_E_DTYPE, "tokens have 32 or 64 bits, not %d", token_bits);
    if (n_tokens < 0 || n_tokens >= kMaxTokens) return fail(QM_E_SHAPE, "bad number of tokens");
    if (vocab < 0 || vocab >= kMaxTokens) return fail(QM_E_SHAPE, "bad vocabulary");
    if (n_tokens && !tokens) return fail(QM_E_ARG, "tokens is null");
    if (n_tokens && !aligned(tokens, token_bits / 8)) return fail(QM_E_ALIGN, "tokens must be aligned to their size");
    return QM_OK;
}

// The workspace of embedding_grad: offsets of its arrays.
struct Space {
    size_t sorted, start, head, part, bytes;
    int64_t chunks, part_ld;
    Space(int64_t n_tokens, int64_t vocab, int64_t cols) {
        auto up = [](size_t n) { return (n + 255) / 256 * 256; };
        chunks = n_tokens > kChunk ? (n_tokens + kChunk - 1) / kChunk : 0;
        part_ld = (cols + 7) / 8 * 8;
        sorted = 0;
        start = up((size_t)n_tokens * sizeof(Sorted));
        head = start + up((size_t)(vocab + 1) * 4);
        part = head + up((size_t)chunks * 4);
        bytes = part + up((size_t)chunks * 2 * part_ld * 4);
    }
};

}  // namespace
}  // namespace qm

using namespace qm;

extern "C" qm_status embedding_lookup(const void *tokens, int32_t token_bits, int64_t n_tokens, const void *table,
                                      int32_t table_dtype, int64_t ld_table, int64_t vocab, int64_t cols, float scale,
                                      void *out, int32_t out_dtype, int64_t ld_out, qm_stream_t stream) {
    clear_error();
    if (qm_status e = check_tokens(tokens, token_bits, n_tokens, vocab)) return e;
    if (qm_status e = check_matrix("table", table, table_dtype, vocab, cols, ld_table)) return e;
    if (qm_status e = check_matrix("out", out, out_dtype, n_tokens, cols, ld_out)) return e;
    if (n_tokens == 0 || cols == 0) return QM_OK;
    Spans s;
    s.bytes(tokens, n_tokens * (token_bits / 8), false);
    s.matrix(table, table_dtype, vocab, cols, ld_table, false);
    s.matrix(out, out_dtype, n_tokens, cols, ld_out, true);
    if (s.clash()) return fail(QM_E_ARG, "out overlaps another buffer");
    const int64_t pieces = (cols + 7) / 8, each = kLookupThreads * kLookupEach, wgs = (n_tokens * pieces + each - 1) / each;
    if (wgs >= (int64_t)1 << 24) return fail(QM_E_UNSUPPORTED, "more than 2^34 pieces of 8 columns");
    const LookupArgs a{addr(tokens), addr(table), addr(out), n_tokens, ld_table, ld_out, (int)vocab, (int)cols, (int)pieces,
                       token_bits, scale};
    with_dtype(table_dtype, [&](auto dt) {
        with_dtype(out_dtype, [&](auto ot) {
            embedding_lookup_kernel<decltype(dt)::value, decltype(ot)::value>
                <<<(unsigned)wgs, kLookupThreads, 0, static_cast<hipStream_t>(stream)>>>(a);
        });
    });
    return launch_status("embedding_lookup");
}

extern "C" size_t embedding_grad_workspace_bytes(int64_t n_tokens, int64_t vocab, int64_t cols) {
    if (n_tokens < 0 || vocab < 0 || cols < 0 || n_tokens >= kMaxTokens || vocab >= kMaxTokens || cols > kMaxPitch) return 0;
    return Space(n_tokens, vocab, cols).bytes;
}

extern "C" qm_status embedding_grad(const void *tokens, int32_t token_bits, int64_t n_tokens, const void *dy,
                                    int32_t dy_dtype, int64_t ld_dy, void *grad, int32_t grad_dtype, int64_t ld_grad,
                                    int64_t vocab, int64_t cols, float scale, int32_t accumulate, void *ws,
                                    size_t ws_bytes, qm_stream_t stream) {
    clear_error();
    if (accumulate != 0 && accumulate != 1) return fail(QM_E_ARG, "accumulate must be 0 or 1");
    if (qm_status e = check_tokens(tokens, token_bits, n_tokens, vocab)) return e;
    if (qm_status e = check_matrix("dy", dy, dy_dtype, n_tokens, cols, ld_dy)) return e;
    if (qm_status e = check_matrix("grad", grad, grad_dtype, vocab, cols, ld_grad)) return e;
    if (vocab == 0 || cols == 0 || (n_tokens == 0 && accumulate)) return QM_OK;
    const Space sp(n_tokens, vocab, cols);
    if (!ws || ws_bytes < sp.bytes) return fail(QM_E_WORKSPACE, "workspace: need %zu bytes", sp.bytes);
    if (!aligned(ws, 16)) return fail(QM_E_ALIGN, "workspace needs 16-byte alignment");
    Spans s;
    s.bytes(tokens, n_tokens * (token_bits / 8), false);
    s.matrix(dy, dy_dtype, n_tokens, cols, ld_dy, false);
    s.matrix(grad, grad_dtype, vocab, cols, ld_grad, true);
    s.bytes(ws, (int64_t)sp.bytes, true);
    if (s.clash()) return fail(QM_E_ARG, "grad or workspace overlaps another buffer");

    const uint64_t w = addr(ws);
    // 256 workgroups where the vocabulary allows it
    const int values = (int)std::min<int64_t>(kSortValues, (vocab + 255) / 256);
    int value_bits = 0;
    while ((1 << value_bits) < values) value_bits++;
    const SortArgs sort{addr(tokens), w + sp.sorted, w + sp.start, (int)n_tokens, (int)vocab, token_bits, values, value_bits};
    const int lanes = cols <= 64 ? 8 : cols <= 128 ? 16 : cols <= 256 ? 32 : 64;
    SumArgs a{};
    a.sorted = sort.sorted, a.start = sort.start, a.head = w + sp.head, a.part = w + sp.part;
    a.dy = addr(dy), a.grad = addr(grad), a.ld_dy = ld_dy, a.ld_grad = ld_grad;
    a.vocab = (int)vocab, a.cols = (int)cols, a.n_tokens = (int)n_tokens;
    a.slabs = (int)((cols + lanes * 8 - 1) / (lanes * 8)), a.part_ld = (int)sp.part_ld;
    a.chunks = (int)sp.chunks, a.rows = accumulate ? (int)n_tokens : (int)vocab;
    a.accumulate = accumulate, a.scale = scale;
    const int64_t units = ((int64_t)a.chunks + a.rows) * a.slabs, each = kSumWaves * 64 / lanes;
    const int64_t sum_wgs = (units + each - 1) / each, join_wgs = sp.chunks * ((cols + 511) / 512);
    if (sum_wgs >= (int64_t)1 << 24 || join_wgs >= (int64_t)1 << 23)
        return fail(QM_E_UNSUPPORTED, "more than 2^32 threads");
    const hipStream_t q = static_cast<hipStream_t>(stream);
    embedding_sort_kernel<<<(unsigned)((vocab + values - 1) / values), kSortWaves * 64, 0, q>>>(sort);
    if (qm_status e = launch_status("embedding_grad")) return e;
    with_dtype(dy_dtype, [&](auto dt) {
        with_dtype(grad_dtype, [&](auto gt) {
            constexpr int DT = decltype(dt)::value, GT = decltype(gt)::value;
            const unsigned grid = (unsigned)sum_wgs;
            if (lanes == 8) embedding_sum_kernel<DT, GT, 8><<<grid, kSumWaves * 64, 0, q>>>(a);
            else if (lanes == 16) embedding_sum_kernel<DT, GT, 16><<<grid, kSumWaves * 64, 0, q>>>(a);
            else if (lanes == 32) embedding_sum_kernel<DT, GT, 32><<<grid, kSumWaves * 64, 0, q>>>(a);
            else embedding_sum_kernel<DT, GT, 64><<<grid, kSumWaves * 64, 0, q>>>(a);
        });
    });
    if (qm_status e = launch_status("embedding_grad")) return e;
    if (join_wgs == 0) return QM_OK;
    with_dtype(grad_dtype, [&](auto gt) { embedding_join_kernel<decltype(gt)::value><<<(unsigned)join_wgs, kJoinWaves * 64, 0, q>>>(a); });
    return launch_status("embedding_grad");
}
