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
//          values) and looks at every token twice, which 256 workgroups do from
//          their caches as fast as one does (up to 32768 tokens are read once
//          and kept in registers).  What lies below its range tells
//          it where its own part of the order starts, so no workgroup waits
//          for another.  Counts are per wave and value: a wave owns a
//          contiguous part of the tokens, so (value, wave, position) is the
//          order, and the place of equal values among a wave's 64 comes from
//          one ballot per bit of the value, or per value where those are fewer.
//   sum    A wave takes the rows that start in a range of up to 16 positions of
//          the order (per 1024 columns) and runs through their tokens, several rows
//          of dy in flight whichever row of the table they go to.  Rows of more
//          than 32 tokens are cut where multiples of 32 positions lie: a cut
//          part is summed by one wave into the workspace.  A gradient that is
//          written whole also gets its zeros here, one that is added to is
//          touched in rows that have tokens.
//   join   The parts of a long row are added, in order, by one workgroup.
//
// 50257 x 2048 fp32 written whole from 32768 skewed tokens: sort 20 us, sum 104 to
// 121 (412 MB written, 134 read: 84 at the rate of a large copy), join 9; the sort
// is bound by its instructions (256 workgroups look at every token; 131072 tokens
// of 64 columns 74 us, 32768 25, one value only 316 and 91: one workgroup then
// places all), the sum by the latency of start, order and rows in turn.  No tokens:
// 79 us, torch's fill 61.  Added to 32000 x 4096 bf16 from 16384 tokens: 13, 54 and
// 9 us.  The lookup of 32768 such rows takes 60 us, 47 at the rate of a large copy
// by the bytes that it moves.
#include <algorithm>
#include <type_traits>

#include "act_host.h"
#include "list_device.h"

namespace qm {
namespace {

constexpr int kChunk = 32;        // positions of a part, and the longest row without parts
constexpr int kSortWaves = 16, kSortValues = 1024;
constexpr int kSumWaves = 4, kJoinWaves = 8, kJoinChunks = 8;
constexpr int kRange = 16;        // most positions whose rows a wave starts
constexpr int kFill = 16;         // rows that a wave looks at for empty ones
constexpr int64_t kMaxTokens = (int64_t)1 << 30;     // tokens, and values: their counts stay 32-bit numbers

// A lane's n <= V elements at `at` as fp32.  V is 8 where everything a kernel
// moves has 16 bits and 4 where a part has 32: an access of a wave is then one
// run of 1 KiB of the widest type, and never every other 16 bytes of one.
template <int DT, int V> __device__ __forceinline__ void load_cols(uint64_t at, int n, float *x) {
    PackedOf<DT, V> r = {};
    if (n == V) r = load_bytes<V * kSizeOf<DT>>(at, 0);
    else {
#pragma unroll
        for (int j = 0; j < V; j++) {
            if (j >= n) continue;
            if constexpr (DT == QM_F32) r.w[j] = gmem<const uint32_t>(at)[j];
            else r.w[j / 2] |= (unsigned)gmem<const uint16_t>(at)[j] << (16 * (j % 2));
        }
    }
#pragma unroll
    for (int j = 0; j < V; j++) x[j] = unpack<DT>(r, j);
}
template <int DT, int V> __device__ __forceinline__ void store_cols(uint64_t at, int n, const float *x) {
    if (n == V) {
        store_bytes(at, 0, qm::pack<DT, V>(x));
        return;
    }
#pragma unroll
    for (int j = 0; j < V; j++)
        if (j < n) store_one<DT>(at, j, x[j]);
}

__device__ __forceinline__ int64_t token_at(uint64_t tokens, int bits, int64_t i) {
    return bits == 64 ? gmem<const int64_t>(tokens)[i] : (int64_t)gmem<const int32_t>(tokens)[i];
}

// The token as a 32-bit number, what a table cannot have as the largest.
__device__ __forceinline__ uint32_t token32_at(uint64_t tokens, int bits, int64_t i) {
    if (bits == 32) return gmem<const uint32_t>(tokens)[i];      // negative: large
    const uint64_t t = gmem<const uint64_t>(tokens)[i];
    return t >> 32 ? 0xffffffffu : (uint32_t)t;
}

// ------------------------------------------------------------------ lookup

struct LookupArgs {
    uint64_t tokens, table, out;
    int64_t n_tokens, ld_table, ld_out;
    int vocab, cols, pieces, token_bits;     // pieces: of a thread's columns, in a row
    float scale;
};

constexpr int kLookupThreads = 256, kLookupEach = 4;
template <int DT, int OUT> constexpr int kLookupCols = DT == QM_F32 || OUT == QM_F32 ? 4 : 8;

template <int DT, int OUT> __global__ __launch_bounds__(kLookupThreads) void embedding_lookup_kernel(LookupArgs a) {
    constexpr int V = kLookupCols<DT, OUT>;
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
        col[k] = (int)(at % (uint32_t)a.pieces) * V;
        tok[k] = row[k] < a.n_tokens ? token_at(a.tokens, a.token_bits, row[k]) : -1;
    }
    float x[kLookupEach][V], scale[kLookupEach];
#pragma unroll
    for (int k = 0; k < kLookupEach; k++) {
        const bool inside = (uint64_t)tok[k] < (uint64_t)a.vocab;
        scale[k] = inside ? a.scale : 0.0f;      // zeros whatever the scale
        const int n = inside ? min(V, a.cols - col[k]) : 0;
        load_cols<DT, V>(a.table + (uint64_t)(tok[k] * a.ld_table + col[k]) * kSizeOf<DT>, n, x[k]);
    }
#pragma unroll
    for (int k = 0; k < kLookupEach; k++) {
        if (row[k] >= a.n_tokens) continue;
#pragma unroll
        for (int j = 0; j < V; j++) x[k][j] = in_fp32(x[k][j] * scale[k]);
        store_cols<OUT, V>(a.out + (uint64_t)(row[k] * a.ld_out + col[k]) * kSizeOf<OUT>, min(V, a.cols - col[k]), x[k]);
    }
}

// -------------------------------------------------------------------- sort

// Between LDS accesses by which lanes of a wave hand values to one another.  LDS
// serves a wave's accesses in the order of its instructions, so there is nothing
// to wait for; this holds the compiler to that order.
__device__ __forceinline__ void wave_lds_order() { asm volatile("" ::: "memory"); }

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

    // A lane's tokens, 16 in flight; the first 32 (all of them up to 32768
    // tokens) stay in registers for the second time.
    constexpr int kAhead = 16, kHeld = 32;
    uint32_t held[kHeld];
    auto load = [&](int c, uint32_t *t) {
#pragma unroll
        for (int k = 0; k < kAhead; k++) {
            const int i = c + k * 64 + lane;
            t[k] = i < end ? token32_at(a.tokens, a.token_bits, i) : 0xffffffffu;
        }
    };
    int less = 0;                // of the wave
    auto tally = [&](const uint32_t *t) {
#pragma unroll
        for (int k = 0; k < kAhead; k++) {
            less += __popcll(__ballot(t[k] < (uint32_t)lo));
            if (t[k] - lo < (uint32_t)values) atomicAdd(&mine[t[k] - lo], 1);
        }
    };
    constexpr int kBatch = 64 * kAhead;
#pragma unroll
    for (int h = 0; h < kHeld; h += kAhead) {
        if (begin + h * 64 >= end) break;
        load(begin + h * 64, held + h);
        tally(held + h);
    }
    for (int c = begin + kHeld * 64; c < end; c += kBatch) {
        uint32_t t[kAhead];
        load(c, t);
        tally(t);
    }
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

    auto place = [&](int c, const uint32_t *t) {
#pragma unroll
        for (int k = 0; k < kAhead; k++) {
            const bool in = t[k] - lo < (uint32_t)values;
            uint64_t same = __ballot(in);
            if (same == 0) continue;
            const int value = in ? (int)(t[k] - lo) : -1;
            if (__popcll(same) > a.value_bits) {
                for (int b = 0; b < a.value_bits; b++) {
                    const uint64_t set = __ballot(value >> b & 1);
                    same &= value >> b & 1 ? set : ~set;
                }
            } else {
                // few: one ballot for each value that is there
                for (uint64_t left = same; left;) {
                    const uint64_t these = __ballot(value == __builtin_amdgcn_readlane(value, __ffsll((unsigned long long)left) - 1));
                    same = these >> lane & 1 ? these : same;
                    left &= ~these;
                }
            }
            // all lanes of a value read its place, the first of them moves it on,
            // for the next 64 tokens' lanes to read
            if (in) {
                const int before = __popcll(same & ((1ull << lane) - 1)), next = mine[value];
                wave_lds_order();
                if (before == 0) mine[value] = next + __popcll(same);
                gmem<Sorted>(a.sorted)[next + before] = Sorted{(int32_t)t[k], c + k * 64 + lane};
            }
            wave_lds_order();
        }
    };
#pragma unroll
    for (int h = 0; h < kHeld; h += kAhead) {
        if (begin + h * 64 >= end) break;
        place(begin + h * 64, held + h);
    }
    for (int c = begin + kHeld * 64; c < end; c += kBatch) {
        uint32_t t[kAhead];
        load(c, t);
        place(c, t);
    }
}

// --------------------------------------------------------------------- sum

struct SumArgs {
    uint64_t sorted, start, head, part, dy, grad;
    int64_t ld_dy, ld_grad;
    int vocab, cols;
    int slabs, part_ld;                     // slabs: units across a row; part_ld: columns rounded up to 8
    int chunks, ranges, range, fills;       // units down: chunks, ranges of `range` positions, kFill rows each
    int accumulate, grad_dtype;
    float scale;
};

__device__ __forceinline__ int start_of(uint64_t start, int v) { return gmem<const int32_t>(start)[v]; }

// A lane's columns: P pieces of V.
template <int V, int P> struct Columns {
    int first, cols;        // the lane's first column; the row's columns
    __device__ __forceinline__ Columns(int slab, int lane, int n) : first(slab * (64 * V * P) + lane * V), cols(n) {}
    __device__ __forceinline__ int col(int p) const { return first + p * (64 * V); }
    // how many of piece p exist.  The empty asm has it looked at anew at each
    // use: kept, the outcomes for V elements of every piece fill the scalar
    // registers.
    __device__ __forceinline__ int n(int p) const {
        int r = max(0, min(V, cols - col(p)));
        asm volatile("" : "+v"(r));
        return r;
    }
};

template <int DT, int V, int P> struct Piece {
    PackedOf<DT, V> w[P];
    __device__ __forceinline__ void load(uint64_t row, const Columns<V, P> &c) {
#pragma unroll
        for (int p = 0; p < P; p++) {
            const uint64_t at = row + (uint64_t)c.col(p) * kSizeOf<DT>;
            const int n = c.n(p);
            w[p] = {};
            if (n == V) w[p] = load_bytes<V * kSizeOf<DT>>(at, 0);
            else {
#pragma unroll
                for (int j = 0; j < V; j++) {
                    if (j >= n) continue;
                    if constexpr (DT == QM_F32) w[p].w[j] = gmem<const uint32_t>(at)[j];
                    else w[p].w[j / 2] |= (unsigned)gmem<const uint16_t>(at)[j] << (16 * (j % 2));
                }
            }
        }
    }
};

// Sums dy rows along the order: entries `from` .. `to` - 1 of a window of 64
// whose positions lanes hold, several rows in flight whatever they belong to.
// ends(w): whether a row of the table ends with entry w; then old.load has its
// gradient under way with the entry's own loads and leave(w, acc, old) takes the
// sum.
template <int DT, int V, int P, typename Old, typename Ends, typename Fetch, typename Leave>
__device__ __forceinline__ void stream(const SumArgs &a, int pos, int from, int to, const Columns<V, P> &c, Ends ends,
                                       Fetch fetch, Leave leave) {
    constexpr int kAhead = P * V >= 16 ? 4 : 8;
    float acc[P][V] = {};
    for (int w = from; w < to; w += kAhead) {
        Piece<DT, V, P> x[kAhead];
        Old old[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; u++) {
            if (w + u >= to) continue;
            const int at = __builtin_amdgcn_readlane(pos, w + u);
            x[u].load(a.dy + (uint64_t)(at * a.ld_dy) * kSizeOf<DT>, c);
            if (ends(w + u)) fetch(w + u, old[u]);
        }
#pragma unroll
        for (int u = 0; u < kAhead; u++) {
            if (w + u >= to) continue;
#pragma unroll
            for (int p = 0; p < P; p++)
#pragma unroll
                for (int j = 0; j < V; j++) acc[p][j] += unpack<DT>(x[u].w[p], j);
            if (ends(w + u)) {
                leave(w + u, acc, old[u]);
#pragma unroll
                for (int p = 0; p < P; p++)
#pragma unroll
                    for (int j = 0; j < V; j++) acc[p][j] = 0.0f;
            }
        }
    }
}

struct Nothing {};
template <int N> using zeros_t = unsigned __attribute__((ext_vector_type(N), aligned(1)));

template <int DT, int GT, int V, int P, bool ACC> __global__ __launch_bounds__(kSumWaves * 64) void embedding_sum_kernel(SumArgs a) {
    const int lane = threadIdx.x & 63;
    const int unit = __builtin_amdgcn_readfirstlane((int)(blockIdx.x * kSumWaves + (threadIdx.x >> 6)));
    const int slab = unit % a.slabs;
    int down = unit / a.slabs;
    const Columns<V, P> c(slab, lane, a.cols);
    const int n_sorted = start_of(a.start, a.vocab);
    auto sorted_at = [&](int i) { return gmem<const Sorted>(a.sorted)[i]; };

    if (down < a.chunks) {
        // the parts of long rows that end, pass through or start in this chunk
        const int first = down * kChunk, last = min(first + kChunk, n_sorted) - 1;
        int head = -1;
        if (first <= last) {
            const Sorted e = sorted_at(min(first + lane, last));
            const int t0 = __builtin_amdgcn_readlane(e.token, 0), t1 = __builtin_amdgcn_readlane(e.token, last - first);
            const int s0 = start_of(a.start, t0), e0 = start_of(a.start, t0 + 1), s1 = start_of(a.start, t1), e1 = start_of(a.start, t1 + 1);
            auto part = [&](int slot, int from, int to) {
                stream<DT, V, P, Nothing>(a, e.position, from, to, c, [&](int w) { return w == to - 1; }, [](int, Nothing &) {},
                                          [&](int, float (*acc)[V], Nothing &) {
#pragma unroll
                                              for (int p = 0; p < P; p++)
                                                  store_cols<QM_F32, V>(a.part + (((uint64_t)down * 2 + slot) * a.part_ld + c.col(p)) * 4,
                                                                        c.n(p), acc[p]);
                                          });
            };
            if (e0 - s0 > kChunk) {
                if (s0 == first) head = t0;
                part(0, 0, min(e0 - 1, last) - first + 1);
            }
            if (t1 != t0 && e1 - s1 > kChunk) {
                head = t1;
                part(1, s1 - first, last - first + 1);
            }
        }
        if (slab == 0 && lane == 0) gmem<int32_t>(a.head)[down] = head;
        return;
    }
    down -= a.chunks;
    if (down < a.ranges) {
        // the rows that start in this range of the order, but for long ones;
        // window entry w is position begin - 1 + w.  The last row starts at most
        // at entry kRange: one that the window does not see end is a long one.
        static_assert(kRange + kChunk < 64, "window");
        const int begin = down * a.range;
        if (begin >= n_sorted) return;
        auto entry = [&](int i) { return i < 0 || i >= n_sorted ? Sorted{i < 0 ? -2 : -3, 0} : sorted_at(i); };
        const Sorted e = entry(begin - 1 + lane);
        const int before = __shfl_up(e.token, 1);
        const uint64_t heads = __ballot(lane > 0 && e.token != before);
        const uint64_t here = heads & ((2ull << a.range) - 2);
        if (here == 0) return;
        const int from = __ffsll((unsigned long long)here) - 1, last = 63 - __clzll((long long)here);
        const uint64_t after = heads & ~((2ull << last) - 1);
        int to = after ? __ffsll((unsigned long long)after) - 1 : 64;
        if (to - last > kChunk) to = last;      // a long row: its parts are summed elsewhere
        auto ends = [&](int w) { return w + 1 == to || heads >> (w + 1) & 1; };
        auto row = [&](int w) {
            const int token = __builtin_amdgcn_readlane(e.token, w);
            return a.grad + (uint64_t)(token * a.ld_grad) * kSizeOf<GT>;
        };
        using Old = std::conditional_t<ACC, Piece<GT, V, P>, Nothing>;
        stream<DT, V, P, Old>(
            a, e.position, from, to, c, ends,
            [&](int w, Old &old) {
                if constexpr (ACC) old.load(row(w), c);
            },
            [&](int w, float (*acc)[V], Old &old) {
                const uint64_t to_row = row(w);
#pragma unroll
                for (int p = 0; p < P; p++) {
                    float y[V];
#pragma unroll
                    for (int j = 0; j < V; j++) {
                        y[j] = a.scale * acc[p][j];
                        if constexpr (ACC) y[j] += unpack<GT>(old.w[p], j);
                        y[j] = in_fp32(y[j]);
                    }
                    store_cols<GT, V>(to_row + (uint64_t)c.col(p) * kSizeOf<GT>, c.n(p), y);
                }
            });
        return;
    }
    down -= a.ranges;
    if (down < a.fills) {
        // rows without tokens, of a gradient that is written whole
        const int row0 = down * kFill;
        const int s = start_of(a.start, min(row0 + lane, a.vocab)), next = __shfl_down(s, 1);
        uint64_t empty = __ballot(lane < kFill && row0 + lane < a.vocab && s == next);
        const float zero[V] = {};
        while (empty) {
            const int row = row0 + __ffsll((unsigned long long)empty) - 1;
            empty &= empty - 1;
            const uint64_t to = a.grad + (uint64_t)(row * a.ld_grad) * kSizeOf<GT>;
#pragma unroll
            for (int p = 0; p < P; p++) {
                if (c.n(p) == V) *reinterpret_cast<zeros_t<V * kSizeOf<GT> / 4> *>(gmem<char>(to) + (int64_t)c.col(p) * kSizeOf<GT>) = 0;
                else store_cols<GT, V>(to + (uint64_t)c.col(p) * kSizeOf<GT>, c.n(p), zero);
            }
        }
    }
}

template <int GT, int V> __device__ __forceinline__ void finish_as(const SumArgs &a, int token, int col, int n, const float *acc) {
    if (n == 0) return;
    const uint64_t at = a.grad + (uint64_t)(token * a.ld_grad + col) * kSizeOf<GT>;
    float y[V] = {};
    if (a.accumulate) load_cols<GT, V>(at, n, y);
#pragma unroll
    for (int j = 0; j < V; j++) y[j] = in_fp32(y[j] + a.scale * acc[j]);
    store_cols<GT, V>(at, n, y);
}

// One workgroup per eight chunks and 256 columns: the long rows that start in
// those chunks, one after the other.
__global__ __launch_bounds__(kJoinWaves * 64) void embedding_join_kernel(SumArgs a) {
    constexpr int V = 4, kAhead = 8;
    __shared__ float sums[kJoinWaves][64 * V];
    const int slabs = (a.cols + 64 * V - 1) / (64 * V);
    const int chunk0 = blockIdx.x / slabs * kJoinChunks, slab = blockIdx.x % slabs;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int col = slab * 64 * V + lane * V, cols = max(0, min(V, a.cols - col));
    const int head = lane < min(kJoinChunks, a.chunks - chunk0) ? gmem<const int32_t>(a.head)[chunk0 + lane] : -1;
    for (uint64_t left = __ballot(head >= 0); left; left &= left - 1) {
        const int k = __ffsll((unsigned long long)left) - 1, chunk = chunk0 + k, token = __builtin_amdgcn_readlane(head, k);
        const int s = start_of(a.start, token), last = (start_of(a.start, token + 1) - 1) / kChunk;
        // wave w adds an eighth of the parts, contiguous, so that the order stays
        const int parts = last - chunk + 1, each = (parts + kJoinWaves - 1) / kJoinWaves;
        const int p0 = min(wave * each, parts), p1 = min(p0 + each, parts);
        float acc[V] = {};
        for (int p = p0; p < p1; p += kAhead) {
            float x[kAhead][V];
#pragma unroll
            for (int u = 0; u < kAhead; u++) {
                const int c = chunk + min(p + u, p1 - 1);
                const int slot = c == chunk && s % kChunk != 0 ? 1 : 0;
                load_cols<QM_F32, V>(a.part + (((uint64_t)c * 2 + slot) * a.part_ld + col) * 4, cols, x[u]);
            }
#pragma unroll
            for (int u = 0; u < kAhead; u++)
#pragma unroll
                for (int j = 0; j < V; j++) acc[j] += p + u < p1 ? x[u][j] : 0.0f;
        }
        __syncthreads();      // the row before has been read
#pragma unroll
        for (int j = 0; j < V; j++) sums[wave][lane * V + j] = acc[j];
        __syncthreads();
        if (wave != 0) continue;
        for (int w = 1; w < kJoinWaves; w++)
#pragma unroll
            for (int j = 0; j < V; j++) acc[j] += sums[w][lane * V + j];
        if (a.grad_dtype == QM_F32) finish_as<QM_F32, V>(a, token, col, cols, acc);
        else if (a.grad_dtype == QM_BF16) finish_as<QM_BF16, V>(a, token, col, cols, acc);
        else finish_as<QM_F16, V>(a, token, col, cols, acc);
    }
}

// -------------------------------------------------------------------- host

uint64_t addr(const void *p) { return (uint64_t)(uintptr_t)p; }

template <typename F> void with_dtype(int32_t dtype, F f) {
    if (dtype == QM_F32) f(std::integral_constant<int, QM_F32>());
    else if (dtype == QM_BF16) f(std::integral_constant<int, QM_BF16>());
    else f(std::integral_constant<int, QM_F16>());
}

template <int DT, int GT, int V, int P> void launch_sum(const SumArgs &a, unsigned grid, hipStream_t q) {
    if (a.accumulate) embedding_sum_kernel<DT, GT, V, P, true><<<grid, kSumWaves * 64, 0, q>>>(a);
    else embedding_sum_kernel<DT, GT, V, P, false><<<grid, kSumWaves * 64, 0, q>>>(a);
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
    const int per = table_dtype == QM_F32 || out_dtype == QM_F32 ? 4 : 8;
    const int64_t pieces = (cols + per - 1) / per, each = kLookupThreads * kLookupEach, wgs = (n_tokens * pieces + each - 1) / each;
    if (wgs >= (int64_t)1 << 24) return fail(QM_E_UNSUPPORTED, "more than 2^34 pieces of 4 or 8 columns");
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
    // a unit's columns: 1024, or 256 or 512 where a row is no longer
    const int v = dy_dtype == QM_F32 || grad_dtype == QM_F32 ? 4 : 8, pieces = cols <= 64 * v ? 1 : 1024 / (64 * v);
    const int span = 64 * v * pieces;
    SumArgs a{};
    a.sorted = sort.sorted, a.start = sort.start, a.head = w + sp.head, a.part = w + sp.part;
    a.dy = addr(dy), a.grad = addr(grad), a.ld_dy = ld_dy, a.ld_grad = ld_grad;
    a.vocab = (int)vocab, a.cols = (int)cols;
    a.slabs = (int)((cols + span - 1) / span), a.part_ld = (int)sp.part_ld;
    // positions of a range: fewer as long as there are less than 4096 units
    a.range = kRange;
    while (a.range > 1 && n_tokens * a.slabs / a.range < 4096) a.range /= 2;
    a.chunks = (int)sp.chunks, a.ranges = (int)((n_tokens + a.range - 1) / a.range);
    a.fills = accumulate ? 0 : (int)((vocab + kFill - 1) / kFill);
    a.accumulate = accumulate, a.grad_dtype = grad_dtype, a.scale = scale;
    const int64_t units = ((int64_t)a.chunks + a.ranges + a.fills) * a.slabs, join_wgs = (sp.chunks + kJoinChunks - 1) / kJoinChunks * ((cols + 255) / 256);
    if (units >= (int64_t)1 << 25 || join_wgs >= (int64_t)1 << 22) return fail(QM_E_UNSUPPORTED, "more than 2^31 threads");
    const unsigned sum_wgs = (unsigned)((units + kSumWaves - 1) / kSumWaves);
    const hipStream_t q = static_cast<hipStream_t>(stream);
    embedding_sort_kernel<<<(unsigned)((vocab + values - 1) / values), kSortWaves * 64, 0, q>>>(sort);
    if (qm_status e = launch_status("embedding_grad")) return e;
    with_dtype(dy_dtype, [&](auto dt) {
        with_dtype(grad_dtype, [&](auto gt) {
            constexpr int DT = decltype(dt)::value, GT = decltype(gt)::value, V = DT == QM_F32 || GT == QM_F32 ? 4 : 8;
            if (pieces == 1) launch_sum<DT, GT, V, 1>(a, sum_wgs, q);
            else launch_sum<DT, GT, V, 1024 / (64 * V)>(a, sum_wgs, q);
        });
    });
    if (qm_status e = launch_status("embedding_grad")) return e;
    if (join_wgs == 0) return QM_OK;
    embedding_join_kernel<<<(unsigned)join_wgs, kJoinWaves * 64, 0, q>>>(a);
    return launch_status("embedding_grad");
}
