// Activations kept in 8 bits between the forward and the backward pass, and
// the gated activation that writes and reads them.
//
//   e      = the smallest integer with max|x| <= 448 * 2^e over 32 rows of a
//            column, between -95 and 119
//   data   = E4M3(x * 2^-e), rounded to nearest even;  scale = e + 127
//   value  = data * 2^e: exact in fp32 and in bf16
//
//   h  = act(g) u;    dg = dh u act'(g),  du = dh act(g)
//   silu: act = g s, act' = s (1 + g (1 - s)), s = 1 / (1 + exp(-g))
//   gelu (tanh form): act = g s, act' = s + g s (1 - s) z', s = 1 / (1 + exp(-z)),
//         z = 2 sqrt(2 / pi) (g + 0.044715 g^3)      (1 + tanh(z / 2) = 2 s)
//
// Every kernel passes once over its elements.  The forward of the gated
// activation codes g and u from the registers that h is formed from; the
// backward reads 2 bytes of g and u an element instead of 4.
//
// HBM bounds all of them (8192 x 14336 bf16, a large copy reaches 6.5 TB/s): pack
// 56.5 us, 6.3 TB/s; read 57.8 us, 6.2; forward 158 us, 6.0 (gelu 160); backward
// 160 us, 6.0 (163), with h 204 us, 5.8 (207).  A layer's 8192 x 4096 runs at 5.4
// to 5.6 TB/s, with a start and an end of a few us each; rows at odd addresses
// (3001 x 6145 f16) at 4.2, each access of a wave then touching one more line than
// it covers; fp32 (4096 x 4096) forward 46 us, 5.9 TB/s, backward with h 63, 4.8.
#include <algorithm>
#include <type_traits>

#include "act8_device.h"
#include "act_host.h"
#include "cu_share.h"
#include "reserve_lds.h"

namespace qm {
namespace {

constexpr int kWaves = kPatchWaves;

template <bool WIDE> __device__ __forceinline__ int patch_of() {
    return WIDE ? (int)blockIdx.x : __builtin_amdgcn_readfirstlane((int)(blockIdx.x * kWaves + threadIdx.x / 64));
}

// ------------------------------------------------------------ pack and read

struct PackArgs {
    uint64_t x, data, scale;
    int64_t rows, cols, ld, ld8;
    int patches, across;
};

// LINES: the rows that are written start on cache lines.
template <int DT, bool LINES, bool WIDE> __global__ __launch_bounds__(kWaves * 64) void act_pack_kernel(PackArgs a) {
    const int patch = patch_of<WIDE>();
    if (patch >= a.patches) return;
    const Patch<DT, WIDE> p(a.rows, a.cols, patch, a.across);
    PackedOf<DT, 8> r[kLaneRows];
#pragma unroll
    for (int i = 0; i < kLaneRows; i++) r[i] = patch_load(a.x, a.ld, p, i);
    uint32_t top[1][8];
    lane_tops<DT>(r, top[0]);
    group_tops<Patch<DT, WIDE>>(top);
    unpack_anew(r);
    encode<LINES>(p, r, top[0], a.data, a.scale, a.ld8);
}

template <int DT, bool LINES, bool WIDE> __global__ __launch_bounds__(kWaves * 64) void act_read_kernel(PackArgs a) {
    const int patch = patch_of<WIDE>();
    if (patch >= a.patches) return;
    const Patch<DT, WIDE> p(a.rows, a.cols, patch, a.across);
    Packed<8> w[kLaneRows];
#pragma unroll
    for (int i = 0; i < kLaneRows; i++) w[i] = load_codes(p, a.data, a.ld8, i);
    float unit[8];
    load_scales(p, a.scale, a.ld8, unit);
#pragma unroll
    for (int i = 0; i < kLaneRows; i++) {
        float x[8];
        decode(w[i], unit, x);
        patch_store<LINES>(a.x, a.ld, p, i, x);
    }
}

// --------------------------------------------------------- gated activation

enum { kSilu = QM_ACT_SILU, kGelu = QM_ACT_GELU };

// 1 / (1 + exp(-z)).  16-bit results: the hardware's exponential and
// reciprocal, each within an ulp of fp32.  The exponential's argument is rounded,
// which is worth |z| 2^-23 of its result and the larger part: at most 2^-16 before
// s is 0 (a bf16 half step is 2^-8, an f16 one 2^-11).
template <bool FAST> __device__ __forceinline__ float sigmoid(float z) {
    if constexpr (FAST) return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504f * z));
    else return 1.0f / (1.0f + expf(-z));
}

constexpr float kGeluA = 1.5957691216057308f;             // 2 sqrt(2 / pi)
constexpr float kGeluB = 3.0f * 0.044715f;

template <int ACT, bool FAST> __device__ __forceinline__ float act_value(float g) {
    if constexpr (ACT == kSilu) return g * sigmoid<FAST>(g);
    else return g * sigmoid<FAST>(kGeluA * (g + 0.044715f * g * g * g));
}
// The value and the slope.  s is 0 or 1 in fp32 long before |g| = 32; from
// there on the slope's second term is left at its limit 0, where g^2 would
// overflow for the largest g.  The limit is a compare and a select: minimum and
// maximum would turn a NaN into -32 and its slope into 0.
template <int ACT, bool FAST> __device__ __forceinline__ float act_slope(float g, float &value) {
    if constexpr (ACT == kSilu) {
        const float s = sigmoid<FAST>(g);
        value = g * s;
        return s * (1.0f + g * (1.0f - s));
    } else {
        const float b = fabsf(g) > 32.0f ? copysignf(32.0f, g) : g;
        const float s = sigmoid<FAST>(kGeluA * (b + 0.044715f * b * b * b));
        value = g * s;
        return s + b * (s * (1.0f - s)) * (kGeluA * (1.0f + kGeluB * b * b));
    }
}

struct GatedArgs {
    uint64_t gate, up, h;                      // forward in: g, u; backward out: dg, du
    uint64_t dh;
    uint64_t gate_data, gate_scale, up_data, up_scale;
    int64_t rows, cols, ld_gate, ld_up, ld_h, ld_dh, ld_gate8, ld_up8;
    int patches, across;
};

template <int DT, int ACT, bool LINES, bool WIDE> __global__ __launch_bounds__(kWaves * 64) void gated_forward_kernel(GatedArgs a) {
    const int patch = patch_of<WIDE>();
    if (patch >= a.patches) return;
    const Patch<DT, WIDE> p(a.rows, a.cols, patch, a.across);
    PackedOf<DT, 8> g[kLaneRows], u[kLaneRows];
#pragma unroll
    for (int i = 0; i < kLaneRows; i++) {
        g[i] = patch_load(a.gate, a.ld_gate, p, i);
        u[i] = patch_load(a.up, a.ld_up, p, i);
    }
#pragma unroll
    for (int i = 0; i < kLaneRows; i++) {
        float h[8];
#pragma unroll
        for (int j = 0; j < 8; j++) h[j] = in_fp32(act_value<ACT, DT != QM_F32>(unpack<DT>(g[i], j)) * unpack<DT>(u[i], j));
        patch_store<LINES>(a.h, a.ld_h, p, i, h);
    }
    if (a.gate_data) {
        unpack_anew(g);
        unpack_anew(u);
        uint32_t top[2][8];
        lane_tops<DT>(g, top[0]);
        lane_tops<DT>(u, top[1]);
        group_tops<Patch<DT, WIDE>>(top);
        unpack_anew(g);
        unpack_anew(u);
        encode<LINES>(p, g, top[0], a.gate_data, a.gate_scale, a.ld_gate8);
        encode<LINES>(p, u, top[1], a.up_data, a.up_scale, a.ld_up8);
    }
}

template <int DT, int ACT, bool LINES, bool WIDE> __global__ __launch_bounds__(kWaves * 64) void gated_backward_kernel(GatedArgs a) {
    const int patch = patch_of<WIDE>();
    if (patch >= a.patches) return;
    const Patch<DT, WIDE> p(a.rows, a.cols, patch, a.across);
    Packed<8> g8[kLaneRows], u8[kLaneRows];
    PackedOf<DT, 8> d[kLaneRows];
    float gs[8], us[8];
#pragma unroll
    for (int i = 0; i < kLaneRows; i++) {
        g8[i] = load_codes(p, a.gate_data, a.ld_gate8, i);
        u8[i] = load_codes(p, a.up_data, a.ld_up8, i);
        d[i] = patch_load(a.dh, a.ld_dh, p, i);
    }
    load_scales(p, a.gate_scale, a.ld_gate8, gs);
    load_scales(p, a.up_scale, a.ld_up8, us);
#pragma unroll
    for (int i = 0; i < kLaneRows; i++) {
        float g[8], u[8], dg[8], du[8], h[8];
        decode(g8[i], gs, g);
        decode(u8[i], us, u);
#pragma unroll
        for (int j = 0; j < 8; j++) {
            float v;
            const float slope = act_slope<ACT, DT != QM_F32>(g[j], v), dh = unpack<DT>(d[i], j);
            dg[j] = in_fp32(dh * u[j] * slope);
            du[j] = in_fp32(dh * v);
            h[j] = in_fp32(v * u[j]);
        }
        patch_store<LINES>(a.gate, a.ld_gate, p, i, dg);
        patch_store<LINES>(a.up, a.ld_up, p, i, du);
        if (a.h) patch_store<LINES>(a.h, a.ld_h, p, i, h);
    }
}

// ------------------------------------------------------------------- host

// Patches of a rows x cols matrix, one a wave or (wide) a workgroup; a launch
// has less than 2^32 threads.
bool is_wide(int64_t cols) { return cols >= 512; }
qm_status patch_grid(int64_t rows, int64_t cols, int &patches, int &across) {
    if ((cols + 127) / 128 * ((rows + kGroupRows - 1) / kGroupRows) > (int64_t)1 << 25)
        return fail(QM_E_UNSUPPORTED, "more than 2^25 patches of 32 x 128 elements");
    const int64_t span = is_wide(cols) ? Patch<QM_F32, true>::kCols : Patch<QM_F32, false>::kCols;
    across = (int)((cols + span - 1) / span);
    patches = (int)(across * ((rows + kGroupRows - 1) / kGroupRows));
    return QM_OK;
}
// Workgroups a CU, of those that fit, for the stream's sake, chosen on wide 16-bit
// matrices (us, 8192 x 14336 bf16): pack 56.6 with 4, 66.7 with 3, 56.8 with all
// (6); read 57.8 with 3, 60.6 with all (8); forward 158.1 with 2, 159.4 with 3, at
// 4096 columns 49.1 and 50.7; backward 203.1 with 2, 211.2 with 4.  Other types and
// shapes take the same: gelu on 8192 x 4096 f16 forward 51.6 with 2, 49.8 with 4,
// 3001 x 6145 f16 36.1 and 34.1, backward within 2 %; 4096 x 4096 fp32 within 2 %
// whatever the number.  What the wide kernels use themselves is taken off; the
// narrow ones, which use none, hold as much (pack 5 a CU, forward 2): 65536 x 256
// bf16 forward 30.0, with 4 26.8, backward 33.6 and 30.8, fp32 56.6 and 60.4;
// 65536 x 500 f16 forward 117, with 8 85.
constexpr unsigned kPackShare = wgs_per_cu(4) - (8u << 10), kReadShare = wgs_per_cu(3);
constexpr unsigned kForwardShare = wgs_per_cu(2) - (16u << 10), kBackwardShare = wgs_per_cu(2);

unsigned wgs(int patches, int64_t cols) { return (unsigned)(is_wide(cols) ? patches : (patches + kWaves - 1) / kWaves); }
uint64_t addr(const void *p) { return (uint64_t)(uintptr_t)p; }

// Whether every row starts on a cache line.
bool on_lines(const void *p, int64_t pitch_bytes) { return aligned(p, 128) && pitch_bytes % 128 == 0; }

// Calls f with the type, `lines` and is_wide(cols) as constants.
template <typename F> void with_kind(int32_t dtype, bool lines, int64_t cols, F f) {
    auto as = [&](auto l, auto w) {
        if (dtype == QM_F32) f(std::integral_constant<int, QM_F32>(), l, w);
        else if (dtype == QM_BF16) f(std::integral_constant<int, QM_BF16>(), l, w);
        else f(std::integral_constant<int, QM_F16>(), l, w);
    };
    if (!is_wide(cols)) as(std::false_type(), std::false_type());
    else if (lines) as(std::true_type(), std::true_type());
    else as(std::false_type(), std::true_type());
}

}  // namespace
}  // namespace qm

using namespace qm;

extern "C" qm_status act_pack(const void *x, int32_t dtype, int64_t ld, const qm_act8 *kept, qm_stream_t stream) {
    clear_error();
    if (!kept) return fail(QM_E_ARG, "kept is null");
    const int64_t rows = kept->rows, cols = kept->cols;
    if (qm_status e = check_kept("kept", kept, rows, cols)) return e;
    if (qm_status e = check_matrix("x", x, dtype, rows, cols, ld)) return e;
    if (rows == 0 || cols == 0) return QM_OK;
    Spans s;
    s.matrix(x, dtype, rows, cols, ld, false);
    s.kept(kept, true);
    if (s.clash()) return fail(QM_E_ARG, "x and kept overlap");
    PackArgs a{addr(x), addr(kept->data), addr(kept->scale), rows, cols, ld, kept->ld, 0, 0};
    if (qm_status e = patch_grid(rows, cols, a.patches, a.across)) return e;
    with_kind(dtype, on_lines(kept->data, kept->ld), cols, [&](auto dt, auto lines, auto wide) {
        act_pack_kernel<decltype(dt)::value, decltype(lines)::value, decltype(wide)::value><<<wgs(a.patches, cols), kWaves * 64, kPackShare, static_cast<hipStream_t>(stream)>>>(a);
    });
    return launch_status("act_pack");
}

extern "C" qm_status act_read(const qm_act8 *kept, void *out, int32_t dtype, int64_t ld, qm_stream_t stream) {
    clear_error();
    if (!kept) return fail(QM_E_ARG, "kept is null");
    const int64_t rows = kept->rows, cols = kept->cols;
    if (qm_status e = check_kept("kept", kept, rows, cols)) return e;
    if (qm_status e = check_matrix("out", out, dtype, rows, cols, ld)) return e;
    if (rows == 0 || cols == 0) return QM_OK;
    Spans s;
    s.matrix(out, dtype, rows, cols, ld, true);
    s.kept(kept, false);
    if (s.clash()) return fail(QM_E_ARG, "out and kept overlap");
    PackArgs a{addr(out), addr(kept->data), addr(kept->scale), rows, cols, ld, kept->ld, 0, 0};
    if (qm_status e = patch_grid(rows, cols, a.patches, a.across)) return e;
    with_kind(dtype, on_lines(out, ld * elem_size(dtype)), cols, [&](auto dt, auto lines, auto wide) {
        act_read_kernel<decltype(dt)::value, decltype(lines)::value, decltype(wide)::value><<<wgs(a.patches, cols), kWaves * 64, kReadShare, static_cast<hipStream_t>(stream)>>>(a);
    });
    return launch_status("act_read");
}

extern "C" qm_status gated_act_forward(const void *gate, int64_t ld_gate, const void *up, int64_t ld_up, int32_t dtype,
                                       int64_t rows, int64_t cols, int32_t act, void *h, int64_t ld_h,
                                       const qm_act8 *gate8, const qm_act8 *up8, qm_stream_t stream) {
    clear_error();
    if (act != kSilu && act != kGelu) return fail(QM_E_ARG, "unknown activation %d", act);
    if (!gate8 != !up8) return fail(QM_E_ARG, "gate8 and up8: both or neither");
    if (qm_status e = check_matrix("gate", gate, dtype, rows, cols, ld_gate)) return e;
    if (qm_status e = check_matrix("up", up, dtype, rows, cols, ld_up)) return e;
    if (qm_status e = check_matrix("h", h, dtype, rows, cols, ld_h)) return e;
    if (gate8) {
        if (qm_status e = check_kept("gate8", gate8, rows, cols)) return e;
        if (qm_status e = check_kept("up8", up8, rows, cols)) return e;
    }
    if (rows == 0 || cols == 0) return QM_OK;
    Spans s;
    s.matrix(gate, dtype, rows, cols, ld_gate, false);
    s.matrix(up, dtype, rows, cols, ld_up, false);
    s.matrix(h, dtype, rows, cols, ld_h, true);
    s.kept(gate8, true);
    s.kept(up8, true);
    if (s.clash()) return fail(QM_E_ARG, "an output overlaps another buffer");
    GatedArgs a{};
    a.gate = addr(gate), a.up = addr(up), a.h = addr(h);
    a.rows = rows, a.cols = cols, a.ld_gate = ld_gate, a.ld_up = ld_up, a.ld_h = ld_h;
    if (gate8) {
        a.gate_data = addr(gate8->data), a.gate_scale = addr(gate8->scale), a.ld_gate8 = gate8->ld;
        a.up_data = addr(up8->data), a.up_scale = addr(up8->scale), a.ld_up8 = up8->ld;
    }
    if (qm_status e = patch_grid(rows, cols, a.patches, a.across)) return e;
    const hipStream_t q = static_cast<hipStream_t>(stream);
    const bool on = on_lines(h, ld_h * elem_size(dtype)) && (!gate8 || (on_lines(gate8->data, gate8->ld) && on_lines(up8->data, up8->ld)));
    with_kind(dtype, on, cols, [&](auto dt, auto lines, auto wide) {
        constexpr int DT = decltype(dt)::value;
        constexpr bool LINES = decltype(lines)::value, WIDE = decltype(wide)::value;
        if (act == kSilu) gated_forward_kernel<DT, kSilu, LINES, WIDE><<<wgs(a.patches, cols), kWaves * 64, kForwardShare, q>>>(a);
        else gated_forward_kernel<DT, kGelu, LINES, WIDE><<<wgs(a.patches, cols), kWaves * 64, kForwardShare, q>>>(a);
    });
    return launch_status("gated_act_forward");
}

extern "C" qm_status gated_act_backward(const qm_act8 *gate8, const qm_act8 *up8, const void *dh, int64_t ld_dh,
                                        int32_t dtype, int32_t act, void *dgate, int64_t ld_dgate, void *dup,
                                        int64_t ld_dup, void *h, int64_t ld_h, qm_stream_t stream) {
    clear_error();
    if (act != kSilu && act != kGelu) return fail(QM_E_ARG, "unknown activation %d", act);
    if (!gate8) return fail(QM_E_ARG, "gate8 is null");
    const int64_t rows = gate8->rows, cols = gate8->cols;
    if (qm_status e = check_kept("gate8", gate8, rows, cols)) return e;
    if (qm_status e = check_kept("up8", up8, rows, cols)) return e;
    if (qm_status e = check_matrix("dh", dh, dtype, rows, cols, ld_dh)) return e;
    if (qm_status e = check_matrix("dgate", dgate, dtype, rows, cols, ld_dgate)) return e;
    if (qm_status e = check_matrix("dup", dup, dtype, rows, cols, ld_dup)) return e;
    if (h)
        if (qm_status e = check_matrix("h", h, dtype, rows, cols, ld_h)) return e;
    if (rows == 0 || cols == 0) return QM_OK;
    Spans s;
    s.kept(gate8, false);
    s.kept(up8, false);
    s.matrix(dh, dtype, rows, cols, ld_dh, false);
    s.matrix(dgate, dtype, rows, cols, ld_dgate, true);
    s.matrix(dup, dtype, rows, cols, ld_dup, true);
    s.matrix(h, dtype, rows, cols, ld_h, true);
    if (s.clash()) return fail(QM_E_ARG, "an output overlaps another buffer");
    GatedArgs a{};
    a.gate = addr(dgate), a.up = addr(dup), a.h = addr(h), a.dh = addr(dh);
    a.gate_data = addr(gate8->data), a.gate_scale = addr(gate8->scale), a.ld_gate8 = gate8->ld;
    a.up_data = addr(up8->data), a.up_scale = addr(up8->scale), a.ld_up8 = up8->ld;
    a.rows = rows, a.cols = cols, a.ld_gate = ld_dgate, a.ld_up = ld_dup, a.ld_h = ld_h, a.ld_dh = ld_dh;
    if (qm_status e = patch_grid(rows, cols, a.patches, a.across)) return e;
    const hipStream_t q = static_cast<hipStream_t>(stream);
    qm_status st = QM_OK;
    const int64_t size = elem_size(dtype);
    const bool on = on_lines(dgate, ld_dgate * size) && on_lines(dup, ld_dup * size) && (!h || on_lines(h, ld_h * size));
    with_kind(dtype, on, cols, [&](auto dt, auto lines, auto wide) {
        constexpr int DT = decltype(dt)::value;
        constexpr bool LINES = decltype(lines)::value, WIDE = decltype(wide)::value;
        auto kern = act == kSilu ? gated_backward_kernel<DT, kSilu, LINES, WIDE> : gated_backward_kernel<DT, kGelu, LINES, WIDE>;
        static std::atomic<bool> set[2][kMaxDevices] = {};
        st = reserve_lds(reinterpret_cast<const void *>(kern), kBackwardShare, set[act]);
        if (st == QM_OK) kern<<<wgs(a.patches, cols), kWaves * 64, kBackwardShare, q>>>(a);
    });
    return st != QM_OK ? st : launch_status("gated_act_backward");
}
