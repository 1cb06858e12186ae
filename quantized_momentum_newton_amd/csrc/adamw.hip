// AdamW over many tensors for gfx950 (wave64), with 32-bit states or with
// 8-bit states in blocks of 256.  Compiled with -ffp-contract=off: the coding
// of 8-bit states is defined by binary32 operations with one rounding each,
// so the codes match a CPU run of the same operations bit for bit.
//
// "Decoupled Weight Decay Regularization" (Loshchilov and Hutter, ICLR 2019)
// gives the step.  Both kernels are bound by HBM: every byte of gradient,
// weight and state is touched once.  One wave64 owns a task of 1024
// consecutive elements of one tensor; a lane takes 4 consecutive elements in
// each of the task's four 256-element blocks, so that a wave's access covers
// one contiguous span, and a block of the 8-bit states is one element group
// of the whole wave.
#include <hip/hip_runtime.h>

#include <math.h>
#include <stdint.h>

#include "internal.h"
#include "list_device.h"
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
    int32_t stochastic;
};

// New weight from the new moments.  The root and the quotient are the
// hardware's to within an ulp or two: the update is a small part of w.
__device__ __forceinline__ float new_weight(float w, float m, float v, float step, float decay, const AdamArgs &A) {
    const float denom = sqrtf(v) * A.root + A.eps;
    return (w - w * decay) - step * (m / denom);
}

template <int DT> __device__ __forceinline__ void store_weight(const ListTensor &T, int64_t e, int n, const float *w) {
    store_upto4<DT>(T.weight, e, n, w);
    if (T.copy == 0) return;
    if (T.copy_dtype == QM_BF16) store_upto4<QM_BF16>(T.copy, e, n, w);
    else store_upto4<QM_F16>(T.copy, e, n, w);
}

template <int DT> __device__ __forceinline__ Raw4<DT> load_n(uint64_t base, int64_t e, int n) {
    return n == 4 ? load4<DT>(base, e) : load_upto4<DT>(base, e, n);
}

// ------------------------------------------------------------ 32-bit states

template <int GDT, int WDT>
__device__ __forceinline__ void task32(const ListTensor &T, int64_t e_task, int nvalid, int lane, float c, const AdamArgs &A) {
    const float step = A.step * T.lr_scale, decay = A.lr * T.lr_scale * T.weight_decay;
    for (int p = 0; p < kListTask / 256; p++) {
        const int e0 = p * 256 + lane * 4;
        const int n = min(4, nvalid - e0);
        if (n <= 0) continue;
        const int64_t e = e_task + e0;
        const Raw4<GDT> rg = load_grad<GDT>(T, e, n);
        const Raw4<WDT> rw = load_n<WDT>(T.weight, e, n);
        const Raw4<QM_F32> rm = load_n<QM_F32>(T.m, e, n), rv = load_n<QM_F32>(T.v, e, n);
        float m[4], v[4], w[4];
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const float g = elem<GDT>(rg, j) * c;
            m[j] = A.b1 * elem<QM_F32>(rm, j) + A.omb1 * g;
            v[j] = A.b2 * elem<QM_F32>(rv, j) + A.omb2 * (g * g);
            w[j] = new_weight(elem<WDT>(rw, j), m[j], v[j], step, decay, A);
        }
        store_upto4<QM_F32>(T.m, e, n, m);
        store_upto4<QM_F32>(T.v, e, n, v);
        store_weight<WDT>(T, e, n, w);
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

// Largest of the bit patterns over the wave.  Patterns of values without
// their sign order as the values do, with infinity above every number and
// NaN above that.
__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
#pragma unroll
    for (int k = 1; k < 64; k <<= 1) x = max(x, (uint32_t)xor_lanes((int)x, k));
    return x;
}

// m's code: x = m (127 / absmax) rounded, |x| <= 127 (1 + 2^-23).
__device__ __forceinline__ int m_code(float x, uint32_t word, int stochastic) {
    if (!stochastic) return (int)rintf(x);
    const float k = floorf(x);
    const float up = (float)(word >> 16) * 0x1p-16f < x - k ? 1.0f : 0.0f;
    return (int)fminf(fmaxf(k + up, -127.0f), 127.0f);
}

// v's code: y = v (65025 / max) in [0, 65025 (1 + 2^-23)].  k = floor(sqrt y)
// exactly (k and k^2 are whole numbers below 2^17, y - k^2 is exact); the
// code is k + 1 where y - k^2 is past u (2k + 1), u = 1/2 for nearest.  u
// has 15 bits and 2k + 1 at most 9, so their product is exact.
__device__ __forceinline__ int v_code(float y, float v, uint32_t word, int stochastic) {
    float k = floorf(sqrtf(y));
    float d = y - k * k;
    if (d < 0.0f) {   // the root rounded up to a whole number
        k -= 1.0f;
        d = y - k * k;
    }
    const float u = stochastic ? (float)(word & 0x7fffu) * 0x1p-15f : 0.5f;
    const int code = (int)k + (d > u * (2.0f * k + 1.0f) ? 1 : 0);
    return v > 0.0f ? max(1, min(code, 255)) : 0;
}

template <int GDT, int WDT>
__device__ __forceinline__ void task8(const ListTensor &T, int32_t tensor, int64_t e_task, int nvalid, int lane, float c,
                                      const AdamArgs &A) {
    const float step = A.step * T.lr_scale, decay = A.lr * T.lr_scale * T.weight_decay;
    for (int p = 0; p < kListTask / 256; p++) {
        if (p * 256 >= nvalid) break;
        const int e0 = p * 256 + lane * 4;
        const int n = max(0, min(4, nvalid - e0));
        const int64_t e = e_task + e0, block = (e_task >> 8) + p;
        Raw4<GDT> rg = {};
        Raw4<WDT> rw = {};
        uint32_t qm = 0, qv = 0;
        if (n > 0) {
            rg = load_grad<GDT>(T, e, n);
            rw = load_n<WDT>(T.weight, e, n);
            qm = load_codes(T.m, e, n);
            qv = load_codes(T.v, e, n);
        }
        float *pm = gmem<float>(T.m_absmax) + block, *pv = gmem<float>(T.v_absmax) + block;
        const float step_m = (*pm / 127.0f) * A.b1, step_v = (*pv / 65025.0f) * A.b2;
        float m[4], v[4], w[4];
        uint32_t top_m = 0, top_v = 0;
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const float g = elem<GDT>(rg, j) * c;
            const float cv = (float)((qv >> (8 * j)) & 0xffu);
            m[j] = (float)(int8_t)(qm >> (8 * j)) * step_m + A.omb1 * g;
            v[j] = (cv * cv) * step_v + A.omb2 * (g * g);
            w[j] = new_weight(elem<WDT>(rw, j), m[j], v[j], step, decay, A);
            if (j < n) {
                top_m = max(top_m, __float_as_uint(m[j]) & 0x7fffffffu);
                top_v = max(top_v, __float_as_uint(v[j]) & 0x7fffffffu);
            }
        }
        store_weight<WDT>(T, e, n, w);
        float am = __uint_as_float(wave_max(top_m)), av = __uint_as_float(wave_max(top_v));
        if (am < kTiny) am = 0.0f;
        if (av < kTiny) av = 0.0f;
        const float im = am > 0.0f ? 127.0f / am : 0.0f, iv = av > 0.0f ? 65025.0f / av : 0.0f;
        uint32_t word[4] = {};
        if (A.stochastic) {
            const uint64_t quad = (uint64_t)e >> 2;
            philox4x32_10((uint32_t)quad, (uint32_t)(quad >> 32), A.offset, (uint32_t)tensor, (uint32_t)A.seed,
                          (uint32_t)(A.seed >> 32), word);
        }
        uint32_t nm = 0, nv = 0;
        if (am < INFINITY)
#pragma unroll
            for (int j = 0; j < 4; j++) nm |= (uint32_t)(m_code(m[j] * im, word[j], A.stochastic) & 0xff) << (8 * j);
        if (av < INFINITY && av > 0.0f)
#pragma unroll
            for (int j = 0; j < 4; j++) nv |= (uint32_t)v_code(v[j] * iv, v[j], word[j], A.stochastic) << (8 * j);
        store_codes(T.m, e, n, nm);
        store_codes(T.v, e, n, nv);
        if (lane == 0) {
            *pm = am;
            *pv = av;
        }
    }
}

// ------------------------------------------------------------ kernels

template <int BITS, int GDT, int WDT>
__device__ __forceinline__ void run_task(const ListTensor &T, int32_t tensor, int64_t lt, int lane, float c, const AdamArgs &A) {
    const int64_t e_task = lt * kListTask, rem = T.numel - e_task;
    const int nvalid = rem < kListTask ? (int)rem : kListTask;
    if constexpr (BITS == 32) task32<GDT, WDT>(T, e_task, nvalid, lane, c, A);
    else task8<GDT, WDT>(T, tensor, e_task, nvalid, lane, c, A);
}

template <int BITS> __global__ __launch_bounds__(kThreads) void adamw_kernel(AdamArgs A) {
    const int lane = threadIdx.x & 63;
    const int task = A.task_lo + __builtin_amdgcn_readfirstlane((int)(blockIdx.x * kWavesPerWG + (threadIdx.x >> 6)));
    if (task >= A.task_hi) return;
    float c = 1.0f;
    if (A.grad_scale) {
        c = *gmem<const float>(A.grad_scale);
        if (c != c) return;   // the gradient's norm is not finite: leave everything as it is
    }
    const int32_t ti = __builtin_amdgcn_readfirstlane(gmem<const int32_t>(A.owner)[task]);
    const ListTensor &T = gmem<const ListTensor>(A.tensors)[ti];
    const int64_t lt = task - T.task_offset;
    switch (T.grad_dtype * 3 + T.weight_dtype) {
        case QM_F32 * 3 + QM_F32: run_task<BITS, QM_F32, QM_F32>(T, ti, lt, lane, c, A); break;
        case QM_F32 * 3 + QM_BF16: run_task<BITS, QM_F32, QM_BF16>(T, ti, lt, lane, c, A); break;
        case QM_F32 * 3 + QM_F16: run_task<BITS, QM_F32, QM_F16>(T, ti, lt, lane, c, A); break;
        case QM_BF16 * 3 + QM_F32: run_task<BITS, QM_BF16, QM_F32>(T, ti, lt, lane, c, A); break;
        case QM_BF16 * 3 + QM_BF16: run_task<BITS, QM_BF16, QM_BF16>(T, ti, lt, lane, c, A); break;
        case QM_BF16 * 3 + QM_F16: run_task<BITS, QM_BF16, QM_F16>(T, ti, lt, lane, c, A); break;
        case QM_F16 * 3 + QM_F32: run_task<BITS, QM_F16, QM_F32>(T, ti, lt, lane, c, A); break;
        case QM_F16 * 3 + QM_BF16: run_task<BITS, QM_F16, QM_BF16>(T, ti, lt, lane, c, A); break;
        default: run_task<BITS, QM_F16, QM_F16>(T, ti, lt, lane, c, A); break;
    }
}

// The values the states stand for, one task of the list per wave.
__global__ __launch_bounds__(kThreads) void adamw_read_kernel(const ListTensor *tensors, const int32_t *owner, int n_tasks,
                                                             float *m_out, float *v_out) {
    const int lane = threadIdx.x & 63;
    const int task = __builtin_amdgcn_readfirstlane((int)(blockIdx.x * kWavesPerWG + (threadIdx.x >> 6)));
    if (task >= n_tasks) return;
    const int32_t ti = __builtin_amdgcn_readfirstlane(gmem<const int32_t>(owner)[task]);
    const ListTensor &T = gmem<const ListTensor>(tensors)[ti];
    const int64_t e_task = (task - T.task_offset) * kListTask;
    const int64_t rem = T.numel - e_task;
    const int nvalid = rem < kListTask ? (int)rem : kListTask;
    const int64_t out = T.block_offset * kBlock + e_task;
    for (int p = 0; p < kListTask / 256; p++) {
        if (p * 256 >= nvalid) break;
        const int e0 = p * 256 + lane * 4;
        const int n = max(0, min(4, nvalid - e0));
        const int64_t e = e_task + e0;
        float m[4], v[4];
        if (T.state_bits == 32) {
            const Raw4<QM_F32> rm = n > 0 ? load_n<QM_F32>(T.m, e, n) : Raw4<QM_F32>{};
            const Raw4<QM_F32> rv = n > 0 ? load_n<QM_F32>(T.v, e, n) : Raw4<QM_F32>{};
#pragma unroll
            for (int j = 0; j < 4; j++) {
                m[j] = elem<QM_F32>(rm, j);
                v[j] = elem<QM_F32>(rv, j);
            }
        } else {
            const uint32_t qm = load_codes(T.m, e, n), qv = load_codes(T.v, e, n);
            const int64_t block = (e_task >> 8) + p;
            const float sm = gmem<const float>(T.m_absmax)[block] / 127.0f;
            const float sv = gmem<const float>(T.v_absmax)[block] / 65025.0f;
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const float cv = (float)((qv >> (8 * j)) & 0xffu);
                m[j] = j < n ? (float)(int8_t)(qm >> (8 * j)) * sm : 0.0f;
                v[j] = j < n ? (cv * cv) * sv : 0.0f;
            }
        }
        store4<QM_F32>((uint64_t)m_out, out + e0, m);
        store4<QM_F32>((uint64_t)v_out, out + e0, v);
    }
}

qm_status launched(const char *what) {
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? QM_OK : fail(QM_E_HIP, "%s launch: %s", what, hipGetErrorString(e));
}

unsigned grid_for(int64_t tasks) { return (unsigned)((tasks + kWavesPerWG - 1) / kWavesPerWG); }

const ListHeader *list_args(const void *host_plan, const void *dev_plan, qm_status *st) {
    const ListHeader *h = list_header(host_plan, kListAdamW, st);
    if (!h) return nullptr;
    if (!dev_plan) {
        *st = fail(QM_E_ARG, "device copy of the list is null");
        return nullptr;
    }
    if (!aligned(dev_plan, 64)) {
        *st = fail(QM_E_ALIGN, "device copy of the list must be 64-byte aligned");
        return nullptr;
    }
    return h;
}

}  // namespace
}  // namespace qm

using namespace qm;

extern "C" qm_status adamw_step(const void *host_plan, const void *dev_plan, const qm_adamw_hparams *hp,
                                const float *grad_scale, qm_stream_t stream) {
    clear_error();
    qm_status st;
    const ListHeader *h = list_args(host_plan, dev_plan, &st);
    if (!h) return st;
    if (!hp) return fail(QM_E_ARG, "hyperparameters are null");
    if (!isfinite(hp->lr)) return fail(QM_E_ARG, "lr must be finite");
    if (!(hp->beta1 >= 0.0 && hp->beta1 < 1.0) || !(hp->beta2 >= 0.0 && hp->beta2 < 1.0))
        return fail(QM_E_ARG, "beta1 and beta2 must lie in [0, 1)");
    if (!((float)hp->eps > 0.0f) || !isfinite((float)hp->eps)) return fail(QM_E_ARG, "eps must be positive and finite");
    if (hp->step < 1) return fail(QM_E_ARG, "step is 1-based");
    if (hp->rounding != QM_ROUND_NEAREST && hp->rounding != QM_ROUND_STOCHASTIC)
        return fail(QM_E_ARG, "unknown rounding mode %d", hp->rounding);
    if (!aligned(grad_scale, 4)) return fail(QM_E_ALIGN, "grad_scale needs 4-byte alignment");
    AdamArgs A = {};
    const char *dev = static_cast<const char *>(dev_plan);
    A.tensors = reinterpret_cast<const ListTensor *>(dev + h->off_tensors);
    A.owner = reinterpret_cast<const int32_t *>(dev + h->off_task_tensor);
    A.grad_scale = grad_scale;
    A.b1 = (float)hp->beta1;
    A.omb1 = (float)(1.0 - hp->beta1);
    A.b2 = (float)hp->beta2;
    A.omb2 = (float)(1.0 - hp->beta2);
    A.step = (float)(hp->lr / (1.0 - pow(hp->beta1, (double)hp->step)));
    A.lr = (float)hp->lr;
    A.root = (float)(1.0 / sqrt(1.0 - pow(hp->beta2, (double)hp->step)));
    A.eps = (float)hp->eps;
    A.seed = hp->seed;
    A.offset = hp->offset;
    A.stochastic = hp->rounding == QM_ROUND_STOCHASTIC;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (h->n_tasks32 > 0) {
        A.task_lo = 0;
        A.task_hi = (int32_t)h->n_tasks32;
        adamw_kernel<32><<<grid_for(A.task_hi - A.task_lo), kThreads, 0, s>>>(A);
        if (qm_status e = launched("AdamW")) return e;
    }
    if (h->n_tasks > h->n_tasks32) {
        A.task_lo = (int32_t)h->n_tasks32;
        A.task_hi = (int32_t)h->n_tasks;
        adamw_kernel<8><<<grid_for(A.task_hi - A.task_lo), kThreads, 0, s>>>(A);
        if (qm_status e = launched("AdamW with 8-bit states")) return e;
    }
    return QM_OK;
}

extern "C" qm_status adamw_read_state(const void *host_plan, const void *dev_plan, float *m_out, float *v_out,
                                      qm_stream_t stream) {
    clear_error();
    qm_status st;
    const ListHeader *h = list_args(host_plan, dev_plan, &st);
    if (!h) return st;
    if (h->n_tasks == 0) return QM_OK;
    if (!m_out || !v_out) return fail(QM_E_ARG, "m_out and v_out must not be null");
    if (!aligned(m_out, 16) || !aligned(v_out, 16)) return fail(QM_E_ALIGN, "m_out and v_out need 16-byte alignment");
    const char *dev = static_cast<const char *>(dev_plan);
    adamw_read_kernel<<<grid_for(h->n_tasks), kThreads, 0, static_cast<hipStream_t>(stream)>>>(
        reinterpret_cast<const ListTensor *>(dev + h->off_tensors),
        reinterpret_cast<const int32_t *>(dev + h->off_task_tensor), (int)h->n_tasks, m_out, v_out);
    return launched("AdamW state read");
}
