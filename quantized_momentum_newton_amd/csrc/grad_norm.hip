// Global gradient norm and clip factor over a list of gradients, and the
// scaling of the list in place, for gfx950 (wave64).
//
// norm = sqrt(sum g*g), summed in fp64: squares of fp32 gradients leave its
// range long before the norm does, and sums of 10^9 of them lose digits in
// fp32.  Two launches: every workgroup adds its tasks in order into one
// partial sum, one workgroup adds the partials in order, so the result does
// not depend on timing.  Bound by HBM: the norm reads the gradients once (1.3G
// in bf16: 0.40 ms, 6.6 TB/s), the scaling reads and writes them (0.81 ms, 6.5
// TB/s, the rate of a large copy).
#include <hip/hip_runtime.h>

#include <math.h>
#include <stdint.h>

#include "internal.h"
#include "list_device.h"
#include "list_host.h"
#include "list_layout.h"
#include "qmuon.h"

namespace qm {
namespace {

constexpr int kThreads = 256;
constexpr int kWavesPerWG = kThreads / 64;
constexpr int kMaxParts = 2048;      // workgroups of the first pass: 8 per CU, a read-only stream's best
constexpr int kFinishThreads = 1024; // two parts a thread: the pass over the parts is one load deep twice
// Lists of at most so many tasks take one launch of one workgroup: 2.1 to 4.5
// us for 1 to 64 tasks against 3.5 to 4.1 for the two launches, which cost
// their caller 7.3 us where one costs 4.6; at 128 tasks 7.4 against 4.1.
constexpr int kSmallTasks = 64;
// Workgroups of the scaling pass: 0.84 ms for 1.3G bf16 gradients with 128
// threads, 0.87 with 256 or 64, 0.96 with 1024 (as many waves as fit; 0.81
// with the limit at the launch).
constexpr int kScaleThreads = 128;

// Sum over the workgroup of WAVES waves, valid in thread 0.
template <int WAVES> __device__ __forceinline__ double wg_sum(double s) {
    __shared__ double lds[WAVES];
#pragma unroll
    for (int k = 1; k < 64; k <<= 1) s += xor_lanes(s, k);
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = s;
    __syncthreads();
    double t = 0.0;
    if (threadIdx.x == 0)
        for (int k = 0; k < WAVES; k++) t += lds[k];
    return t;
}

// Elements per lane in one 16-byte access, and such accesses in a task.
template <int DT> constexpr int kPer = 16 / kSizeOf<DT>;
template <int DT> constexpr int kParts = kListTask / (64 * kPer<DT>);

// Sum of squares of a lane's PARTS groups: one running sum per group, so that
// the fp64 additions do not wait for each other.
template <int DT, int PARTS> __device__ __forceinline__ double sum_groups(const Packed<16> *r) {
    double s[PARTS] = {};
#pragma unroll
    for (int j = 0; j < kPer<DT>; j++)
#pragma unroll
        for (int p = 0; p < PARTS; p++) {
            const double x = (double)unpack<DT>(r[p], j);
            s[p] += x * x;
        }
    double t = 0.0;
#pragma unroll
    for (int p = 0; p < PARTS; p++) t += s[p];
    return t;
}

template <int DT> __device__ __forceinline__ double task_sum_full(const ListTensor &T, int64_t e_task, int lane) {
    Packed<16> r[kParts<DT>];
    load_grad_task<DT, kPer<DT>, kParts<DT>>(T, e_task, lane, r);
    return sum_groups<DT, kParts<DT>>(r);
}

template <int DT> __device__ __forceinline__ double task_sum(const ListTensor &T, int64_t e_task, int nvalid, int lane) {
    if (nvalid == kListTask) return task_sum_full<DT>(T, e_task, lane);
    const int n = max(0, min(4, nvalid - lane * 4));
    const PackedOf<DT, 4> r = load_grad<DT>(T, e_task + lane * 4, n);   // zeros past the end
    double s = 0.0;
#pragma unroll
    for (int j = 0; j < 4; j++) {
        const double x = (double)unpack<DT>(r, j);
        s += x * x;
    }
    return s;
}

// Sum over the tasks wave, wave + waves, ... of the list.
__device__ __forceinline__ double list_sum(const ListTensor *tensors, const int32_t *owner, int n_tasks, int wave, int waves, int lane) {
    double s = 0.0;
    for (int task = wave; task < n_tasks; task += waves) {
        const int32_t ti = __builtin_amdgcn_readfirstlane(gmem<const int32_t>(owner)[task]);
        const ListTensor T = gmem<const ListTensor>(tensors)[ti];
        int nvalid;
        const int64_t e_task = task_start(T, task - T.task_offset, nvalid);
        if (T.grad_dtype == QM_F32) s += task_sum<QM_F32>(T, e_task, nvalid, lane);
        else if (T.grad_dtype == QM_BF16) s += task_sum<QM_BF16>(T, e_task, nvalid, lane);
        else s += task_sum<QM_F16>(T, e_task, nvalid, lane);
    }
    return s;
}

__device__ __forceinline__ void finish(double s, double max_norm, double eps, float *norm_out, float *coef_out) {
    const double norm = sqrt(s), c = max_norm / (norm + eps);
    *norm_out = (float)norm;
    *coef_out = !(s < (double)INFINITY) ? NAN : c < 1.0 ? (float)c : 1.0f;
}

__global__ __launch_bounds__(kThreads) void grad_sumsq_kernel(const ListTensor *tensors, const int32_t *owner, int n_tasks,
                                                             double *parts) {
    const int wave = __builtin_amdgcn_readfirstlane((int)(blockIdx.x * kWavesPerWG + (threadIdx.x >> 6)));
    const double s = wg_sum<kWavesPerWG>(list_sum(tensors, owner, n_tasks, wave, (int)gridDim.x * kWavesPerWG, threadIdx.x & 63));
    if (threadIdx.x == 0) parts[blockIdx.x] = s;
}

__global__ __launch_bounds__(kFinishThreads) void grad_norm_finish_kernel(const double *parts, int n_parts, double max_norm, double eps,
                                                                         float *norm_out, float *coef_out) {
    double x[kMaxParts / kFinishThreads], s = 0.0;
#pragma unroll
    for (int k = 0; k < kMaxParts / kFinishThreads; k++) {
        const int i = k * kFinishThreads + (int)threadIdx.x;
        x[k] = i < n_parts ? parts[i] : 0.0;
    }
#pragma unroll
    for (int k = 0; k < kMaxParts / kFinishThreads; k++) s += x[k];
    s = wg_sum<kFinishThreads / 64>(s);
    if (threadIdx.x == 0) finish(s, max_norm, eps, norm_out, coef_out);
}

__global__ __launch_bounds__(kFinishThreads) void grad_norm_small_kernel(const ListTensor *tensors, const int32_t *owner, int n_tasks,
                                                                        double max_norm, double eps, float *norm_out, float *coef_out) {
    constexpr int waves = kFinishThreads / 64;
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const double s = wg_sum<waves>(list_sum(tensors, owner, n_tasks, wave, waves, threadIdx.x & 63));
    if (threadIdx.x == 0) finish(s, max_norm, eps, norm_out, coef_out);
}

template <int DT> __device__ __forceinline__ void task_scale(const ListTensor &T, int64_t e_task, int nvalid, int lane, float c) {
    if (nvalid == kListTask) {
        constexpr int N = kPer<DT>, P = kParts<DT>;
        PackedOf<DT, N> r[P];
        load_grad_task<DT, N, P>(T, e_task, lane, r);
#pragma unroll
        for (int p = 0; p < P; p++) {
            float x[N];
#pragma unroll
            for (int j = 0; j < N; j++) x[j] = in_fp32(unpack<DT>(r[p], j) * c);
            r[p] = pack<DT, N>(x);
        }
        store_grad_task<DT, N, P>(T, e_task, lane, r);
        return;
    }
    const int n = max(0, min(4, nvalid - lane * 4));
    const PackedOf<DT, 4> r = load_grad<DT>(T, e_task + lane * 4, n);
    float x[4];
#pragma unroll
    for (int j = 0; j < 4; j++) x[j] = in_fp32(unpack<DT>(r, j) * c);
    store_grad<DT>(T, e_task + lane * 4, n, x);
}

__global__ __launch_bounds__(kScaleThreads) void grad_scale_kernel(const ListTensor *tensors, const int32_t *owner, int n_tasks,
                                                             const float *coef) {
    const int lane = threadIdx.x & 63;
    const int task = __builtin_amdgcn_readfirstlane((int)(blockIdx.x * (kScaleThreads / 64) + (threadIdx.x >> 6)));
    if (task >= n_tasks) return;
    const float c = *gmem<const float>(coef);
    if (c != c) return;
    const int32_t ti = __builtin_amdgcn_readfirstlane(gmem<const int32_t>(owner)[task]);
    const ListTensor T = gmem<const ListTensor>(tensors)[ti];
    int nvalid;
    const int64_t e_task = task_start(T, task - T.task_offset, nvalid);
    if (T.grad_dtype == QM_F32) task_scale<QM_F32>(T, e_task, nvalid, lane, c);
    else if (T.grad_dtype == QM_BF16) task_scale<QM_BF16>(T, e_task, nvalid, lane, c);
    else task_scale<QM_F16>(T, e_task, nvalid, lane, c);
}

unsigned parts_of(const ListHeader *h) {
    const int64_t wgs = (h->n_tasks + kWavesPerWG - 1) / kWavesPerWG;
    return (unsigned)(wgs < kMaxParts ? wgs : kMaxParts);
}

}  // namespace
}  // namespace qm

using namespace qm;

extern "C" size_t grad_norm_workspace_bytes(const void *host_plan) {
    qm_status st;
    const ListHeader *h = list_header(host_plan, kListGrads, &st);
    return h ? (size_t)(parts_of(h) + 1) * sizeof(double) : 0;
}

extern "C" qm_status grad_norm(const void *host_plan, const void *dev_plan, double max_norm, double eps, float *norm_out,
                               float *coef_out, void *ws, size_t ws_bytes, qm_stream_t stream) {
    clear_error();
    const ListArgs list = list_args(host_plan, dev_plan, kListGrads);
    const ListHeader *h = list.h;
    if (!h) return list.st;
    if (!(max_norm > 0.0)) return fail(QM_E_ARG, "max_norm must be positive");
    if (!(eps >= 0.0 && eps < (double)INFINITY)) return fail(QM_E_ARG, "eps must be finite and not negative");
    if (!norm_out || !coef_out) return fail(QM_E_ARG, "norm_out and coef_out must not be null");
    if (!aligned(norm_out, 4) || !aligned(coef_out, 4)) return fail(QM_E_ALIGN, "norm_out and coef_out need 4-byte alignment");
    const unsigned parts = parts_of(h);
    if (!ws || ws_bytes < (parts + 1) * sizeof(double))
        return fail(QM_E_WORKSPACE, "workspace: need %zu bytes", (size_t)(parts + 1) * sizeof(double));
    if (!aligned(ws, 8)) return fail(QM_E_ALIGN, "workspace needs 8-byte alignment");
    if (norm_out == coef_out) return fail(QM_E_ARG, "norm_out and coef_out must not share memory");
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (h->n_tasks <= kSmallTasks) {
        grad_norm_small_kernel<<<1, kFinishThreads, 0, s>>>(list.tensors, list.owner, (int)h->n_tasks, max_norm, eps, norm_out, coef_out);
        return launched("gradient norm");
    }
    double *part = static_cast<double *>(ws);
    grad_sumsq_kernel<<<parts, kThreads, 0, s>>>(list.tensors, list.owner, (int)h->n_tasks, part);
    if (qm_status e = launched("gradient norm")) return e;
    grad_norm_finish_kernel<<<1, kFinishThreads, 0, s>>>(part, (int)parts, max_norm, eps, norm_out, coef_out);
    return launched("gradient norm");
}

extern "C" qm_status grad_scale(const void *host_plan, const void *dev_plan, const float *coef, qm_stream_t stream) {
    clear_error();
    const ListArgs list = list_args(host_plan, dev_plan, kListGrads);
    const ListHeader *h = list.h;
    if (!h) return list.st;
    if (!coef) return fail(QM_E_ARG, "coef must not be null");
    if (!aligned(coef, 4)) return fail(QM_E_ALIGN, "coef needs 4-byte alignment");
    if (h->n_tasks == 0) return QM_OK;
    constexpr int waves = kScaleThreads / 64;
    // Workgroups a CU: as many as fit (16), 11, 4.  fp32: 17M elements 23.0, 22.5,
    // 22.5 us, 108M 149, 143, 137; nine tenths of the tasks fp32: 22.2, 22.1, 22.0
    // and 141, 136, 132; three quarters: 20.3, 20.1, 20.7 and 130, 124, 124; bf16:
    // 12.2, 12.2, 15.3 and 69, 68, 87.
    const unsigned lds = 10 * h->n_wide_grad >= 9 * h->n_tasks ? wgs_per_cu(4) : wgs_per_cu(11);
    grad_scale_kernel<<<(unsigned)((h->n_tasks + waves - 1) / waves), kScaleThreads, lds, static_cast<hipStream_t>(stream)>>>(
        list.tensors, list.owner, (int)h->n_tasks, coef);
    return launched("gradient scale");
}
