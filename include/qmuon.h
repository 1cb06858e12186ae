/*
 * qmuon.h -- C ABI of libqmuon.so: one Muon optimizer step on an AMD MI355X
 * (gfx950), as a blockwise-int8 momentum update followed by quintic
 * Newton-Schulz orthogonalisation; next to it the AdamW step of the
 * parameters Muon does not fit, the global gradient norm, and the operators
 * that make the gradients from activations kept in 8 bits.
 *
 * Conventions shared by every entry point
 *   - Pointers are device pointers unless a parameter says "host".
 *   - The caller owns every buffer (state, grads, weights, plan copies,
 *     workspace).  The library never allocates or frees device memory, never
 *     synchronises the stream and never prints.
 *   - Work is enqueued asynchronously on `stream` (a hipStream_t; NULL is the
 *     null stream).  A call returns after enqueueing.
 *   - All arguments are validated on the host before anything is enqueued;
 *     on any validation error nothing is launched and no buffer is written.
 *     A launch failure returns QM_E_HIP; buffers may then be partly updated.
 *   - qm_last_error() gives a per-thread description of the last failure.
 *   - Calls that share buffers or workspace on one stream run in order; the
 *     same workspace must not be used by two streams at once.
 *   - Entry points may be called from several host threads at once, each
 *     with its own buffers, workspace and stream; results do not depend on
 *     what else runs (every reduction has one fixed order).
 */
#ifndef QMUON_H
#define QMUON_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define QM_ABI_VERSION 4
#define QM_BLOCK 256           /* quantisation block: elements per absmax */

typedef void *qm_stream_t;     /* hipStream_t */

#ifndef QM_API
#define QM_API __attribute__((visibility("default")))
#endif

typedef enum {
    QM_OK = 0,
    QM_E_ARG = 1,          /* null pointer, bad count, bad hyperparameter   */
    QM_E_ALIGN = 2,        /* pointer or segment alignment violated          */
    QM_E_DTYPE = 3,        /* unknown or unsupported dtype                   */
    QM_E_SHAPE = 4,        /* shapes inconsistent or not divisible           */
    QM_E_WORKSPACE = 5,    /* workspace missing or too small                 */
    QM_E_HIP = 6,          /* a HIP launch or runtime call failed            */
    QM_E_UNSUPPORTED = 7,  /* valid request outside what is implemented      */
    QM_E_PLAN = 8          /* plan blob malformed or of another version      */
} qm_status;

typedef enum { QM_F32 = 0, QM_BF16 = 1, QM_F16 = 2 } qm_dtype;

/* Newton-Schulz arithmetic: bf16 operands with fp32 accumulation (X, A, B
 * all held in bf16); fp32 operands with fp32 accumulation on fp32 MFMAs; or
 * fp32 operands held in fp32, each product formed on bf16 MFMAs from a
 * hi + lo split of both factors (hi = bf16(x), lo = bf16(x - hi); terms
 * hi hi' + hi lo' + lo hi', fp32 accumulation; the dropped lo lo' is below
 * 2^-16 of each product), "bf16x3". */
typedef enum { QM_NS_BF16 = 0, QM_NS_F32 = 1, QM_NS_BF16X3 = 2 } qm_ns_precision;

/* ------------------------------------------------------------------------
 * q8 momentum state and norm plans
 *
 * State of one tensor ("Quantized Muon Momentum", section "What Exists"):
 * `codes` of the tensor's size and one fp32 absmax per 256-element block
 * (the last block of a tensor covers the remainder).  Codes lie in
 * [-127, 127]; element i dequantises to codes[i] * (absmax[i/256] / 127).
 * The page allows int8 or uint8 storage for the codes; a uint8 buffer holds
 * the same two's-complement bytes (no offset), so both are passed here as
 * `codes`.  Blocks follow the tensor's logical (row-major) element order.
 *
 * The codes and absmax are contiguous.  The grad may be contiguous
 * (grad_cols = 0) or a 2-D view of numel / grad_cols rows of grad_cols
 * elements with row pitch grad_ld elements, e.g. one slice of a fused
 * buffer; the page lists "contiguous only" among the limitations of its
 * kernel ("Known Limitations").
 * ---------------------------------------------------------------------- */
typedef struct {
    int8_t *codes;      /* [numel] int8 (or uint8 bytes), 16-byte aligned,
                           in/out                                            */
    float *absmax;      /* [ceil(numel/256)], 4-byte aligned, in/out         */
    void *grad;         /* grad_dtype, 16-byte aligned; in: g, out: m
                           (optionally normalised)                           */
    int64_t numel;      /* > 0                                               */
    int32_t grad_dtype; /* qm_dtype                                          */
    int32_t reserved;   /* must be 0                                         */
    int64_t grad_cols;  /* 0: grad contiguous; else row length, a multiple
                           of 8 dividing numel                               */
    int64_t grad_ld;    /* grad_cols > 0: row pitch in elements, a multiple
                           of 8, >= grad_cols; ignored otherwise             */
} qm_q8_tensor;

/* One slice of a tensor assigned to a norm group ("Quantized Muon Momentum",
 * section "Grouped QKV And Sharding": fused Q, K and V use one group each).
 * `start` and `length` are element offsets into the flattened tensor.  A
 * segment starts on a 256-element boundary and ends on one unless it ends at
 * the tensor's last element.  Every block of every tensor must belong to
 * exactly one segment. */
typedef struct {
    int32_t tensor_index;
    int32_t group_id;   /* 0 .. n_groups-1                                   */
    int64_t start;
    int64_t length;
} qm_norm_segment;

/* Build a plan blob (host only; touches no GPU).  The blob records the
 * tensors' device pointers, one group id per block and the blocks of every
 * group; it is built once and reused for every step.  The caller copies the
 * bytes verbatim into device memory once (8-byte aligned) and passes both
 * copies to the update calls.
 *   host_blob == NULL: only *inout_blob_bytes is set to the size needed.
 *   Otherwise *inout_blob_bytes must be >= that size; it is set to the size
 *   written.
 * Errors: QM_E_ARG (null/counts/group ids), QM_E_ALIGN (pointer alignment or
 * segment boundaries), QM_E_SHAPE (overlap or an uncovered block), QM_E_DTYPE. */
QM_API qm_status qm_plan_encode(const qm_q8_tensor *tensors, int32_t n_tensors,
                         const qm_norm_segment *segments, int32_t n_segments,
                         int32_t n_groups, void *host_blob,
                         size_t *inout_blob_bytes);

/* Plan facts read back from a host blob (any out pointer may be NULL). */
QM_API qm_status qm_plan_info(const void *host_blob, int32_t *n_tensors,
                       int32_t *n_groups, int64_t *n_blocks,
                       int64_t *total_numel);

/* Workspace bytes qmuon_update_normalize_groups needs for this plan. */
QM_API size_t qm_update_workspace_bytes(const void *host_blob);

/* Requantisation rounding.  Nearest: round half to even.  Stochastic (the
 * page lists it under "Known Limitations" as not yet implemented; this is
 * the reading taken): x = m * (127 / absmax') as for nearest; the code is
 * floor(x) + 1 if u < x - floor(x), else floor(x), clamped to [-127, 127],
 * both operations in binary32; u = (r >> 8) * 2^-24 where r is word (e mod 4)
 * of Philox4x32-10 ("Parallel random numbers: as easy as 1, 2, 3", Salmon,
 * Moraes, Dror and Shaw, SC 2011) with counter (e / 4 low word, e / 4 high
 * word, offset, the tensor's index in the plan) and key (seed low word, seed
 * high word), e the element's index in its tensor.  The codes remain
 * bit-identical to a CPU run of the same definition. */
typedef enum { QM_ROUND_NEAREST = 0, QM_ROUND_STOCHASTIC = 1 } qm_rounding;

typedef struct {
    int32_t rounding;   /* qm_rounding                                        */
    uint32_t offset;    /* counter word 2 (e.g. the step number)              */
    uint64_t seed;      /* Philox key                                         */
} qm_round_opts;

/* In-place multi-tensor q8 update in one launch ("Quantized Muon Momentum",
 * sections "What Exists" and "Algorithm"): for every block of every tensor,
 * dequantise the old momentum in fp32, m = beta*old + (1-beta)*g (two
 * separately rounded products, one rounded sum), write m to the grad buffer
 * (round to nearest even into its dtype), absmax' = max|m| over the block,
 * codes' = clamp(rint(m * (127/absmax')), -127, 127), or codes 0 and absmax 0
 * for an all-zero block.  Codes and absmax are bit-identical to a CPU run of
 * the same IEEE binary32 operations.
 *   block_sumsq: nullable; if given, [n_blocks] fp64 receives each block's
 *   sum of m*m (fp32 m, fp64 accumulation), indexed by global block (tensors
 *   in plan order).
 * Errors: QM_E_ARG, QM_E_PLAN, QM_E_HIP. */
QM_API qm_status qmuon_update_multi(const void *host_plan, const void *dev_plan,
                             float beta, double *block_sumsq,
                             qm_stream_t stream);

/* qmuon_update_multi with the requantisation rounding chosen by `opts`
 * (nullable: nearest).  Errors: as qmuon_update_multi; QM_E_ARG for an
 * unknown rounding mode. */
QM_API qm_status qmuon_update_multi_ex(const void *host_plan, const void *dev_plan,
                                float beta, const qm_round_opts *opts,
                                double *block_sumsq, qm_stream_t stream);

/* The update plus grouped Frobenius normalisation ("Quantized Muon
 * Momentum", section "Grouped QKV And Sharding"): the update kernel
 * accumulates per-block sums of m*m; S_g sums them per group (fp64, fixed
 * order, no atomics); inv_g = (float)(1 / (sqrt(S_g) + eps)).
 *   write_normalized = 1: every grad element becomes
 *     round(float(m_stored) * inv_g) (the page's in-place semantics: the
 *     value an in-place scale of the stored m gives).  Run as two streaming
 *     passes: block sums of m first, then the update with the normalised
 *     value written in place of m (m recomputed bit for bit), so the grad
 *     buffer never holds the unnormalised m;
 *   write_normalized = 0: grads keep m and only inv_g is produced, for a
 *     Newton-Schulz call to fold in.
 *   group_inv_norm: nullable [n_groups] fp32 out.
 *   group_sumsq:    nullable [n_groups] fp64 out (S_g).
 *   ws: >= qm_update_workspace_bytes(host_plan) bytes, 256-byte aligned.
 * Errors: QM_E_ARG, QM_E_PLAN, QM_E_WORKSPACE, QM_E_HIP. */
QM_API qm_status qmuon_update_normalize_groups(const void *host_plan,
                                        const void *dev_plan, float beta,
                                        float eps, int32_t write_normalized,
                                        float *group_inv_norm,
                                        double *group_sumsq, void *ws,
                                        size_t ws_bytes, qm_stream_t stream);

/* qmuon_update_normalize_groups with the requantisation rounding chosen by
 * `opts` (nullable: nearest).  Errors: as qmuon_update_normalize_groups;
 * QM_E_ARG for an unknown rounding mode. */
QM_API qm_status qmuon_update_normalize_groups_ex(const void *host_plan,
                                           const void *dev_plan, float beta,
                                           float eps, int32_t write_normalized,
                                           const qm_round_opts *opts,
                                           float *group_inv_norm,
                                           double *group_sumsq, void *ws,
                                           size_t ws_bytes, qm_stream_t stream);

/* qmuon_update_normalize_groups without a workspace argument, for callers
 * that cannot allocate device memory (code under HIP graph capture, tight
 * serving loops, harnesses that forbid hipMalloc).  The workspace is a fixed
 * QM_NOALLOC_SCRATCH_BYTES array in device memory, one per GPU, set up on
 * the first call on that GPU and held until the process ends; the call
 * itself allocates nothing.  Every call on one GPU uses the same array:
 * calls that overlap on one GPU (two streams, or two host threads) race and
 * must be ordered by the caller.  Nothing in the array needs to start at
 * zero; a call writes every byte it reads.  Semantics and outputs as
 * qmuon_update_normalize_groups with nearest rounding.
 * Errors: as qmuon_update_normalize_groups; QM_E_WORKSPACE when the plan
 * needs more than QM_NOALLOC_SCRATCH_BYTES (qm_update_workspace_bytes tells:
 * about 8 bytes per 256-element block, so up to about 2e9 elements). */
#define QM_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)
QM_API qm_status qmuon_update_normalize_groups_noalloc(const void *host_plan,
                                                       const void *dev_plan,
                                                       float beta, float eps,
                                                       int32_t write_normalized,
                                                       float *group_inv_norm,
                                                       double *group_sumsq,
                                                       qm_stream_t stream);

/* The update emitting a row-wise MXFP8 carrier of m instead of writing m
 * to the grads ("Quantized Muon Momentum", section "Wave18B MXFP8 Carrier
 * Probe": uint8 E4M3 data, uint8 E8M0 inverse scales per 32 elements of a
 * row, one fp32 inverse Frobenius norm).  State: as qmuon_update_multi
 * with nearest rounding; the grads are only read.  Per 32 consecutive
 * elements of a tensor: amax = max|m|, scale byte
 * sb = clamp(floor(log2 amax) - 8, -127, 127) + 127 (0 when amax == 0),
 * data bytes = E4M3 of m * 2^(127 - sb) rounded to nearest even and
 * saturated at +-448 (1 sign, 4 exponent bits with bias 7, 3 mantissa bits,
 * subnormals, no infinities); m ~ E4M3 * 2^(sb - 127).  inv_norm: as
 * group_inv_norm of qmuon_update_normalize_groups, the input scale of
 * Newton-Schulz being inv_norm[g] times the decoded carrier.
 *   Layout: both arrays cover every tensor of the plan; tensor t occupies
 *   data bytes [256 B_t, 256 B_t + numel_t) and scale bytes
 *   [8 B_t, 8 B_t + numel_t / 32), B_t = sum of ceil(numel_s / 256) over the
 *   tensors s before t.  A row-major rows x cols tensor with cols % 32 == 0
 *   therefore has data shaped (rows, cols) and scales (rows, cols / 32).
 *   rowwise_data:      [n_blocks * 256] bytes, 8-byte aligned.
 *   rowwise_scale_inv: [n_blocks * 8] bytes.
 *   inv_norm:          [n_groups] fp32 out, required.
 *   group_sumsq:       nullable [n_groups] fp64 out.
 *   ws: >= qm_update_workspace_bytes(host_plan) bytes, 256-byte aligned.
 * Every tensor's numel must be a multiple of 32 (else QM_E_SHAPE); the
 * carrier arrays must not overlap each other or any tensor's codes, absmax
 * or grad span (QM_E_ARG).  Errors: QM_E_ARG, QM_E_ALIGN, QM_E_SHAPE,
 * QM_E_PLAN, QM_E_WORKSPACE, QM_E_HIP. */
QM_API qm_status qmuon_update_mxfp8_carrier(const void *host_plan,
                                            const void *dev_plan, float beta,
                                            float eps, uint8_t *rowwise_data,
                                            uint8_t *rowwise_scale_inv,
                                            float *inv_norm,
                                            double *group_sumsq, void *ws,
                                            size_t ws_bytes, qm_stream_t stream);

/* ------------------------------------------------------------------------
 * Newton-Schulz orthogonalisation
 *
 * Per matrix X0 (rows x cols, row stride ld elements): if rows > cols the
 * iteration runs on X0^T so the Gram matrix is min(rows, cols) square
 * ("MuonBP ...", key design 1, FLOP model with m <= n).  X0 is the input
 * times inv_norm[i] when given, else the input / (||input||_F + eps).  Then
 * T times ("NVIDIA ... Megatron", "Newton-Schulz distribuido": three products
 * per iteration):   A = X X^T;  B = b A + c A A;  X = a X + B X.
 * The first two products are symmetric and computed on lower-triangle tiles
 * only ("SYRK y reducción fusionada").  The result overwrites x in its dtype.
 * ---------------------------------------------------------------------- */

/* Workspace bytes for ns_orthogonalize on `batch` matrices of this shape.
 * For the fp32-operand precisions (QM_NS_F32, QM_NS_BF16X3) the figure
 * includes, where the symmetric products take the stream-K path, two part
 * slots per workgroup slot of the GPU, so it depends on the compute-unit
 * count of the current device: query it with the device that will run the
 * call current (the same holds for the muon_step, muon_apply and GRASP
 * workspace queries). */
QM_API size_t ns_workspace_bytes(int64_t rows, int64_t cols, int32_t batch,
                          int32_t precision);

/*   x: batch matrices; matrix i starts at x + i*batch_stride elements;
 *      dtype QM_F32 / QM_BF16 / QM_F16; ld >= cols.
 *   inv_norm: nullable device fp32 [batch].
 *   precision: qm_ns_precision.  steps >= 0.
 *   ws: >= ns_workspace_bytes(rows, cols, batch, precision), 256-byte aligned.
 * Errors: QM_E_ARG, QM_E_SHAPE, QM_E_DTYPE, QM_E_WORKSPACE, QM_E_HIP. */
QM_API qm_status ns_orthogonalize(void *x, int32_t dtype, int64_t rows, int64_t cols,
                           int64_t ld, int32_t batch, int64_t batch_stride,
                           int32_t steps, float a, float b, float c, float eps,
                           const float *inv_norm, int32_t precision, void *ws,
                           size_t ws_bytes, qm_stream_t stream);

/* Blockwise NS ("MuonBP ...", key design 1; "NVIDIA ... Megatron", blockwise
 * mode): the rows x cols matrix is cut into (rows/block_rows) x
 * (cols/block_cols) blocks, each orthogonalised independently with its own
 * norm and orientation, all in one batched run.  inv_norm: nullable device
 * fp32 [number of blocks], row-major block order.
 * Errors: as ns_orthogonalize; QM_E_SHAPE if the blocks do not tile. */
QM_API size_t ns_blocked_workspace_bytes(int64_t rows, int64_t cols,
                                  int64_t block_rows, int64_t block_cols,
                                  int32_t precision);
QM_API qm_status ns_orthogonalize_blocked(void *x, int32_t dtype, int64_t rows,
                                   int64_t cols, int64_t ld,
                                   int64_t block_rows, int64_t block_cols,
                                   int32_t steps, float a, float b, float c,
                                   float eps, const float *inv_norm,
                                   int32_t precision, void *ws,
                                   size_t ws_bytes, qm_stream_t stream);

/* Newton-Schulz of one rows x cols matrix handed over as an MXFP8 carrier
 * ("Quantized Muon Momentum", section "Wave18B MXFP8 Carrier Probe"; the
 * carrier of qmuon_update_mxfp8_carrier): X0 = inv_norm[0] * decode(data,
 * scale), decode(r, c) = E4M3(rowwise_data[r * cols + c]) *
 * 2^(rowwise_scale_inv[r * (cols / 32) + c / 32] - 127), then the iteration
 * of ns_orthogonalize; O is written to out (rows x cols, row pitch out_ld
 * elements, out_dtype).
 *   rowwise_data: [rows * cols] bytes, 8-byte aligned; cols % 32 == 0.
 *   rowwise_scale_inv: [rows * cols / 32] bytes.  inv_norm: device fp32
 *   [1], required.  ws: >= ns_workspace_bytes(rows, cols, 1, precision).
 * Errors: as ns_orthogonalize. */
QM_API qm_status ns_orthogonalize_mxfp8(const uint8_t *rowwise_data,
                                        const uint8_t *rowwise_scale_inv,
                                        const float *inv_norm, int64_t rows,
                                        int64_t cols, void *out,
                                        int32_t out_dtype, int64_t out_ld,
                                        int32_t steps, float a, float b,
                                        float c, int32_t precision, void *ws,
                                        size_t ws_bytes, qm_stream_t stream);

/* ------------------------------------------------------------------------
 * One full optimizer step
 * ---------------------------------------------------------------------- */
typedef struct {
    float beta;          /* momentum EMA factor                              */
    float eps;           /* Frobenius-normalisation epsilon                  */
    float a, b, c;       /* quintic coefficients                             */
    float lr_full;       /* step size on full steps                          */
    float lr_block;      /* step size on block steps                         */
    float weight_decay;  /* lambda, decoupled                                */
    float rms_scale;     /* update scale = rms_scale * sqrt(max(p, q))       */
    int32_t ns_steps;    /* T                                                */
    int32_t period;      /* P: step t is full iff t % P == 0 (P <= 1: all)   */
    int32_t precision;   /* qm_ns_precision                                  */
    int32_t rounding;    /* qm_rounding of the requantisation; stochastic uses
                            the step number as the counter offset            */
    int32_t carrier;     /* 1: the update hands m to Newton-Schulz as the
                            MXFP8 carrier of qmuon_update_mxfp8_carrier (in
                            the workspace; grads only read until O is
                            written; nearest rounding; cols and block_cols
                            multiples of 32); a tall matrix orthogonalised
                            whole (rows > cols, rows % 128 == 0, cols % 256
                            == 0, among the first 64) travels instead as the
                            row-wise carrier of m^T (one scale per 32 rows of
                            a column), which the first Gram product reads
                            along its contraction; 0: m is written to the
                            grads */
    uint64_t seed;       /* Philox key for stochastic rounding               */
} qm_muon_hparams;

typedef struct {
    int64_t rows, cols;              /* tensor i of the plans, row-major       */
    int64_t block_rows, block_cols;  /* partition used on block steps        */
    float *weight;                   /* fp32 [rows*cols], nullable           */
} qm_muon_matrix;

/* Workspace for muon_step over these matrices (both step kinds), with
 * carrier = 0. */
QM_API size_t muon_step_workspace_bytes(const void *host_plan_full,
                                 const void *host_plan_block,
                                 const qm_muon_matrix *mats, int32_t n_mats,
                                 int32_t precision);

/* Workspace for muon_step with these hyperparameters: as above, plus
 * 264 bytes per 256-element block for the carrier when hp->carrier = 1.
 * 0 if the plans, matrices or hp are unusable. */
QM_API size_t muon_step_workspace_bytes_ex(const void *host_plan_full,
                                    const void *host_plan_block,
                                    const qm_muon_matrix *mats, int32_t n_mats,
                                    const qm_muon_hparams *hp);

/* One Muon step with block-periodic orthogonalisation ("MuonBP ...",
 * flowchart and key designs 2-3):
 *   full = (period <= 1) || (step % period == 0) || no block plan;
 *   the q8 update with plan_full (one norm group per matrix, group i =
 *   tensor i) or plan_block (one group per block, row-major block order,
 *   numbered consecutively across matrices);
 *   NS of every matrix (full) or of every block (block step), input
 *   m * inv_g, output written over the grad buffer in its dtype;
 *   W <- W - lr (s O + weight_decay W), lr = lr_full or lr_block,
 *   s = rms_scale * sqrt(max(p, q)) for the p x q matrix orthogonalised.
 * step is 1-based.  With more than one block per matrix, every block must
 * consist of whole 256-element quantisation blocks (cols and block_cols
 * multiples of 256, or one column block with block_rows * cols a multiple
 * of 256), else QM_E_SHAPE; the block plan must give each quantisation block
 * the group of the block holding it, and both plans must name the same
 * tensors (codes, absmax, grad, size, dtype), else QM_E_PLAN.
 * Errors: as the calls above. */
QM_API qm_status muon_step(const void *host_plan_full, const void *dev_plan_full,
                    const void *host_plan_block, const void *dev_plan_block,
                    const qm_muon_matrix *mats, int32_t n_mats, int64_t step,
                    const qm_muon_hparams *hp, void *ws, size_t ws_bytes,
                    qm_stream_t stream);

/* The orthogonalise-and-apply half of muon_step on its own: given the group
 * inverse norms inv_norm (device fp32 [n_groups of the plan], e.g. from
 * qmuon_update_normalize_groups with write_normalized = 0) and the grads
 * holding m, run NS on every matrix (full = 1) or every block (full = 0) of
 * the plan's tensors, write O over the grads and apply the weight update.
 * muon_step is qmuon_update_normalize_groups followed by this call.
 * ws: >= muon_step_workspace_bytes(...) bytes (the same workspace works).
 * Errors: as muon_step. */
QM_API qm_status muon_apply(const void *host_plan, const qm_muon_matrix *mats,
                            int32_t n_mats, int32_t full,
                            const float *inv_norm, const qm_muon_hparams *hp,
                            void *ws, size_t ws_bytes, qm_stream_t stream);

/* ------------------------------------------------------------------------
 * GRASP 4-bit momentum ("4-bit-Muon-GRASP")
 *
 * The momentum of one rows x cols matrix is a rank-k factor P R^T (P rows x
 * k, R cols x k, 8-bit) plus a residual (4-bit), all grid-quantised over
 * 64 x 64 blocks (clipped at the edges): an entry is divided by the smaller
 * of its row's and its column's absolute maximum inside its block, and coded
 * as clamp(rint((x / d) * L), -L, L), L = 7 (4-bit) or 127 (8-bit), d = 0
 * giving code 0; it dequantises to code * (d / L).  The state starts as all
 * zeros.  Layout (all caller-owned device buffers):
 * ---------------------------------------------------------------------- */
typedef struct {
    uint8_t *res_codes;  /* [rows][ceil(cols/2)]: two 4-bit two's-complement
                            codes per byte, even column in the low nibble   */
    float *res_rmax;     /* [rows][ceil(cols/64)] row maxima per block      */
    float *res_cmax;     /* [ceil(rows/64)][cols] column maxima per block   */
    int8_t *p_codes;     /* [rows][k]                                       */
    float *p_rmax;       /* [rows]                                          */
    float *p_cmax;       /* [ceil(rows/64)][k]                              */
    int8_t *r_codes;     /* [cols][k]                                       */
    float *r_rmax;       /* [cols]                                          */
    float *r_cmax;       /* [ceil(cols/64)][k]                              */
} qm_grasp_state;

QM_API size_t grasp_workspace_bytes(int64_t rows, int64_t cols, int32_t rank);

/* One GRASP step (the page's update equations):
 *   M_{t-1} = deq(res) + deq(P) deq(R)^T;   M_t = mu M_{t-1} + g (no (1-mu))
 *   Q = R_{t-1} with unit columns (a zero column is replaced by the same
 *   column of `warm`, cols x k fp32, normalised);  P = MGS(M_t Q) (modified
 *   Gram-Schmidt, positive diagonal);  R = M_t^T P;  residual M_t - P R^T;
 *   requantise residual, P, R;  O = NS_T(M_t) on fp32 operands (ns_precision
 *   QM_NS_F32 or QM_NS_BF16X3), written over grad in its dtype;
 *   W <- W - lr (O + weight_decay W) if weight.
 * Reductions accumulate in fp64 in a fixed order; P, R are rounded to fp32
 * before the residual.  rank in {1, 2, 4, 8, 16}; grid must be 64.
 *   grad: in g, out O (rows x cols contiguous, dtype grad_dtype).
 *   ws: >= grasp_workspace_bytes(rows, cols, rank), 256-byte aligned.
 * Errors: QM_E_ARG, QM_E_SHAPE, QM_E_DTYPE, QM_E_ALIGN, QM_E_UNSUPPORTED,
 * QM_E_WORKSPACE, QM_E_HIP. */
QM_API qm_status grasp_step(const qm_grasp_state *state, int64_t rows,
                            int64_t cols, int32_t rank, int32_t grid,
                            void *grad, int32_t grad_dtype, const float *warm,
                            float mu, int32_t ns_steps, float a, float b,
                            float c, float eps, int32_t ns_precision,
                            float *weight, float lr, float weight_decay,
                            void *ws, size_t ws_bytes, qm_stream_t stream);

/* ------------------------------------------------------------------------
 * Global gradient norm and clipping
 *
 * Over the grads of a whole model (those Muon steps and those AdamW steps):
 *   S = sum of g*g over every element (fp64);  norm = sqrt(S);
 *   coef = min(1, max_norm / (norm + eps)),  NaN if S is not finite.
 * coef stays on the device: adamw_step multiplies it into the gradients it
 * reads, grad_scale into gradients in place (those of the Muon step).  A NaN
 * coef stops adamw_step and grad_scale, not muon_step, muon_apply or
 * grasp_step: these read the gradients whatever they hold, and an infinity
 * or a NaN stays in their momentum.  A program that may meet one copies coef
 * to the host and leaves the Muon step out where it is NaN.
 * ---------------------------------------------------------------------- */
typedef struct {
    void *grad;         /* dtype, aligned to its element                     */
    int64_t numel;      /* >= 0                                              */
    int64_t cols, ld;   /* cols = 0: contiguous; else rows of cols elements
                           (a divisor of numel) at pitch ld >= cols; numel
                           < 2^32 then                                       */
    int32_t dtype;      /* qm_dtype                                          */
    int32_t reserved;   /* must be 0                                         */
} qm_grad_tensor;

/* Build a grad-list blob (host only; touches no GPU), used like a norm plan:
 * the caller copies it verbatim to the device once (64-byte aligned) and
 * passes both copies.  The blob holds the buffers' addresses: a buffer that
 * moves (a gradient allocated anew each step) needs a new blob.
 * host_blob == NULL asks for the size, as in qm_plan_encode.  Errors: QM_E_ARG (null, counts, overlapping buffers),
 * QM_E_ALIGN, QM_E_DTYPE, QM_E_SHAPE, QM_E_UNSUPPORTED. */
QM_API qm_status qm_grad_plan_encode(const qm_grad_tensor *grads, int32_t n_grads,
                                     void *host_blob, size_t *inout_blob_bytes);

/* Workspace bytes of grad_norm for this blob (0 if it is not a grad list). */
QM_API size_t grad_norm_workspace_bytes(const void *host_plan);

/* norm_out[0], coef_out[0]: device fp32 out, as defined above (max_norm > 0,
 * infinity allowed: coef is then 1; eps >= 0), two different numbers.  Fixed
 * summation order, no atomics.  ws: >= grad_norm_workspace_bytes, 8-byte aligned.
 * Errors: QM_E_ARG, QM_E_PLAN, QM_E_ALIGN, QM_E_WORKSPACE, QM_E_HIP. */
QM_API qm_status grad_norm(const void *host_plan, const void *dev_plan,
                           double max_norm, double eps, float *norm_out,
                           float *coef_out, void *ws, size_t ws_bytes,
                           qm_stream_t stream);

/* Every grad of the list times coef[0] (device fp32), rounded to nearest
 * even into its dtype; a NaN coef leaves the grads as they are.
 * Errors: QM_E_ARG, QM_E_PLAN, QM_E_ALIGN, QM_E_HIP. */
QM_API qm_status grad_scale(const void *host_plan, const void *dev_plan,
                            const float *coef, qm_stream_t stream);

/* ------------------------------------------------------------------------
 * AdamW over many tensors ("Decoupled Weight Decay Regularization",
 * Loshchilov and Hutter, ICLR 2019), for the parameters a Muon step does not
 * fit: embeddings, heads, norm gains, biases.  Per element, with t the step,
 * g the gradient (times *grad_scale if given), lr_t = lr * lr_scale:
 *   m <- beta1 m + (1 - beta1) g;   v <- beta2 v + (1 - beta2) g g;
 *   w <- w - lr_t weight_decay w
 *          - lr_t (m / (1 - beta1^t)) / (sqrt(v / (1 - beta2^t)) + eps)
 * in fp32, the new w rounded to nearest even into its dtype, and into `copy`
 * if given (the low-precision weight a model computes with next to its fp32
 * weight).  Grads are only read.
 *
 * States in 32 bits: m and v are fp32.  States in 8 bits, per 256-element
 * block (the last block of a tensor covers the remainder):
 *   m = m_code * (m_absmax / 127),         m_code int8 in [-127, 127];
 *   v = v_code^2 * (v_absmax / 65025),     v_code uint8 (65025 = 255^2).
 * v_code is proportional to sqrt(v), the number the update divides by: a
 * block spans a factor of 255 in it, and decoding needs no root.  The weight
 * sees the new m and v before they are coded.  Coding, in binary32 with one
 * rounding per operation: step_m = beta1 (m_absmax / 127), step_v = beta2
 * (v_absmax / 65025), m = m_code step_m + (1 - beta1) g, v = (v_code v_code)
 * step_v + (1 - beta2) (g g); m_absmax' = max|m|, v_absmax' = max v over the
 * block (0 if below 2^-100: the block then holds zeros);
 *   x = m (127 / m_absmax'),   m_code' = x rounded to nearest even;
 *   y = v (65025 / v_absmax'), k = floor(sqrt(y)), v_code' = k + 1 if
 *   y - k^2 > k + 1/2, else k (the code whose square is nearest), and at
 *   least 1 where v > 0, so that no update is divided by eps alone.
 * A block whose maximum is not finite gets codes 0 and that maximum (a NaN
 * counts as the largest), and decodes to NaN from then on.
 *
 * Nearest rounding holds an 8-bit v still once its change per step is less
 * than half a code's, which with beta2 near 1 is soon the case; stochastic
 * rounding keeps the mean: with r the element's random word (the counter and
 * key of qm_rounding, the tensor's index in this list), m_code' =
 * floor(x) + 1 if (r >> 16) 2^-16 < x - floor(x), else floor(x); v_code' =
 * k + 1 if y - k^2 > (r mod 2^15) 2^-15 (2k + 1), else k: the mean of the
 * code's square is y for y >= 1.  For 0 < y < 1 the code is 1 always (as with
 * nearest rounding, no smaller one is kept where v > 0), so v reads too large
 * there, by the factor 1 / y, until it passes its block's smallest code or
 * its block's maximum falls.  Clamped to the codes' ranges.  The two sides of every
 * comparison here and above are exact numbers: x and y are binary32, the
 * differences and products made from them are not rounded.
 * ---------------------------------------------------------------------- */
typedef struct {
    void *weight;        /* weight_dtype [numel], in/out                     */
    const void *grad;    /* grad_dtype                                       */
    void *m, *v;         /* [numel] fp32 (state_bits 32), or int8 and uint8
                            codes (state_bits 8), in/out                     */
    float *m_absmax;     /* state_bits 8: [ceil(numel/256)], in/out; else
                            null                                             */
    float *v_absmax;     /* the same                                         */
    void *copy;          /* nullable: copy_dtype [numel], out                */
    int64_t numel;       /* >= 0                                             */
    int64_t grad_cols, grad_ld;  /* as cols, ld of qm_grad_tensor            */
    int32_t weight_dtype, grad_dtype;   /* qm_dtype                          */
    int32_t copy_dtype;  /* QM_BF16 or QM_F16; ignored without copy          */
    int32_t state_bits;  /* 32 or 8                                          */
    float lr_scale;      /* finite                                           */
    float weight_decay;  /* finite                                           */
} qm_adamw_tensor;

typedef struct {
    double lr, beta1, beta2, eps;  /* 0 <= beta < 1, eps >= 2^-126; lr and
                                      lr / (1 - beta1^t) finite in fp32      */
    int64_t step;        /* t, 1-based                                       */
    int32_t rounding;    /* qm_rounding of 8-bit states                      */
    uint32_t offset;     /* counter word 2 of stochastic rounding            */
    uint64_t seed;       /* its key                                          */
} qm_adamw_hparams;

/* Build an AdamW list blob (host only); use as qm_grad_plan_encode's.  All
 * buffers aligned to their elements, none overlapping another.  A list has
 * at most 2^25 - 4 tasks of 1024 elements (256 at a tensor's end, and
 * throughout a tensor whose grad's rows are strided and no multiple of 8),
 * else QM_E_UNSUPPORTED; so has a grad list. */
QM_API qm_status qm_adamw_plan_encode(const qm_adamw_tensor *tensors, int32_t n_tensors,
                                      void *host_blob, size_t *inout_blob_bytes);

/* Blocks of all tensors of a grad or AdamW list, in list order (tensor t's
 * first block is the sum of ceil(numel / 256) over the tensors before it);
 * -1 if the blob is neither. */
QM_API int64_t qm_list_blocks(const void *host_plan);

/* One AdamW step over every tensor of the list.  grad_scale: nullable device
 * fp32 [1]; if it is NaN (a gradient norm that is not finite) nothing is
 * written.  Errors: QM_E_ARG, QM_E_ALIGN, QM_E_PLAN, QM_E_HIP. */
QM_API qm_status adamw_step(const void *host_plan, const void *dev_plan,
                            const qm_adamw_hparams *hp, const float *grad_scale,
                            qm_stream_t stream);

/* The values the states stand for, e.g. for a checkpoint that does not
 * depend on the state's form: element e of tensor t goes to m_out and v_out
 * [256 * (t's first block) + e] (fp32 [256 * qm_list_blocks], 16-byte
 * aligned, not overlapping); what lies between two tensors is set to 0.
 * Errors: QM_E_ARG, QM_E_ALIGN, QM_E_PLAN, QM_E_HIP. */
QM_API qm_status adamw_read_state(const void *host_plan, const void *dev_plan,
                                  float *m_out, float *v_out, qm_stream_t stream);

/* ------------------------------------------------------------------------
 * What makes the gradients: activations kept in 8 bits from the forward to
 * the backward pass, the weight gradient that is formed from them, the gated
 * activation between two products, the embedding and its gradient.  Results go
 * to the gradient buffers that the steps above read, whole or added to what
 * they hold (accumulate = 1: several batches a step, a tied table).
 *
 * Matrices are rows x cols with a row pitch ld in elements (cols <= ld <=
 * 2^24 - 16) and aligned to their elements; a matrix without elements may be
 * null.  Fastest are rows of a multiple of 8 elements at 16-byte addresses.
 * An output shares no memory with another buffer of its call (columns of one
 * wider buffer are separate buffers).
 * ---------------------------------------------------------------------- */

/* A rows x cols matrix in 8 bits: one E4M3 byte an element (format of
 * qmuon_update_mxfp8_carrier) and one scale byte for 32 consecutive rows of a
 * column (the last group takes the remainder):
 *   value(r, c) = E4M3(data[r * ld + c]) * 2^(scale[(r / 32) * ld + c] - 127).
 * Coding: scale - 127 = e, the smallest integer with max|x| <= 448 * 2^e over
 * the group, between -95 and 119; data = E4M3(x * 2^-e), rounded to nearest
 * even, at most 448.  A value is off by at most 1/16 of itself, or by 2^-10 *
 * 2^e where it is below 2^-6 * 2^e, and exact in fp32 and bf16; magnitudes past
 * 448 * 2^119 = 2.98e38 become that.  A group that holds an infinity or a NaN
 * decodes to NaN as a whole.  Scale bytes are 32 to 246; what others stand for
 * is not defined, but that 0 beside zero bytes (cleared buffers) is 0.  Rows
 * share a scale, not columns: an activation's outliers keep to their columns,
 * and a weight gradient contracts over the rows. */
typedef struct {
    uint8_t *data;       /* [rows * ld], 16-byte aligned                     */
    uint8_t *scale;      /* [ceil(rows / 32) * ld], 16-byte aligned          */
    int64_t rows, cols;
    int64_t ld;          /* multiple of 16, cols <= ld <= 2^24 - 16; bytes
                            past cols may be written                         */
} qm_act8;

/* kept = x in 8 bits.  Errors: QM_E_ARG, QM_E_ALIGN, QM_E_DTYPE, QM_E_SHAPE,
 * QM_E_UNSUPPORTED (more than 2^25 patches of 32 x 128), QM_E_HIP. */
QM_API qm_status act_pack(const void *x, int32_t dtype, int64_t ld,
                          const qm_act8 *kept, qm_stream_t stream);

/* out = the values kept stands for, rounded to nearest even into its dtype.
 * f16 numbers of magnitude 63488 and more are kept as 65536, an infinity in f16.
 * Errors: as act_pack. */
QM_API qm_status act_read(const qm_act8 *kept, void *out, int32_t dtype,
                          int64_t ld, qm_stream_t stream);

/* Gradient of a linear layer's weight (n x k) over rows tokens:
 *   out[i][j] (= or +=) sum over t of dy[t][i] * x[t][j]
 * dy: rows x n, bf16 or f16.  x: rows x k of the same type, or null with
 * `kept` in its place (its values, in f16 rounded as act_read does).  Products exact,
 * sums in fp32 in an order that the sizes determine; the result is rounded
 * once.  out: any dtype, ld_out < 2^21.  rows = 0: zeros, or nothing to add.
 *   ws: >= weight_grad_workspace_bytes(rows, n, k) bytes (0: none needed),
 *   16-byte aligned.
 * Errors: QM_E_ARG, QM_E_ALIGN, QM_E_DTYPE, QM_E_SHAPE, QM_E_WORKSPACE,
 * QM_E_UNSUPPORTED (more than 2^22 tiles of 128 x 128), QM_E_HIP. */
QM_API size_t weight_grad_workspace_bytes(int64_t rows, int64_t n, int64_t k);
QM_API qm_status weight_grad(const void *dy, int32_t dtype, int64_t ld_dy,
                             const void *x, int64_t ld_x, const qm_act8 *kept,
                             int64_t rows, int64_t n, int64_t k, void *out,
                             int32_t out_dtype, int64_t ld_out,
                             int32_t accumulate, void *ws, size_t ws_bytes,
                             qm_stream_t stream);

/* Gated activation of a feed-forward block: h = act(gate) * up, in fp32,
 * rounded once.  QM_ACT_SILU: act(g) = g / (1 + exp(-g)); QM_ACT_GELU:
 * act(g) = g / 2 * (1 + tanh(sqrt(2 / pi) * (g + 0.044715 g^3))).
 *   gate8, up8: both null, or what receives gate and up in 8 bits (as
 *   act_pack codes them) for the backward pass, which reads those alone.
 * gate, up and h: rows x cols, one dtype.  Errors: as act_pack. */
typedef enum { QM_ACT_SILU = 0, QM_ACT_GELU = 1 } qm_act;
QM_API qm_status gated_act_forward(const void *gate, int64_t ld_gate,
                                   const void *up, int64_t ld_up, int32_t dtype,
                                   int64_t rows, int64_t cols, int32_t act,
                                   void *h, int64_t ld_h, const qm_act8 *gate8,
                                   const qm_act8 *up8, qm_stream_t stream);

/* Its backward pass at the kept values g, u of gate and up:
 *   dgate = dh * u * act'(g);   dup = dh * act(g);
 *   h (nullable): act(g) * u, for the weight gradient of the product that
 *   follows.
 * dh, dgate, dup and h: one dtype.  Errors: as act_pack. */
QM_API qm_status gated_act_backward(const qm_act8 *gate8, const qm_act8 *up8,
                                    const void *dh, int64_t ld_dh, int32_t dtype,
                                    int32_t act, void *dgate, int64_t ld_dgate,
                                    void *dup, int64_t ld_dup, void *h,
                                    int64_t ld_h, qm_stream_t stream);

/* out[i] = scale * table[tokens[i]], rounded once; a token outside [0, vocab)
 * (padding) gives a row of zeros, whatever the scale.  tokens: contiguous int32
 * or int64 (token_bits); fewer than 2^30 tokens and values.  Errors: QM_E_ARG,
 * QM_E_ALIGN, QM_E_DTYPE, QM_E_SHAPE, QM_E_UNSUPPORTED (2^34 pieces of 4 or 8
 * columns, or more), QM_E_HIP. */
QM_API qm_status embedding_lookup(const void *tokens, int32_t token_bits,
                                  int64_t n_tokens, const void *table,
                                  int32_t table_dtype, int64_t ld_table,
                                  int64_t vocab, int64_t cols, float scale,
                                  void *out, int32_t out_dtype, int64_t ld_out,
                                  qm_stream_t stream);

/* Its gradient: grad[v] (= or +=) scale * sum of dy[i] over tokens[i] = v, in
 * fp32, in an order that the tokens determine, rounded once.  With accumulate
 * only rows that have tokens are touched.  A token outside [0, vocab) has no
 * part in it.
 *   ws: >= embedding_grad_workspace_bytes(n_tokens, vocab, cols) bytes,
 *   16-byte aligned.
 * Errors: as embedding_lookup, and QM_E_WORKSPACE; QM_E_UNSUPPORTED: a launch of
 * 2^31 threads or more, which 2^27 tokens of up to 1024 columns and a vocabulary
 * of 2^27 stay below. */
QM_API size_t embedding_grad_workspace_bytes(int64_t n_tokens, int64_t vocab,
                                             int64_t cols);
QM_API qm_status embedding_grad(const void *tokens, int32_t token_bits,
                                int64_t n_tokens, const void *dy,
                                int32_t dy_dtype, int64_t ld_dy, void *grad,
                                int32_t grad_dtype, int64_t ld_grad,
                                int64_t vocab, int64_t cols, float scale,
                                int32_t accumulate, void *ws, size_t ws_bytes,
                                qm_stream_t stream);

/* ------------------------------------------------------------------------
 * Launch timing (measurement aid, off by default).
 *
 * While enabled, the launches of each class below carry two HIP events on
 * their dispatches (hipExtLaunchKernel: the start event on the first kernel
 * of the class's launch group, the stop event on its last), so a reader gets
 * the same per-launch device time a kernel-trace profiler reports.  The events
 * still cost the stream a few microseconds per launch group, so a caller
 * timing whole calls may record on some steps only (mode 2 below).  Enabling
 * clears earlier records unless resumed with mode 2; disabling keeps them for
 * qm_timing_read.  Not for use inside HIP graph capture.  The recorder is
 * process-wide and locked; launches from several threads are recorded but
 * interleave in one list.
 */
typedef enum {
    QM_K_Q8_UPDATE = 0,     /* blockwise q8 momentum update kernel */
    QM_K_GROUP_REDUCE = 1,  /* per-group sum of squares (both stages) */
    QM_K_Q8_SCALE = 2,      /* in-place normalisation pass: no longer launched (the
                             * normalising update writes normalised values itself) */
    QM_K_NS_NORM = 3,       /* Frobenius norm of NS inputs (both stages) */
    QM_K_NS_PROLOGUE = 4,   /* orientation, scaling, X and X^T */
    QM_K_NS_GRAM = 5,       /* A = X X^T (symmetric product) */
    QM_K_NS_POLY = 6,       /* B = b A + c A A (symmetric product) */
    QM_K_NS_XUPDATE = 7,    /* X = a X + B X */
    QM_K_NS_WRITEBACK = 8,  /* output and fused weight update */
    QM_K_Q8_SUMS = 9,       /* block sums of m only: first pass of the normalising update */
    QM_K_CLASSES = 10
} qm_kernel_class;

/* on == 1: clear records and start recording; on == 2: resume recording,
 * keeping the records so far; on == 0: stop.
 * Errors: QM_E_ARG (another value), QM_E_HIP (event creation failed). */
QM_API qm_status qm_timing_enable(int32_t on);

/* Sum of the recorded launch durations of one class (milliseconds) and the
 * number of launches.  Waits for the recorded events to complete.
 * Errors: QM_E_ARG (class out of range, null outputs), QM_E_HIP. */
QM_API qm_status qm_timing_read(int32_t kernel_class, double *total_ms,
                                int64_t *launches);

/* Measurement aid: copy `bytes` from src to dst (device pointers, 16-byte
 * aligned, bytes a multiple of 16, not overlapping) with the q8 update
 * kernel's access pattern (16-byte non-temporal loads and stores, each wave
 * instruction one contiguous 1 KiB span).  It gives the achievable HBM rate
 * for a 50/50 read/write stream, the ceiling the update kernels are measured
 * against, and a kernel of exactly known traffic to calibrate HBM byte
 * counters.  Errors: QM_E_ARG (null, overlap), QM_E_ALIGN, QM_E_HIP. */
QM_API qm_status qm_hbm_stream_copy(const void *src, void *dst, size_t bytes,
                                    qm_stream_t stream);

/* ------------------------------------------------------------------------ */
QM_API const char *qm_status_string(qm_status s);
QM_API const char *qm_last_error(void);
QM_API int qm_abi_version(void);

#ifdef __cplusplus
}
#endif
#endif /* QMUON_H */
