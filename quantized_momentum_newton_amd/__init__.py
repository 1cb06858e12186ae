"""Python binding of libqmuon.so: one quantized-momentum Muon step on MI355X.

Argument marshalling only: every step of the computation runs in the HIP
kernels of libqmuon.so.  PyTorch supplies device memory and the stream
(torch's current stream unless one is given).  There is no CPU or PyTorch
fallback; if the library is missing the import fails.

Entry points (same names as the C ABI in include/qmuon.h):
  Plan(...)                        qm_plan_encode + one host-to-device copy
  qmuon_update_multi               q8 momentum update, many tensors, one launch
  qmuon_update_normalize_groups    update + grouped Frobenius normalisation
  qmuon_update_normalize_groups_noalloc
                                   the same without a workspace (fixed per-GPU
                                   scratch; for callers that cannot allocate)
  MXCarrier, qmuon_update_mxfp8_carrier
                                   update emitting the MXFP8 carrier of m
  ns_orthogonalize_mxfp8           Newton-Schulz of a carrier-held matrix
  ns_orthogonalize                 quintic Newton-Schulz, batched
  ns_orthogonalize_blocked         blockwise Newton-Schulz
  muon_step                        update + NS + weight apply, block-periodic
  muon_apply                       the NS + weight-apply half of muon_step
  GraspState, grasp_step           the GRASP 4-bit momentum variant
  GradPlan, grad_norm, grad_scale  global gradient norm, clip factor, clipping in place
  AdamWState, AdamWPlan, adamw_step, adamw_read_state
                                   AdamW over many tensors, states in 32 or 8 bits
  timing_enable, timing_read       per-kernel-class launch timing (HIP events)
"""
import ctypes

import torch

from . import _lib as L

_LIB = L.load()

QUINTIC = (3.4445, -4.7750, 2.0315)
BLOCK = 256      # elements per absmax block
PRECISION = {"bf16": L.QM_NS_BF16, "f32": L.QM_NS_F32, "bf16x3": L.QM_NS_BF16X3}
_DTYPES = {torch.float32: L.QM_F32, torch.bfloat16: L.QM_BF16, torch.float16: L.QM_F16}


class QmuonError(RuntimeError):
    def __init__(self, status):
        self.status = status
        name = L.STATUS_NAMES.get(status, str(status))
        msg = (_LIB.qm_last_error() or b"").decode()
        super().__init__(f"{name}: {msg}")


def _check(st):
    if st != L.QM_OK:
        raise QmuonError(st)


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def _require(t, name, dtype, device, numel=None, shape=None):
    """Raise unless t is a contiguous `dtype` tensor on `device` with exactly
    `numel` elements / this shape (the C side reads that many elements at
    t.data_ptr())."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name} has {t.numel()} elements, expected {numel}")


def _dtype(t):
    try:
        return _DTYPES[t.dtype]
    except KeyError:
        raise TypeError(f"unsupported dtype {t.dtype}") from None


def abi_version():
    return _LIB.qm_abi_version()


# Kernel classes of qm_timing_read (qm_kernel_class in include/qmuon.h).
KERNEL_CLASSES = {"q8_update": 0, "group_reduce": 1, "q8_scale": 2, "ns_norm": 3, "ns_prologue": 4,
                  "ns_gram": 5, "ns_poly": 6, "ns_xupdate": 7, "ns_writeback": 8, "q8_sums": 9}


def timing_enable(on=True, resume=False):
    """Start (clearing earlier records), resume (keeping them) or stop
    recording launch times."""
    _check(_LIB.qm_timing_enable((2 if resume else 1) if on else 0))


def timing_read(kernel_class):
    """(total milliseconds, launches) recorded for one kernel class."""
    ms, n = ctypes.c_double(), ctypes.c_int64()
    _check(_LIB.qm_timing_read(KERNEL_CLASSES[kernel_class], ctypes.byref(ms), ctypes.byref(n)))
    return ms.value, n.value


class Plan:
    """A norm plan over q8 tensors, encoded once and copied to the device once.

    tensors : list of (codes, absmax fp32, grad) device tensors.  codes are int8,
              or uint8 holding the same bytes; codes and absmax contiguous.  grad
              is contiguous, or a 2-D view with unit column stride (rows of
              grad.shape[1] elements at pitch grad.stride(0)).
    segments: list of (tensor_index, start, length, group_id) element ranges
              (logical row-major element order)
    n_groups: number of norm groups
    """

    def __init__(self, tensors, segments, n_groups, device=None):
        n = len(tensors)
        arr = (L.Q8Tensor * n)()
        for i, (codes, absmax, grad) in enumerate(tensors):
            for t in (codes, absmax):
                if not t.is_contiguous():
                    raise ValueError("codes and absmax must be contiguous")
            if codes.dtype not in (torch.int8, torch.uint8):
                raise TypeError("codes must be int8 or uint8")
            cols, ld = 0, 0
            if not grad.is_contiguous():
                if grad.dim() != 2 or grad.stride(1) != 1:
                    raise ValueError("a non-contiguous grad must be 2-D with unit column stride")
                cols, ld = grad.shape[1], grad.stride(0)
            arr[i] = L.Q8Tensor(codes.data_ptr(), absmax.data_ptr(), grad.data_ptr(),
                                grad.numel(), _dtype(grad), 0, cols, ld)
        segs = (L.NormSegment * len(segments))()
        for k, (ti, start, length, gid) in enumerate(segments):
            segs[k] = L.NormSegment(ti, gid, start, length)
        size = ctypes.c_size_t(0)
        _check(_LIB.qm_plan_encode(arr, n, segs, len(segments), n_groups, None,
                                   ctypes.byref(size)))
        self.host = torch.empty(size.value, dtype=torch.uint8)
        _check(_LIB.qm_plan_encode(arr, n, segs, len(segments), n_groups,
                                   ctypes.c_void_p(self.host.data_ptr()), ctypes.byref(size)))
        dev = device if device is not None else tensors[0][0].device
        self.dev = self.host.to(dev)
        self._keep = [t for trip in tensors for t in trip]
        nt, ng = ctypes.c_int32(), ctypes.c_int32()
        nb, numel = ctypes.c_int64(), ctypes.c_int64()
        _check(_LIB.qm_plan_info(self.hptr, ctypes.byref(nt), ctypes.byref(ng),
                                 ctypes.byref(nb), ctypes.byref(numel)))
        self.n_tensors, self.n_groups = nt.value, ng.value
        self.n_blocks, self.total_numel = nb.value, numel.value
        self.device = dev
        # global index of each tensor's first 256-element block (plan order)
        self.numels = [int(t[2].numel()) for t in tensors]
        self.block_offsets = [0]
        for n_ in self.numels[:-1]:
            self.block_offsets.append(self.block_offsets[-1] + -(-n_ // BLOCK))

    @property
    def hptr(self):
        return ctypes.c_void_p(self.host.data_ptr())

    @property
    def dptr(self):
        return ctypes.c_void_p(self.dev.data_ptr())

    def workspace_bytes(self):
        return _LIB.qm_update_workspace_bytes(self.hptr)

    def workspace(self):
        return torch.empty(max(self.workspace_bytes(), 256), dtype=torch.uint8, device=self.device)


ROUNDING = {"nearest": L.QM_ROUND_NEAREST, "stochastic": L.QM_ROUND_STOCHASTIC}


def _round_opts(rounding, seed, offset):
    if rounding == "nearest":
        return None
    return ctypes.byref(L.RoundOpts(ROUNDING[rounding], offset, seed))


def qmuon_update_multi(plan, beta, block_sumsq=None, stream=None, rounding="nearest", seed=0, offset=0):
    """In-place q8 update of every tensor in the plan; block_sumsq (fp64
    [n_blocks]) optionally receives the per-block sums of m*m.  rounding:
    "nearest" or "stochastic" (random stream chosen by seed and offset)."""
    if rounding == "nearest":
        _check(_LIB.qmuon_update_multi(plan.hptr, plan.dptr, beta, _ptr(block_sumsq), _stream(stream)))
    else:
        _check(_LIB.qmuon_update_multi_ex(plan.hptr, plan.dptr, beta, _round_opts(rounding, seed, offset),
                                          _ptr(block_sumsq), _stream(stream)))


def qmuon_update_normalize_groups(plan, beta, eps, write_normalized=True, group_inv_norm=None,
                                  group_sumsq=None, ws=None, stream=None, rounding="nearest", seed=0,
                                  offset=0):
    if ws is None:
        ws = plan.workspace()
    if rounding == "nearest":
        _check(_LIB.qmuon_update_normalize_groups(
            plan.hptr, plan.dptr, beta, eps, int(write_normalized), _ptr(group_inv_norm),
            _ptr(group_sumsq), _ptr(ws), ws.numel(), _stream(stream)))
    else:
        _check(_LIB.qmuon_update_normalize_groups_ex(
            plan.hptr, plan.dptr, beta, eps, int(write_normalized), _round_opts(rounding, seed, offset),
            _ptr(group_inv_norm), _ptr(group_sumsq), _ptr(ws), ws.numel(), _stream(stream)))


def qmuon_update_normalize_groups_noalloc(plan, beta, eps, write_normalized=True, group_inv_norm=None,
                                          group_sumsq=None, stream=None):
    """qmuon_update_normalize_groups with the library's fixed per-GPU scratch
    instead of a workspace (the call allocates nothing).  Calls that overlap
    on one GPU race: order them.  Plans needing more than
    QM_NOALLOC_SCRATCH_BYTES of workspace are refused."""
    for t, dt, n in ((group_inv_norm, torch.float32, plan.n_groups), (group_sumsq, torch.float64, plan.n_groups)):
        if t is not None:
            _require(t, "group output", dt, plan.device, numel=n)
    _check(_LIB.qmuon_update_normalize_groups_noalloc(plan.hptr, plan.dptr, beta, eps, int(write_normalized),
                                                      _ptr(group_inv_norm), _ptr(group_sumsq), _stream(stream)))


class MXCarrier:
    """Row-wise MXFP8 carrier arrays covering every tensor of a plan (the
    layout qmuon_update_mxfp8_carrier writes): E4M3 bytes [n_blocks * 256],
    E8M0 scale bytes [n_blocks * 8], fp32 inverse norms [n_groups]."""

    def __init__(self, plan):
        self.plan = plan
        dev = plan.device
        self.rowwise_data = torch.empty(plan.n_blocks * BLOCK, dtype=torch.uint8, device=dev)
        self.rowwise_scale_inv = torch.empty(plan.n_blocks * (BLOCK // 32), dtype=torch.uint8, device=dev)
        self.inv_norm = torch.empty(plan.n_groups, dtype=torch.float32, device=dev)

    def data(self, i, shape=None):
        """Tensor i's E4M3 bytes (numel, or shaped (rows, cols))."""
        e0, n = self.plan.block_offsets[i] * BLOCK, self.plan.numels[i]
        v = self.rowwise_data[e0:e0 + n]
        return v.view(shape) if shape is not None else v

    def scale_inv(self, i, shape=None):
        """Tensor i's E8M0 bytes (numel / 32, or shaped (rows, cols / 32))."""
        e0, n = self.plan.block_offsets[i] * (BLOCK // 32), self.plan.numels[i] // 32
        v = self.rowwise_scale_inv[e0:e0 + n]
        return v.view(shape[0], shape[1] // 32) if shape is not None else v


def qmuon_update_mxfp8_carrier(plan, beta, eps, carrier=None, group_sumsq=None, ws=None, stream=None):
    """q8 update of every tensor in the plan emitting the MXFP8 carrier of m
    (and the group inverse norms into carrier.inv_norm); grads are only read.
    Returns the carrier."""
    if carrier is None:
        carrier = MXCarrier(plan)
    if ws is None:
        ws = plan.workspace()
    _check(_LIB.qmuon_update_mxfp8_carrier(plan.hptr, plan.dptr, beta, eps, _ptr(carrier.rowwise_data),
                                           _ptr(carrier.rowwise_scale_inv), _ptr(carrier.inv_norm),
                                           _ptr(group_sumsq), _ptr(ws), ws.numel(), _stream(stream)))
    return carrier


def ns_orthogonalize_mxfp8(data, scale_inv, inv_norm, out, steps=5, coeffs=QUINTIC, precision="bf16",
                           ws=None, stream=None):
    """NS of the rows x cols matrix carried as (data uint8 (rows, cols),
    scale_inv uint8 (rows, cols / 32), inv_norm fp32 [1]); O written to out
    (rows x cols, unit column stride, fp32/bf16/f16)."""
    rows, cols = out.shape
    if out.stride(1) != 1:
        raise ValueError("out rows must be contiguous")
    for t in (data, scale_inv):
        if not t.is_contiguous():
            raise ValueError("carrier arrays must be contiguous")
    if data.numel() != rows * cols or scale_inv.numel() * 32 != rows * cols:
        raise ValueError("carrier arrays do not match out's shape")
    prec = PRECISION[precision]
    if ws is None:
        ws = torch.empty(_LIB.ns_workspace_bytes(rows, cols, 1, prec), dtype=torch.uint8, device=out.device)
    a, b, c = coeffs
    _check(_LIB.ns_orthogonalize_mxfp8(_ptr(data), _ptr(scale_inv), _ptr(inv_norm), rows, cols, _ptr(out),
                                       _dtype(out), out.stride(0), steps, a, b, c, prec, _ptr(ws), ws.numel(),
                                       _stream(stream)))


def _matrix_args(x):
    if x.dim() == 2:
        rows, cols = x.shape
        if x.stride(1) != 1:
            raise ValueError("rows must be contiguous")
        return 1, rows, cols, x.stride(0), 0
    if x.dim() == 3:
        b, rows, cols = x.shape
        if x.stride(2) != 1:
            raise ValueError("rows must be contiguous")
        return b, rows, cols, x.stride(1), x.stride(0)
    raise ValueError("expected a 2-D matrix or a 3-D batch of matrices")


def ns_workspace_bytes(rows, cols, batch=1, precision="bf16"):
    return _LIB.ns_workspace_bytes(rows, cols, batch, PRECISION[precision])


def ns_orthogonalize(x, steps=5, coeffs=QUINTIC, eps=1e-7, inv_norm=None, precision="bf16",
                     ws=None, stream=None):
    """Overwrite x (rows x cols, or batch x rows x cols) with NS_T(x)."""
    batch, rows, cols, ld, bstride = _matrix_args(x)
    prec = PRECISION[precision]
    if ws is None:
        ws = torch.empty(_LIB.ns_workspace_bytes(rows, cols, batch, prec), dtype=torch.uint8,
                         device=x.device)
    a, b, c = coeffs
    _check(_LIB.ns_orthogonalize(_ptr(x), _dtype(x), rows, cols, ld, batch, bstride, steps, a, b, c,
                                 eps, _ptr(inv_norm), prec, _ptr(ws), ws.numel(), _stream(stream)))


def ns_orthogonalize_blocked(x, block_rows, block_cols, steps=5, coeffs=QUINTIC, eps=1e-7,
                             inv_norm=None, precision="bf16", ws=None, stream=None):
    """Overwrite every block_rows x block_cols block of x with its own NS."""
    _, rows, cols, ld, _ = _matrix_args(x)
    prec = PRECISION[precision]
    if ws is None:
        ws = torch.empty(_LIB.ns_blocked_workspace_bytes(rows, cols, block_rows, block_cols, prec),
                         dtype=torch.uint8, device=x.device)
    a, b, c = coeffs
    _check(_LIB.ns_orthogonalize_blocked(_ptr(x), _dtype(x), rows, cols, ld, block_rows, block_cols,
                                         steps, a, b, c, eps, _ptr(inv_norm), prec, _ptr(ws),
                                         ws.numel(), _stream(stream)))


def make_hparams(beta=0.95, eps=1e-7, coeffs=QUINTIC, lr_full=0.02, lr_block=0.01,
                 weight_decay=0.0, rms_scale=0.2, ns_steps=5, period=5, precision="bf16",
                 rounding="nearest", seed=0, carrier=False):
    a, b, c = coeffs
    return L.MuonHparams(beta, eps, a, b, c, lr_full, lr_block, weight_decay, rms_scale,
                         ns_steps, period, PRECISION[precision], ROUNDING[rounding], int(carrier), seed)


def _matrices(mats, device):
    """qm_muon_matrix array; each weight (optional) must be a contiguous fp32
    tensor of rows x cols elements on the plan's device."""
    arr = (L.MuonMatrix * len(mats))()
    for i, (rows, cols, br, bc, w) in enumerate(mats):
        if w is not None:
            _require(w, f"weight {i}", torch.float32, device, numel=rows * cols)
        arr[i] = L.MuonMatrix(rows, cols, br, bc, w.data_ptr() if w is not None else None)
    return arr


def muon_step_workspace_bytes(plan_full, plan_block, mats, precision="bf16", hparams=None):
    arr = _matrices(mats, plan_full.device)
    if hparams is not None:
        return _LIB.muon_step_workspace_bytes_ex(plan_full.hptr, plan_block.hptr if plan_block else None,
                                                 arr, len(mats), ctypes.byref(hparams))
    return _LIB.muon_step_workspace_bytes(plan_full.hptr, plan_block.hptr if plan_block else None,
                                          arr, len(mats), PRECISION[precision])


def muon_step(plan_full, plan_block, mats, step, hparams, ws=None, stream=None):
    """One block-periodic Muon step.  mats: list of (rows, cols, block_rows,
    block_cols, weight fp32 tensor or None), tensor i of both plans."""
    arr = _matrices(mats, plan_full.device)
    if ws is None:
        nbytes = _LIB.muon_step_workspace_bytes_ex(plan_full.hptr,
                                                   plan_block.hptr if plan_block else None,
                                                   arr, len(mats), ctypes.byref(hparams))
        ws = torch.empty(nbytes, dtype=torch.uint8, device=plan_full.device)
    _check(_LIB.muon_step(plan_full.hptr, plan_full.dptr,
                          plan_block.hptr if plan_block else None,
                          plan_block.dptr if plan_block else None,
                          arr, len(mats), step, ctypes.byref(hparams), _ptr(ws), ws.numel(),
                          _stream(stream)))


def muon_apply(plan, mats, full, inv_norm, hparams, ws, stream=None):
    """NS + weight apply for the plan's matrices given group inverse norms
    (device fp32 [plan.n_groups]); muon_step = update + this."""
    _require(inv_norm, "inv_norm", torch.float32, plan.device, numel=plan.n_groups)
    arr = _matrices(mats, plan.device)
    _check(_LIB.muon_apply(plan.hptr, arr, len(mats), int(full), _ptr(inv_norm),
                           ctypes.byref(hparams), _ptr(ws), ws.numel(), _stream(stream)))


def hbm_stream_copy(src, dst, stream=None):
    """Measurement aid: copy src into dst (same byte size, contiguous, 16-byte
    aligned) with the update kernels' access pattern."""
    for t in (src, dst):
        if not t.is_contiguous():
            raise ValueError("stream copy operands must be contiguous")
    n = src.numel() * src.element_size()
    if dst.numel() * dst.element_size() != n:
        raise ValueError("stream copy operands differ in size")
    _check(_LIB.qm_hbm_stream_copy(_ptr(src), _ptr(dst), n, _stream(stream)))


GRASP_GRID = 64


class GraspState:
    """Zero-initialised GRASP state buffers of one rows x cols matrix (the
    layout of qm_grasp_state)."""

    def __init__(self, rows, cols, rank, device="cuda"):
        nbr, nbc = -(-rows // GRASP_GRID), -(-cols // GRASP_GRID)
        z = lambda shape, dt: torch.zeros(shape, dtype=dt, device=device)
        self.rows, self.cols, self.rank = rows, cols, rank
        self.res_codes = z((rows, (cols + 1) // 2), torch.uint8)
        self.res_rmax = z((rows, nbc), torch.float32)
        self.res_cmax = z((nbr, cols), torch.float32)
        self.p_codes = z((rows, rank), torch.int8)
        self.p_rmax = z((rows,), torch.float32)
        self.p_cmax = z((nbr, rank), torch.float32)
        self.r_codes = z((cols, rank), torch.int8)
        self.r_rmax = z((cols,), torch.float32)
        self.r_cmax = z((nbc, rank), torch.float32)

    def c_struct(self):
        return L.GraspStateC(*(t.data_ptr() for t in (
            self.res_codes, self.res_rmax, self.res_cmax, self.p_codes, self.p_rmax, self.p_cmax,
            self.r_codes, self.r_rmax, self.r_cmax)))


def grasp_workspace_bytes(rows, cols, rank):
    return _LIB.grasp_workspace_bytes(rows, cols, rank)


def grasp_step(state, grad, warm, mu=0.95, ns_steps=5, coeffs=QUINTIC, eps=1e-7, weight=None,
               lr=0.02, weight_decay=0.0, ws=None, stream=None, ns_precision="f32"):
    """One GRASP step: state updated in place, grad (in: g) overwritten with
    O = NS(M_t), weight (optional) updated.  ns_precision: "f32" (fp32
    MFMAs) or "bf16x3" (fp32 operands, products from a bf16 hi + lo split)."""
    if grad.dim() != 2:
        raise ValueError("grad must be a 2-D matrix")
    rows, cols = grad.shape
    _require(grad, "grad", grad.dtype, grad.device)
    _dtype(grad)
    if (state.rows, state.cols) != (rows, cols):
        raise ValueError(f"state is {state.rows} x {state.cols}, grad {rows} x {cols}")
    _require(warm, "warm", torch.float32, grad.device, shape=(cols, state.rank))
    if weight is not None:
        _require(weight, "weight", torch.float32, grad.device, numel=rows * cols)
    if ws is None:
        ws = torch.empty(_LIB.grasp_workspace_bytes(rows, cols, state.rank), dtype=torch.uint8,
                         device=grad.device)
    a, b, c = coeffs
    st = state.c_struct()
    _check(_LIB.grasp_step(ctypes.byref(st), rows, cols, state.rank, GRASP_GRID, _ptr(grad),
                           _dtype(grad), _ptr(warm), mu, ns_steps, a, b, c, eps, PRECISION[ns_precision],
                           _ptr(weight), lr,
                           weight_decay, _ptr(ws), ws.numel(), _stream(stream)))


def _encode_list(encode, arr, n):
    """A list blob built by `encode`: (host bytes, their size)."""
    size = ctypes.c_size_t(0)
    _check(encode(arr, n, None, ctypes.byref(size)))
    host = torch.empty(size.value, dtype=torch.uint8)
    _check(encode(arr, n, ctypes.c_void_p(host.data_ptr()), ctypes.byref(size)))
    return host


def _grad_view(t, name):
    """(cols, ld) of a gradient: (0, 0) if contiguous, else those of a 2-D view."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.is_contiguous():
        return 0, 0
    if t.dim() != 2 or t.stride(1) != 1 or t.stride(0) < t.shape[1]:
        raise ValueError(f"{name}: a non-contiguous grad must be 2-D with unit column stride and rows that do not overlap")
    return t.shape[1], t.stride(0)


def _same_order(a, b):
    """Whether two shapes of one size number their elements alike: one merges
    dimensions of the other (a flat view, a matrix for a stack of matrices)."""
    def ends(shape):
        below, n = {1}, 1
        for d in reversed(shape):
            n *= d
            below.add(n)
        return below

    return ends(a) <= ends(b) or ends(b) <= ends(a)


def _plan_device(device, home):
    """The device of a list whose tensors are on `home`: that one; a device that
    is given has to name it."""
    if device is not None:
        given = torch.device(device)
        if given.type == "cuda" and given.index is None:
            given = torch.device("cuda", torch.cuda.current_device())
        if given != home:
            raise ValueError(f"a list is kept where its tensors are: on {home}, not on {given}")
    return home


class _ListPlan:
    """A tensor list encoded once and copied to the device once.  It holds the
    tensors' addresses (and keeps the tensors alive): a call works on the
    buffers that were there when the list was made."""

    def _finish(self, host, device, numels):
        self.host, self.device = host, device
        self.dev = host.to(device)
        # the queues that its memory is known to be used on (torch's allocator orders the one it was made on)
        self.queues = {torch._C._cuda_getCurrentRawStream(device.index)} if device.type == "cuda" else None
        self.only_device = device.type == "cuda" and torch.cuda.device_count() == 1
        self.hptr, self.dptr = ctypes.c_void_p(host.data_ptr()), ctypes.c_void_p(self.dev.data_ptr())
        self.numels = numels
        self.n_blocks = _LIB.qm_list_blocks(self.hptr)
        # index of each tensor's first 256-element block (list order)
        self.block_offsets, at = [], 0
        for n in numels:
            self.block_offsets.append(at)
            at += -(-n // BLOCK)


class GradPlan(_ListPlan):
    """The gradients of a model, for their global norm.

    grads: list of fp32 / bf16 / f16 device tensors, each contiguous or a 2-D
           view with unit column stride; none overlaps another.
           The list keeps their addresses, so they have to stay the buffers
           that backward writes: a gradient that is set to None (the default
           of torch's zero_grad) comes back elsewhere, and the list would go
           on with the old one.  Clear them in place
           (zero_grad(set_to_none=False)), or make a new list.
    device: the tensors' device, if given."""

    def __init__(self, grads, device=None):
        if not grads:
            raise ValueError("no grads")
        home = _plan_device(device, grads[0].device)
        arr = (L.GradTensor * len(grads))()
        for i, g in enumerate(grads):
            cols, ld = _grad_view(g, f"grad {i}")
            if g.device != home:
                raise ValueError(f"grad {i} is on {g.device}, expected {home}")
            arr[i] = L.GradTensor(g.data_ptr(), g.numel(), cols, ld, _dtype(g), 0)
        self._keep = list(grads)
        self._finish(_encode_list(_LIB.qm_grad_plan_encode, arr, len(grads)), home, [g.numel() for g in grads])

    def workspace_bytes(self):
        return _LIB.grad_norm_workspace_bytes(self.hptr)

    def workspace(self):
        return torch.empty(self.workspace_bytes(), dtype=torch.uint8, device=self.device)


def _launch(plan, stream, entry, *args):
    """entry(*args, queue) with the plan's device current (a launch on the
    default queue goes to the device that is).  queue: that of the given
    stream, or of torch's current one on the plan's device, as the raw handle
    (torch.cuda.current_stream() builds a Stream object, which costs as much
    as a launch)."""
    index = plan.device.index
    if stream is None:
        queue = torch._C._cuda_getCurrentRawStream(index)
    else:
        if stream.device != plan.device:
            raise ValueError(f"the stream is on {stream.device}, the list on {plan.device}")
        queue = stream.cuda_stream
    if plan.queues is not None and queue not in plan.queues:
        # freed while the call is pending, the list's device copy must not be given out again
        plan.dev.record_stream(stream if stream is not None else torch.cuda.current_stream(index))
        plan.queues.add(queue)
    if plan.only_device or torch._C._cuda_getDevice() == index:
        status = entry(*args, queue)
    else:
        with torch.cuda.device(index):
            status = entry(*args, queue)
    if status:
        raise QmuonError(status)


def _new(count, dtype, plan, stream):
    """A new tensor on the plan's device, in the pool of the stream that will
    write it (memory freed on another stream may still be in use there)."""
    if stream is None:
        return torch.empty(count, dtype=dtype, device=plan.device)
    with torch.cuda.stream(stream):
        return torch.empty(count, dtype=dtype, device=plan.device)


def _out(t, name, count, plan, stream):
    """t if it is a contiguous fp32 tensor of `count` elements, a new one for None."""
    if t is None:
        return _new(count, torch.float32, plan, stream)
    _require(t, name, torch.float32, plan.device, numel=count)
    return t


def grad_norm(plan, max_norm=float("inf"), eps=1e-6, norm=None, coef=None, ws=None, stream=None):
    """Norm of all gradients of the plan and min(1, max_norm / (norm + eps)),
    NaN where the norm is not finite, as device fp32 [1] tensors (given or
    new): (norm, coef)."""
    norm, coef = _out(norm, "norm", 1, plan, stream), _out(coef, "coef", 1, plan, stream)
    if ws is None:
        ws = _new(plan.workspace_bytes(), torch.uint8, plan, stream)
    elif not isinstance(ws, torch.Tensor) or ws.device != plan.device or not ws.is_contiguous():
        raise ValueError(f"ws must be a contiguous tensor on {plan.device}")
    _launch(plan, stream, _LIB.grad_norm, plan.hptr, plan.dptr, max_norm, eps, norm.data_ptr(), coef.data_ptr(),
            ws.data_ptr(), ws.nbytes)
    return norm, coef


def grad_scale(plan, coef, stream=None):
    """Every gradient of the plan times coef (device fp32 [1]) in place; a NaN
    coef leaves them as they are (and muon_step would read them as they are:
    test coef before it)."""
    _require(coef, "coef", torch.float32, plan.device, numel=1)
    _launch(plan, stream, _LIB.grad_scale, plan.hptr, plan.dptr, coef.data_ptr())


class AdamWState:
    """AdamW state of one tensor of `numel` elements, zero at the start.

    bits = 32: m, v fp32 [numel].  bits = 8: m int8 and v uint8 codes [numel],
    m_absmax and v_absmax fp32, one per 256 elements.  Buffers that are given
    are used as they are."""

    def __init__(self, numel, bits=32, device="cuda", m=None, v=None, m_absmax=None, v_absmax=None):
        if bits not in (8, 32):
            raise ValueError(f"states have 32 or 8 bits, not {bits}")
        if bits == 32 and (m_absmax is not None or v_absmax is not None):
            raise ValueError("32-bit states have no absmax")
        given = [t for t in (m, v, m_absmax, v_absmax) if t is not None]
        dev = given[0].device if given else torch.device(device)

        def take(t, name, count, dt):
            if t is None:
                return torch.zeros(count, dtype=dt, device=dev)
            _require(t, name, dt, dev, numel=count)
            return t

        self.numel, self.bits = numel, bits
        self.m = take(m, "m", numel, torch.float32 if bits == 32 else torch.int8)
        self.v = take(v, "v", numel, torch.float32 if bits == 32 else torch.uint8)
        self.m_absmax = self.v_absmax = None
        if bits == 8:
            self.m_absmax = take(m_absmax, "m_absmax", -(-numel // BLOCK), torch.float32)
            self.v_absmax = take(v_absmax, "v_absmax", -(-numel // BLOCK), torch.float32)

    def tensors(self):
        return [t for t in (self.m, self.v, self.m_absmax, self.v_absmax) if t is not None]


class AdamWPlan(_ListPlan):
    """The parameters an AdamW step covers.

    tensors: list of (weight, grad, state, copy, lr_scale, weight_decay):
             weight fp32 / bf16 / f16, contiguous; grad of any of these types,
             contiguous or a 2-D view with unit column stride; state an
             AdamWState; copy None, or a bf16 / f16 tensor that receives the
             new weight too; lr_scale a factor on the step's lr.  The shapes
             of weight, grad and copy are equal, or one merges dimensions of
             the other (a flat view).
             All of them, the state's buffers too, have to stay where they
             are, as the gradients of a GradPlan.
    device: the tensors' device, if given."""

    def __init__(self, tensors, device=None):
        if not tensors:
            raise ValueError("no tensors")
        home = _plan_device(device, tensors[0][0].device)
        arr = (L.AdamWTensor * len(tensors))()
        keep, numels = [], []
        for i, (weight, grad, state, copy, lr_scale, weight_decay) in enumerate(tensors):
            n = state.numel
            _require(weight, f"weight {i}", weight.dtype, home, numel=n)
            cols, ld = _grad_view(grad, f"grad {i}")
            if grad.numel() != n:
                raise ValueError(f"grad {i} has {grad.numel()} elements, expected {n}")
            if grad.device != home or state.m.device != home:
                raise ValueError(f"tensor {i}: grad and state must be on {home}")
            if copy is not None:
                _require(copy, f"copy {i}", copy.dtype, home, numel=n)
            for t, name in ((grad, "grad"), (copy, "copy")):
                if t is not None and t.shape != weight.shape and not _same_order(t.shape, weight.shape):
                    raise ValueError(f"{name} {i} has shape {tuple(t.shape)}, the weight {tuple(weight.shape)}")
            p = [t.data_ptr() if t is not None else None
                 for t in (weight, grad, state.m, state.v, state.m_absmax, state.v_absmax, copy)]
            arr[i] = L.AdamWTensor(*p, n, cols, ld, _dtype(weight), _dtype(grad),
                                   _dtype(copy) if copy is not None else 0, state.bits, lr_scale, weight_decay)
            keep += [weight, grad, copy, state]
            numels.append(n)
        self._keep = keep
        self._finish(_encode_list(_LIB.qm_adamw_plan_encode, arr, len(tensors)), home, numels)

    def view(self, flat, i):
        """Tensor i's elements of a [256 * n_blocks] buffer (adamw_read_state)."""
        e0 = self.block_offsets[i] * BLOCK
        return flat[e0:e0 + self.numels[i]]


def adamw_step(plan, step, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, grad_scale=None, rounding="nearest", seed=0,
               offset=None, stream=None):
    """One AdamW step (1-based `step`) over every tensor of the plan, in place.
    grad_scale: optional device fp32 [1] factor on the gradients (the coef of
    grad_norm); where it is NaN nothing is written.  rounding of 8-bit states:
    "nearest" or "stochastic" (random stream chosen by seed and offset, the
    step number if not given)."""
    if grad_scale is not None:
        _require(grad_scale, "grad_scale", torch.float32, plan.device, numel=1)
    hp = L.AdamWHparams(lr, betas[0], betas[1], eps, step, ROUNDING[rounding],
                        (step if offset is None else offset) & 0xFFFFFFFF, seed)
    _launch(plan, stream, _LIB.adamw_step, plan.hptr, plan.dptr, ctypes.byref(hp),
            grad_scale.data_ptr() if grad_scale is not None else None)


def adamw_read_state(plan, m=None, v=None, stream=None):
    """The values the states stand for: fp32 [256 * plan.n_blocks] tensors
    (given or new); plan.view(m, i) is tensor i's part.  Returns (m, v)."""
    n = plan.n_blocks * BLOCK
    m, v = _out(m, "m", n, plan, stream), _out(v, "v", n, plan, stream)
    _launch(plan, stream, _LIB.adamw_read_state, plan.hptr, plan.dptr, m.data_ptr(), v.data_ptr())
    return m, v
