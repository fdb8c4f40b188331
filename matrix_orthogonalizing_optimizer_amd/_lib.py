"""ctypes binding of libmuon (include/libmuon.h).  Argument marshalling only:
every step of the optimizer runs in the library's HIP kernels.  Torch
tensors are accepted for device memory (their data_ptr()) and the current
HIP stream; nothing here computes on them.

There is no fallback: if libmuon.so is missing or fails to load, every call
raises."""
from __future__ import annotations

import ctypes
import os
from typing import List, Optional, Sequence

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libmuon.so")

MUON_OK = 0
STATUS = {0: "MUON_OK", -1: "MUON_E_ARG", -2: "MUON_E_SHAPE", -3: "MUON_E_DTYPE",
          -4: "MUON_E_METHOD", -5: "MUON_E_WORKSPACE", -6: "MUON_E_HIP", -7: "MUON_E_PLAN",
          -8: "MUON_E_CAPACITY"}
MUON_NS_STANDARD, MUON_NS_GRAM, MUON_NS_AUTO, MUON_NS_GRAM_RESTART = 0, 1, 2, 3
MUON_F32, MUON_BF16 = 0, 1
MUON_KIND_MUON, MUON_KIND_ADAMW = 0, 1
MUON_SCALE_MOONLIGHT, MUON_SCALE_SPECTRAL, MUON_SCALE_UNIT_RMS = 0, 1, 2
MUON_COEFF_QUINTIC, MUON_COEFF_HYBRID = 0, 1
MUON_NORM_LAYER, MUON_NORM_RMS = 0, 1
MUON_LINEAR8_FORWARD, MUON_LINEAR8_WEIGHT_GRAD, MUON_LINEAR8_INPUT_GRAD = 0, 1, 2

EXPORTED = ["muon_plan_create", "muon_plan_destroy", "muon_plan_workspace_bytes",
            "muon_plan_buckets", "muon_plan_units", "muon_step", "ns_orthogonalize",
            "ns_orthogonalize_workspace_bytes", "muon_timing_enable", "muon_timing_collect",
            "muon_ns_coefficients", "muon_status_string", "muon_version", "muon_probe_mfma",
            "muon_probe_copy", "ns_orthogonalize_noalloc", "muon_probe_copy_lds",
            "muon_rows8_quantize", "muon_rows8_dequantize", "muon_norm_forward", "muon_norm_backward",
            "muon_norm_backward_workspace_bytes", "muon_linear8_forward", "muon_linear8_weight_grad",
            "muon_linear8_input_grad", "muon_linear8_workspace_bytes"]
NOALLOC_SCRATCH_BYTES = 64 << 20


class MuonError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} failed: {STATUS.get(status, status)} ({status})")


class MuonParamShape(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("dtype", ctypes.c_int32), ("rows", ctypes.c_int64),
                ("cols", ctypes.c_int64), ("split_rows", ctypes.c_int64), ("scale_dim", ctypes.c_int64)]


class MuonParamPtrs(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("grad", ctypes.c_void_p), ("momentum", ctypes.c_void_p),
                ("exp_avg", ctypes.c_void_p), ("exp_avg_sq", ctypes.c_void_p),
                ("update_out", ctypes.c_void_p)]


class MuonHparams(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_float), ("momentum", ctypes.c_float), ("weight_decay", ctypes.c_float),
                ("nesterov", ctypes.c_int32), ("ns_steps", ctypes.c_int32),
                ("coeffs", ctypes.POINTER(ctypes.c_float)), ("rms_scale", ctypes.c_float),
                ("adam_lr", ctypes.c_float), ("adam_beta1", ctypes.c_float),
                ("adam_beta2", ctypes.c_float), ("adam_eps", ctypes.c_float),
                ("adam_weight_decay", ctypes.c_float), ("adam_step", ctypes.c_int64),
                ("scale_mode", ctypes.c_int32), ("extra_scale", ctypes.c_float)]


class MuonPlanOptions(ctypes.Structure):
    _fields_ = [("ns_method", ctypes.c_int32), ("ns_dtype", ctypes.c_int32)]


class MuonKernelTiming(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char * 32), ("launches", ctypes.c_int64),
                ("total_ms", ctypes.c_double), ("flops", ctypes.c_double),
                ("bytes", ctypes.c_double)]


_lib = None


def lib():
    """Load libmuon.so from the package directory (raises if absent)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"libmuon.so not built at {LIB_PATH}; run "
                           "python -m matrix_orthogonalizing_optimizer_amd.build")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    L.muon_plan_create.argtypes = [ctypes.POINTER(MuonParamShape), i32, ctypes.POINTER(MuonPlanOptions),
                                   ctypes.POINTER(vp)]
    L.muon_plan_create.restype = i32
    L.muon_plan_destroy.argtypes = [vp]
    L.muon_plan_destroy.restype = None
    L.muon_plan_workspace_bytes.argtypes = [vp, ctypes.POINTER(sz)]
    L.muon_plan_workspace_bytes.restype = i32
    L.muon_plan_buckets.argtypes = [vp, ctypes.POINTER(i32), sz, ctypes.POINTER(sz)]
    L.muon_plan_buckets.restype = i32
    L.muon_plan_units.argtypes = [vp, ctypes.POINTER(i64), sz, ctypes.POINTER(sz)]
    L.muon_plan_units.restype = i32
    L.muon_step.argtypes = [vp, ctypes.POINTER(MuonParamPtrs), i32, ctypes.POINTER(MuonHparams), vp, sz, vp]
    L.muon_step.restype = i32
    L.ns_orthogonalize.argtypes = [vp, i64, i64, i64, i32, i32, ctypes.POINTER(ctypes.c_float), i32, vp,
                                   sz, vp]
    L.ns_orthogonalize.restype = i32
    L.ns_orthogonalize_noalloc.argtypes = [vp, i64, i64, i64, i32, i32, ctypes.POINTER(ctypes.c_float), i32,
                                           vp]
    L.ns_orthogonalize_noalloc.restype = i32
    L.ns_orthogonalize_workspace_bytes.argtypes = [i64, i64, i32, i32, ctypes.POINTER(sz)]
    L.ns_orthogonalize_workspace_bytes.restype = i32
    L.muon_timing_enable.argtypes = [i32]
    L.muon_timing_enable.restype = i32
    L.muon_timing_collect.argtypes = [ctypes.POINTER(MuonKernelTiming), i32, ctypes.POINTER(i32)]
    L.muon_timing_collect.restype = i32
    L.muon_probe_mfma.argtypes = [i32, i32, vp, ctypes.POINTER(ctypes.c_double), vp]
    L.muon_probe_mfma.restype = i32
    L.muon_probe_copy.argtypes = [vp, vp, ctypes.c_size_t, vp]
    L.muon_probe_copy.restype = i32
    L.muon_probe_copy_lds.argtypes = [vp, vp, ctypes.c_size_t, vp]
    L.muon_probe_copy_lds.restype = i32
    f32 = ctypes.c_float
    L.muon_rows8_quantize.argtypes = [vp, i64, i64, i64, i32, vp, i64, vp, vp]
    L.muon_rows8_dequantize.argtypes = [vp, i64, vp, i64, i64, vp, i64, i32, vp]
    L.muon_norm_forward.argtypes = [i32, vp, i64, i64, i64, i32, vp, vp, i32, f32, vp, i64, vp, i64, vp, vp, vp, vp]
    L.muon_norm_backward.argtypes = [i32, vp, i64, vp, i64, i64, i64, i32, vp, i32, vp, vp, vp, i64, vp, vp, i32,
                                     vp, sz, vp]
    L.muon_norm_backward_workspace_bytes.argtypes = [i64, i64, ctypes.POINTER(sz)]
    L.muon_linear8_forward.argtypes = [vp, i64, vp, vp, i64, vp, vp, i32, i64, i64, i64, vp, i64, i32, vp, sz, vp]
    L.muon_linear8_weight_grad.argtypes = [vp, i64, i32, vp, i64, vp, i64, i64, i64, vp, i64, i32, i32, vp, sz, vp]
    L.muon_linear8_input_grad.argtypes = [vp, i64, i32, vp, i64, vp, i64, i64, i64, vp, i64, i32, vp, sz, vp]
    L.muon_linear8_workspace_bytes.argtypes = [i32, i64, i64, i64, vp, i64, i32, ctypes.POINTER(sz)]
    for n in ("muon_rows8_quantize", "muon_rows8_dequantize", "muon_norm_forward", "muon_norm_backward",
              "muon_norm_backward_workspace_bytes", "muon_linear8_forward", "muon_linear8_weight_grad",
              "muon_linear8_input_grad", "muon_linear8_workspace_bytes"):
        getattr(L, n).restype = i32
    L.muon_ns_coefficients.argtypes = [i32, i32, ctypes.POINTER(ctypes.c_float), sz]
    L.muon_ns_coefficients.restype = i32
    L.muon_status_string.argtypes = [i32]
    L.muon_status_string.restype = ctypes.c_char_p
    L.muon_version.argtypes = []
    L.muon_version.restype = i32
    _lib = L
    return L


def _check(fn, st):
    if st != MUON_OK:
        raise MuonError(fn, st)


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _coeff_array(coeffs, steps):
    """Host array of steps x 3 floats for the library, or None (the quintic).
    ``coeffs``: one (a, b, c) triple (used at every step) or exactly ``steps``
    triples of finite numbers; anything else raises ValueError before the
    library reads 3 * steps floats from it."""
    if coeffs is None:
        return None
    import math
    if len(coeffs) == 3 and not hasattr(coeffs[0], "__len__"):
        coeffs = [coeffs] * int(steps)
    if len(coeffs) != steps:
        raise ValueError(f"coeffs: {len(coeffs)} rows for {steps} Newton-Schulz steps")
    flat = []
    for row in coeffs:
        if not hasattr(row, "__len__") or len(row) != 3:
            raise ValueError("coeffs: every row must be an (a, b, c) triple")
        vals = [float(x) for x in row]
        if not all(math.isfinite(v) for v in vals):
            raise ValueError("coeffs: non-finite coefficient")
        flat.extend(vals)
    return (ctypes.c_float * max(len(flat), 3))(*flat)


def _device_index(stream):
    """Index of the GPU the call's kernels run on: the stream's device, or
    the current device when the current stream is used."""
    import torch
    if stream is None or isinstance(stream, int):
        return torch.cuda.current_device()
    return stream.device.index


def _check_device(name, t, device_index):
    """A torch tensor handed to the library must live on the GPU the kernels
    run on: its data_ptr() is used as a device address there."""
    if t is None or isinstance(t, int) or not hasattr(t, "data_ptr"):
        return
    if not t.is_cuda:
        raise ValueError(f"{name}: a {t.device} tensor; the library needs device memory")
    if device_index is not None and t.device.index != device_index:
        raise ValueError(f"{name}: on {t.device}, the kernels run on cuda:{device_index}")


def _check_call_device(name, t, stream):
    """_check_device against the call's GPU, looked up only for device tensors."""
    if t is None or isinstance(t, int) or not hasattr(t, "data_ptr"):
        return
    _check_device(name, t, _device_index(stream) if t.is_cuda else None)


class Plan:
    """Owns a muon_plan handle (released on close / garbage collection)."""

    def __init__(self, handle: int, table):
        self.handle = handle
        self.table = list(table)

    def close(self):
        if self.handle:
            lib().muon_plan_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def muon_plan_create(table: Sequence[Sequence[int]], ns_method: int = MUON_NS_STANDARD,
                     ns_dtype: int = -1) -> Plan:
    """table rows: (kind, dtype, rows, cols, split_rows, scale_dim)."""
    n = len(table)
    arr = (MuonParamShape * max(n, 1))()
    for i, r in enumerate(table):
        arr[i] = MuonParamShape(*[int(x) for x in r])
    opts = MuonPlanOptions(int(ns_method), int(ns_dtype))
    h = ctypes.c_void_p()
    _check("muon_plan_create", lib().muon_plan_create(arr, n, ctypes.byref(opts), ctypes.byref(h)))
    return Plan(h.value, table)


def muon_plan_workspace_bytes(plan: Plan) -> int:
    b = ctypes.c_size_t()
    _check("muon_plan_workspace_bytes", lib().muon_plan_workspace_bytes(plan.handle, ctypes.byref(b)))
    return b.value


def muon_plan_buckets(plan: Plan) -> List[tuple]:
    """[(m, n, tall, param_dtype, compute_dtype, method, first_unit, count), ...]"""
    ln = ctypes.c_size_t()
    _check("muon_plan_buckets", lib().muon_plan_buckets(plan.handle, None, 0, ctypes.byref(ln)))
    buf = (ctypes.c_int32 * max(ln.value, 1))()
    _check("muon_plan_buckets", lib().muon_plan_buckets(plan.handle, buf, ln.value, ctypes.byref(ln)))
    return [tuple(buf[i:i + 8]) for i in range(0, ln.value, 8)]


def muon_plan_units(plan: Plan) -> List[tuple]:
    """[(param, row0, rows, cols, tall, scale_dim), ...] in bucket order."""
    ln = ctypes.c_size_t()
    _check("muon_plan_units", lib().muon_plan_units(plan.handle, None, 0, ctypes.byref(ln)))
    buf = (ctypes.c_int64 * max(ln.value, 1))()
    _check("muon_plan_units", lib().muon_plan_units(plan.handle, buf, ln.value, ctypes.byref(ln)))
    return [tuple(buf[i:i + 6]) for i in range(0, ln.value, 6)]


def make_hparams(lr=0.02, momentum=0.95, weight_decay=0.1, nesterov=True, ns_steps=5, coeffs=None,
                 rms_scale=0.2, adam_lr=3e-4, adam_beta1=0.9, adam_beta2=0.95, adam_eps=1e-8,
                 adam_weight_decay=0.1, adam_step=1, scale_mode=MUON_SCALE_MOONLIGHT, extra_scale=1.0):
    ca = _coeff_array(coeffs, ns_steps)
    hp = MuonHparams(lr, momentum, weight_decay, 1 if nesterov else 0, ns_steps,
                     ctypes.cast(ca, ctypes.POINTER(ctypes.c_float)) if ca is not None else None,
                     rms_scale, adam_lr, adam_beta1, adam_beta2, adam_eps, adam_weight_decay, adam_step,
                     scale_mode, extra_scale)
    hp._keep = ca  # keep the coefficient array alive with the struct
    return hp


def _check_buffer(name, t, rows, cols, dtype, device_index=None):
    """A torch tensor handed to muon_step must be the contiguous rows x cols
    device buffer of the table's dtype, on the GPU the kernels run on: the
    library addresses it from its pointer and the table alone.  Raw integer
    pointers and None pass unchecked (the library rejects a null pointer
    where one is required)."""
    if t is None or isinstance(t, int) or not hasattr(t, "data_ptr"):
        return
    import torch
    want = torch.float32 if dtype == MUON_F32 else torch.bfloat16
    if t.dtype != want:
        raise ValueError(f"{name}: dtype {t.dtype}, the table says {want}")
    if t.numel() != rows * cols or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous {rows} x {cols} tensor, got {tuple(t.shape)}")
    _check_device(name, t, device_index)


def muon_step(plan: Plan, params, grads, moms, exp_avgs, exp_avg_sqs, hp: MuonHparams, workspace,
              stream=None, update_outs=None) -> None:
    """One optimizer step; lists follow the plan's table order (None where a
    buffer does not apply).  workspace: a device tensor (or pointer) of at
    least muon_plan_workspace_bytes(plan) bytes."""
    n = len(plan.table)
    for name, lst in (("params", params), ("grads", grads), ("moms", moms), ("exp_avgs", exp_avgs),
                      ("exp_avg_sqs", exp_avg_sqs), ("update_outs", update_outs)):
        if lst is not None and len(lst) != n:
            raise ValueError(f"{name}: {len(lst)} entries for a table of {n}")
    tensors = [t for lst in (params, grads, moms, exp_avgs, exp_avg_sqs, update_outs or [], [workspace])
               for t in lst if t is not None and hasattr(t, "data_ptr")]
    di = None
    if tensors:
        if not all(t.is_cuda for t in tensors):
            bad = next(t for t in tensors if not t.is_cuda)
            raise ValueError(f"muon_step: a {bad.device} tensor; the library needs device memory")
        di = _device_index(stream)
    _check_device("workspace", workspace, di)
    for i, (kind, dt, rows, cols, _split, _sd) in enumerate(plan.table):
        _check_buffer(f"params[{i}]", params[i], rows, cols, dt, di)
        _check_buffer(f"grads[{i}]", grads[i], rows, cols, dt, di)
        if kind == MUON_KIND_MUON:
            _check_buffer(f"moms[{i}]", moms[i], rows, cols, MUON_F32, di)
            if update_outs is not None:
                _check_buffer(f"update_outs[{i}]", update_outs[i], rows, cols, MUON_F32, di)
        else:
            _check_buffer(f"exp_avgs[{i}]", exp_avgs[i], rows, cols, MUON_F32, di)
            _check_buffer(f"exp_avg_sqs[{i}]", exp_avg_sqs[i], rows, cols, MUON_F32, di)
    arr = (MuonParamPtrs * max(n, 1))()
    for i in range(n):
        arr[i] = MuonParamPtrs(_ptr(params[i]), _ptr(grads[i]), _ptr(moms[i]), _ptr(exp_avgs[i]),
                               _ptr(exp_avg_sqs[i]),
                               _ptr(update_outs[i]) if update_outs is not None else None)
    wsz = workspace.numel() * workspace.element_size() if hasattr(workspace, "numel") else 0
    if isinstance(workspace, tuple):
        workspace, wsz = workspace
    _check("muon_step", lib().muon_step(plan.handle, arr, n, ctypes.byref(hp), _ptr(workspace), wsz,
                                        _stream(stream)))


def ns_orthogonalize_workspace_bytes(rows: int, cols: int, dtype: int, method: int = MUON_NS_STANDARD) -> int:
    b = ctypes.c_size_t()
    _check("ns_orthogonalize_workspace_bytes",
           lib().ns_orthogonalize_workspace_bytes(rows, cols, dtype, method, ctypes.byref(b)))
    return b.value


def ns_orthogonalize(X, steps: int = 5, coeffs=None, method: int = MUON_NS_STANDARD, workspace=None,
                     stream=None, rows=None, cols=None, ld=None, dtype=None) -> None:
    """In place: X <- NewtonSchulz(X / ||X||_F).  X: a 2-D device tensor
    (fp32 or bf16, rows may be strided) or a raw pointer with rows/cols/ld/dtype."""
    ca = _coeff_array(coeffs, steps)
    if hasattr(X, "data_ptr"):
        import torch
        di = _device_index(stream) if X.is_cuda else None
        _check_device("X", X, di)
        if workspace is not None:
            _check_device("workspace", workspace, di)
        if X.dim() != 2 or X.stride(1) != 1:
            raise ValueError("X must be 2-D with unit column stride")
        rows, cols = X.shape
        ld = X.stride(0) if rows > 1 else cols
        dtype = MUON_F32 if X.dtype == torch.float32 else MUON_BF16
        if X.dtype not in (torch.float32, torch.bfloat16):
            raise ValueError("X must be float32 or bfloat16")
        if workspace is None:
            nb = ns_orthogonalize_workspace_bytes(rows, cols, dtype, method)
            workspace = torch.empty(max(nb, 1), dtype=torch.uint8, device=X.device)
    wsz = workspace.numel() * workspace.element_size() if hasattr(workspace, "numel") else 0
    if isinstance(workspace, tuple):
        workspace, wsz = workspace
    _check("ns_orthogonalize",
           lib().ns_orthogonalize(_ptr(X), rows, cols, ld, dtype, steps,
                                  ca, method, _ptr(workspace), wsz, _stream(stream)))


def ns_orthogonalize_noalloc(X, steps: int = 5, coeffs=None, method: int = MUON_NS_STANDARD,
                             stream=None) -> None:
    """ns_orthogonalize with the library's own device scratch array (no
    workspace; nothing is allocated).  X: a 2-D fp32 or bf16 device tensor
    with unit column stride."""
    import torch
    ca = _coeff_array(coeffs, steps)
    di = _device_index(stream) if X.is_cuda else None
    _check_device("X", X, di)
    if X.dim() != 2 or X.stride(1) != 1:
        raise ValueError("X must be 2-D with unit column stride")
    if X.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("X must be float32 or bfloat16")
    rows, cols = X.shape
    ld = X.stride(0) if rows > 1 else cols
    dtype = MUON_F32 if X.dtype == torch.float32 else MUON_BF16
    _check("ns_orthogonalize_noalloc",
           lib().ns_orthogonalize_noalloc(_ptr(X), rows, cols, ld, dtype, steps, ca, method,
                                          _stream(stream)))


def muon_timing_enable(enable: bool = True) -> None:
    _check("muon_timing_enable", lib().muon_timing_enable(1 if enable else 0))


def muon_timing_collect() -> dict:
    """{family: {"launches", "total_ms", "flops", "bytes"}} since the last collect."""
    cap = 32
    arr = (MuonKernelTiming * cap)()
    n = ctypes.c_int32()
    _check("muon_timing_collect", lib().muon_timing_collect(arr, cap, ctypes.byref(n)))
    return {arr[i].name.decode(): {"launches": arr[i].launches, "total_ms": arr[i].total_ms,
                                   "flops": arr[i].flops, "bytes": arr[i].bytes}
            for i in range(min(n.value, cap))}


def muon_probe_mfma(workgroups: int, iters: int, sink, stream=None) -> float:
    """Enqueue the register-only bf16 MFMA loop; returns its FLOPs.  sink:
    device tensor of at least `workgroups` float32."""
    _check_call_device("sink", sink, stream)
    if hasattr(sink, "numel") and sink.numel() * sink.element_size() < 4 * workgroups:
        raise ValueError("sink holds fewer than `workgroups` floats")
    flops = ctypes.c_double()
    _check("muon_probe_mfma", lib().muon_probe_mfma(workgroups, iters, _ptr(sink), ctypes.byref(flops),
                                                     _stream(stream)))
    return flops.value


def _check_copy_buffers(src, dst, nbytes, stream):
    for name, t in (("src", src), ("dst", dst)):
        _check_call_device(name, t, stream)
        if hasattr(t, "numel") and t.numel() * t.element_size() < nbytes:
            raise ValueError("buffer smaller than nbytes")


def muon_probe_copy(src, dst, nbytes: int, stream=None) -> None:
    """Enqueue the streaming copy of nbytes from src to dst (device tensors)."""
    _check_copy_buffers(src, dst, nbytes, stream)
    _check("muon_probe_copy", lib().muon_probe_copy(_ptr(src), _ptr(dst), nbytes, _stream(stream)))


def muon_probe_copy_lds(src, dst, nbytes: int, stream=None) -> None:
    """Enqueue the streaming copy through the GEMMs' global -> LDS load path."""
    _check_copy_buffers(src, dst, nbytes, stream)
    _check("muon_probe_copy_lds", lib().muon_probe_copy_lds(_ptr(src), _ptr(dst), nbytes, _stream(stream)))


def muon_status_string(status: int) -> str:
    return lib().muon_status_string(status).decode()


def muon_ns_coefficients(kind: int, steps: int):
    """steps x 3 Newton-Schulz coefficients of a schedule kind, as a list of
    (a, b, c) tuples."""
    buf = (ctypes.c_float * (3 * steps))() if steps > 0 else (ctypes.c_float * 3)()
    _check("muon_ns_coefficients", lib().muon_ns_coefficients(kind, steps, buf, 3 * max(steps, 0)))
    return [tuple(buf[3 * k:3 * k + 3]) for k in range(steps)]


def muon_version() -> int:
    return lib().muon_version()


# ---------------------------------------------------------------------------
# Operators around the step: norms, 8-bit rows, the linear layer on 8-bit rows

_codes = {}  # torch dtype -> code, filled on first use


def _dtype_code(name, t):
    if not _codes:
        import torch
        _codes.update({torch.bfloat16: MUON_BF16, torch.float32: MUON_F32})
    code = _codes.get(t.dtype)
    if code is None:
        raise ValueError(f"{name}: must be float32 or bfloat16, got {t.dtype}")
    return code


def _matrix(name, t):
    """(rows, cols, ld, dtype code) of a 2-D tensor with unit column stride."""
    if t.dim() != 2:
        raise ValueError(f"{name}: expected a 2-D tensor, got {tuple(t.shape)}")
    rows, cols = t.shape
    ld, unit = t.stride()
    if unit != 1 and cols > 1 and rows > 0:
        raise ValueError(f"{name}: columns must be contiguous")
    if rows <= 1:
        ld = cols
    elif ld < cols:
        raise ValueError(f"{name}: rows overlap (stride {ld} for {cols} columns)")
    return rows, cols, ld, _codes.get(t.dtype) if t.dtype in _codes else _dtype_code(name, t)


def _rows8(name, q, scale, shape=None):
    """(rows, cols, ldq, address) of 8-bit rows, their scales checked: int8,
    rows a multiple of 16 bytes apart, every row's bytes up to the next one in
    the storage."""
    import torch
    if q.dtype != torch.int8 or q.dim() != 2:
        raise ValueError(f"{name}: expected a 2-D int8 tensor, got {q.dtype} {tuple(q.shape)}")
    rows, cols = q.shape
    if shape is not None and (rows, cols) != shape:
        raise ValueError(f"{name}: expected {shape}, got {(rows, cols)}")
    ld, unit = q.stride()
    if unit != 1 and cols > 1 and rows > 0:
        raise ValueError(f"{name}: columns must be contiguous")
    ptr = q.data_ptr()
    if rows <= 1 or cols == 0:
        ld = (cols + 15) // 16 * 16
    if rows > 0 and cols > 0:
        if ld % 16 or ld < cols or ptr % 16:
            raise ValueError(f"{name}: rows must start 16-byte aligned and lie a multiple of 16 bytes apart")
        if ld != cols and q.untyped_storage().nbytes() - q.storage_offset() < rows * ld:
            raise ValueError(f"{name}: the storage ends before the last row's {ld} bytes")
    if scale.dtype != torch.float32 or scale.numel() != rows or not scale.is_contiguous() or scale.dim() != 1:
        _vector(f"scale of {name}", scale, rows, torch.float32)
    return rows, cols, ld, ptr


def _vector(name, t, n, dtype=None):
    if t.dim() != 1 or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous vector of {n}, got {tuple(t.shape)}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name}: must be {dtype}, got {t.dtype}")


def _call_device(stream, names, *tensors):
    """Every tensor of a call lives on the GPU its kernels run on; returns
    that GPU's index.  names: the tensors' names, for the errors."""
    di = tensors[0].get_device()
    for t in tensors:
        if t is not None and t.get_device() != di:
            break
    else:
        if di >= 0 and di == (_current_device() if stream is None else _device_index(stream)):
            return di
    di = None
    for name, t in zip(names.split(), tensors):
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError(f"{name}: a {t.device} tensor; the library needs device memory")
        if di is None:
            di = _device_index(stream)
        if t.get_device() != di:
            raise ValueError(f"{name}: on {t.device}, the kernels run on cuda:{di}")
    return di


def _current_device():
    """torch.cuda.current_device() for a process that has device tensors:
    torch's direct query (0.1 of 0.3 us) where this torch has it."""
    global _current_device
    import torch
    _current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    return _current_device()


def _empty(di, stream, *shape, dtype):
    """A buffer that belongs to the stream that uses it, so the allocator does
    not hand it on while the call's kernels still run."""
    import torch
    dev = torch.device("cuda", di)
    if stream is None:
        return torch.empty(*shape, dtype=dtype, device=dev)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=dev) if stream else torch.cuda.default_stream(dev)
    with torch.cuda.stream(stream):
        return torch.empty(*shape, dtype=dtype, device=dev)


def _empty_rows8(di, stream, rows, cols):
    import torch
    ld = (cols + 15) // 16 * 16
    q = _empty(di, stream, rows, ld, dtype=torch.int8)
    return q if ld == cols else q[:, :cols], _empty(di, stream, rows, dtype=torch.float32)


def _scratch(di, stream, workspace, nbytes):
    """(tensor kept alive, pointer, bytes) of a call's workspace."""
    import torch
    if workspace is None:
        if nbytes == 0:
            return None, None, 0
        workspace = _empty(di, stream, nbytes, dtype=torch.uint8)
    elif not workspace.is_contiguous():
        raise ValueError("workspace: must be contiguous")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


_raw_stream = None  # torch's query of a device's current stream handle


def _launch(fn, di, stream, *args):
    global _raw_stream
    f = getattr(_lib or lib(), fn)
    if stream is None:  # the current stream of the current device (_call_device)
        if _raw_stream is None:
            # torch's direct query where this torch has it (0.1 us; building a
            # Stream object for its handle takes 2.8 us)
            import torch
            _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
                lambda d: torch.cuda.current_stream(d).cuda_stream)
        st = f(*args, _raw_stream(di))
    else:
        import torch
        with torch.cuda.device(di):
            st = f(*args, _stream(stream))
    if st != MUON_OK:
        raise MuonError(fn, st)


def muon_rows8_quantize(x, q=None, scale=None, stream=None):
    """(q, scale): the 8-bit rows of x (2-D, fp32 or bf16, rows may be
    strided).  q: int8, x's shape, rows a multiple of 16 bytes apart (None:
    allocated so; the bytes of a row behind its columns up to the next multiple
    of 16 are set to zero, which the products rely on); scale: fp32, one per
    row, a power of two."""
    rows, cols, ldx, dt = _matrix("x", x)
    if (q is None) != (scale is None):
        raise ValueError("q and scale: give both or neither")
    di = _call_device(stream, "x q scale", x, q, scale)
    if q is None:
        q, scale = _empty_rows8(di, stream, rows, cols)
    _, _, ldq, qp = _rows8("q", q, scale, (rows, cols))
    _launch("muon_rows8_quantize", di, stream, x.data_ptr(), rows, cols, ldx, dt, qp, ldq, scale.data_ptr())
    return q, scale


def muon_rows8_dequantize(q, scale, out=None, dtype=None, stream=None):
    """The matrix that 8-bit rows stand for, q * scale per row, as ``out``
    (2-D, fp32 or bf16) or a new tensor of ``dtype`` (default bfloat16)."""
    import torch
    rows, cols, ldq, qp = _rows8("q", q, scale)
    di = _call_device(stream, "q scale out", q, scale, out)
    if out is None:
        out = _empty(di, stream, rows, cols, dtype=dtype or torch.bfloat16)
    r, c, ldy, dt = _matrix("out", out)
    if (r, c) != (rows, cols):
        raise ValueError(f"out: expected {(rows, cols)}, got {(r, c)}")
    _launch("muon_rows8_dequantize", di, stream, qp, ldq, scale.data_ptr(), rows, cols, out.data_ptr(), ldy, dt)
    return out


def muon_norm_forward(x, gamma, beta=None, eps=1e-5, kind=MUON_NORM_LAYER, y=None, q=None, scale=None, mean=None,
                      rstd=None, stream=None) -> None:
    """Layer norm (or RMS norm) of the rows of x into the buffers given, any
    of: y (x's dtype; may be x), q and scale (8-bit rows, see
    muon_rows8_quantize), mean and rstd (fp32, one per row, what
    muon_norm_backward takes; no mean for MUON_NORM_RMS)."""
    import torch
    rows, cols, ldx, dt = _matrix("x", x)
    _vector("gamma", gamma, cols)
    vdt = _dtype_code("gamma", gamma)
    if beta is not None:
        _vector("beta", beta, cols, gamma.dtype)
    ldy = ldq = 0
    qp = None
    if y is not None:
        r, c, ldy, ydt = _matrix("y", y)
        if (r, c) != (rows, cols) or ydt != dt:
            raise ValueError(f"y: expected {(rows, cols)} of {x.dtype}, got {(r, c)} of {y.dtype}")
    if (q is None) != (scale is None):
        raise ValueError("q and scale: give both or neither")
    if q is not None:
        _, _, ldq, qp = _rows8("q", q, scale, (rows, cols))
    for name, t in (("mean", mean), ("rstd", rstd)):
        if t is not None:
            _vector(name, t, rows, torch.float32)
    di = _call_device(stream, "x gamma beta y q scale mean rstd", x, gamma, beta, y, q, scale, mean, rstd)
    _launch("muon_norm_forward", di, stream, kind, x.data_ptr(), rows, cols, ldx, dt, gamma.data_ptr(), _ptr(beta), vdt,
            eps, _ptr(y), ldy, qp, ldq, _ptr(scale), _ptr(mean), _ptr(rstd))


def muon_norm_backward_workspace_bytes(rows: int, cols: int) -> int:
    b = ctypes.c_size_t()
    _check("muon_norm_backward_workspace_bytes",
           lib().muon_norm_backward_workspace_bytes(rows, cols, ctypes.byref(b)))
    return b.value


def muon_norm_backward(dy, x, gamma, mean, rstd, kind=MUON_NORM_LAYER, dx=None, dgamma=None, dbeta=None,
                       accumulate=False, workspace=None, stream=None):
    """Gradients of muon_norm_forward: writes dx (allocated if None, may be
    dy) and returns it; dgamma and dbeta (gamma's dtype) are written where
    given, or added to with accumulate.  mean: None for MUON_NORM_RMS."""
    import torch
    rows, cols, lddy, dt = _matrix("dy", dy)
    r, c, ldx, xdt = _matrix("x", x)
    if (r, c) != (rows, cols) or xdt != dt:
        raise ValueError(f"x: expected {(rows, cols)} of {dy.dtype}, got {(r, c)} of {x.dtype}")
    _vector("gamma", gamma, cols)
    vdt = _dtype_code("gamma", gamma)
    for name, t in (("mean", mean), ("rstd", rstd)):
        if t is not None:
            _vector(name, t, rows, torch.float32)
    for name, t in (("dgamma", dgamma), ("dbeta", dbeta)):
        if t is not None:
            _vector(name, t, cols, gamma.dtype)
    di = _call_device(stream, "dy x gamma mean rstd dx dgamma dbeta workspace", dy, x, gamma, mean, rstd, dx, dgamma,
                      dbeta, workspace)
    if dx is None:
        dx = _empty(di, stream, rows, cols, dtype=dy.dtype)
    r, c, lddx, ddt = _matrix("dx", dx)
    if (r, c) != (rows, cols) or ddt != dt:
        raise ValueError(f"dx: expected {(rows, cols)} of {dy.dtype}, got {(r, c)} of {dx.dtype}")
    nb = 0
    if workspace is None and (dgamma is not None or dbeta is not None):
        nb = muon_norm_backward_workspace_bytes(rows, cols)
    workspace, wp, wsz = _scratch(di, stream, workspace, nb)
    _launch("muon_norm_backward", di, stream, kind, dy.data_ptr(), lddy, x.data_ptr(), ldx, rows, cols, dt, gamma.data_ptr(), vdt,
            _ptr(mean), _ptr(rstd), dx.data_ptr(), lddx, _ptr(dgamma), _ptr(dbeta), 1 if accumulate else 0, wp, wsz)
    return dx


def muon_linear8_workspace_bytes(kind: int, tokens: int, out: int, in_: int, dy=None) -> int:
    """Workspace of one pass (MUON_LINEAR8_FORWARD, _WEIGHT_GRAD, _INPUT_GRAD);
    dy: the gradient call's tensor (for its dtype and alignment)."""
    b = ctypes.c_size_t()
    p, ld, dt = (0, 0, MUON_BF16) if dy is None else (dy.data_ptr(),) + _matrix("dy", dy)[2:]
    _check("muon_linear8_workspace_bytes",
           lib().muon_linear8_workspace_bytes(kind, tokens, out, in_, p, ld, dt, ctypes.byref(b)))
    return b.value


def muon_linear8_forward(q, scale, wq, wscale, bias=None, y=None, dtype=None, workspace=None, stream=None):
    """y = x W^T + bias on 8-bit rows: x as (q, scale) per token, W (out x in)
    as (wq, wscale) per output channel.  y: tokens x out, fp32 or bf16 (None:
    allocated, of ``dtype``, default bfloat16); returned."""
    import torch
    tokens, in_, ldq, qp = _rows8("q", q, scale)
    out, win, ldw, wqp = _rows8("wq", wq, wscale)
    if win != in_:
        raise ValueError(f"wq: expected {in_} columns, got {win}")
    bdt = 0
    if bias is not None:
        _vector("bias", bias, out)
        bdt = _dtype_code("bias", bias)
    di = _call_device(stream, "q scale wq wscale bias y workspace", q, scale, wq, wscale, bias, y, workspace)
    if y is None:
        y = _empty(di, stream, tokens, out, dtype=dtype or torch.bfloat16)
    r, c, ldy, dt = _matrix("y", y)
    if (r, c) != (tokens, out):
        raise ValueError(f"y: expected {(tokens, out)}, got {(r, c)}")
    # up to 16 tokens the library needs none (and would refuse the call if it did)
    nb = (0 if workspace is not None or tokens <= 16 else
          muon_linear8_workspace_bytes(MUON_LINEAR8_FORWARD, tokens, out, in_))
    workspace, wp, wsz = _scratch(di, stream, workspace, nb)
    _launch("muon_linear8_forward", di, stream, qp, ldq, scale.data_ptr(), wqp, ldw, wscale.data_ptr(), _ptr(bias), bdt,
            tokens, out, in_, y.data_ptr(), ldy, dt, wp, wsz)
    return y


def muon_linear8_weight_grad(dy, q, scale, dw=None, dtype=None, accumulate=False, workspace=None, stream=None):
    """dW = dy^T x (out x in) from the kept 8-bit rows (q, scale) of x: the
    gradient muon_step reads.  dw: written, or added to with accumulate
    (None: allocated, of ``dtype``, default dy's); returned."""
    tokens, out, lddy, dydt = _matrix("dy", dy)
    rows, in_, ldq, qp = _rows8("q", q, scale)
    if rows != tokens:
        raise ValueError(f"q: {rows} rows for {tokens} tokens")
    di = _call_device(stream, "dy q scale dw workspace", dy, q, scale, dw, workspace)
    if dw is None:
        if accumulate:
            raise ValueError("accumulate needs dw")
        dw = _empty(di, stream, out, in_, dtype=dtype or dy.dtype)
    r, c, lddw, dt = _matrix("dw", dw)
    if (r, c) != (out, in_):
        raise ValueError(f"dw: expected {(out, in_)}, got {(r, c)}")
    nb = 0 if workspace is not None else muon_linear8_workspace_bytes(MUON_LINEAR8_WEIGHT_GRAD, tokens, out, in_, dy)
    workspace, wp, wsz = _scratch(di, stream, workspace, nb)
    _launch("muon_linear8_weight_grad", di, stream, dy.data_ptr(), lddy, dydt, qp, ldq, scale.data_ptr(), tokens, out,
            in_, dw.data_ptr(), lddw, dt, 1 if accumulate else 0, wp, wsz)
    return dw


def muon_linear8_input_grad(dy, wq, wscale, dx=None, dtype=None, workspace=None, stream=None):
    """dX = dy W (tokens x in) with W as 8-bit rows (wq, wscale).  dx: None:
    allocated, of ``dtype``, default dy's; returned."""
    tokens, out, lddy, dydt = _matrix("dy", dy)
    rows, in_, ldw, wqp = _rows8("wq", wq, wscale)
    if rows != out:
        raise ValueError(f"wq: {rows} rows for {out} columns of dy")
    di = _call_device(stream, "dy wq wscale dx workspace", dy, wq, wscale, dx, workspace)
    if dx is None:
        dx = _empty(di, stream, tokens, in_, dtype=dtype or dy.dtype)
    r, c, lddx, dt = _matrix("dx", dx)
    if (r, c) != (tokens, in_):
        raise ValueError(f"dx: expected {(tokens, in_)}, got {(r, c)}")
    nb = 0 if workspace is not None else muon_linear8_workspace_bytes(MUON_LINEAR8_INPUT_GRAD, tokens, out, in_, dy)
    workspace, wp, wsz = _scratch(di, stream, workspace, nb)
    _launch("muon_linear8_input_grad", di, stream, dy.data_ptr(), lddy, dydt, wqp, ldw, wscale.data_ptr(), tokens, out,
            in_, dx.data_ptr(), lddx, dt, wp, wsz)
    return dx
