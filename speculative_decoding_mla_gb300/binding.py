"""Thin Python binding of the C ABI in include/verify_attn_mla.h.

Argument marshalling only: every step of the computation runs in the CUDA
library.  The functions keep the C names and take torch tensors for device
(and pinned host) buffers; `stream` defaults to torch's current stream.  A
status other than VMLA_OK raises VmlaError.  If libvmla.so is missing the
import of this module fails: there is no other implementation to fall back to.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libvmla.so")

VMLA_OK = 0
VMLA_ERR_NULL = -1
VMLA_ERR_SHAPE = -2
VMLA_ERR_ALIGN = -3
VMLA_ERR_WORKSPACE = -4
VMLA_ERR_CUDA = -5
VMLA_ERR_TIMEOUT = -6
VMLA_ERR_INDEX = -7
VMLA_ERR_DEVICE = -8
VMLA_ERR_PARENT = -9
VMLA_ERR_PARAM = -10
VMLA_ERR_FULL = -11
VMLA_KERNEL_TC = 0
VMLA_KERNEL_SIMT = 1
VMLA_SPLITS_LANES = -1  # splits value: the tensor-core planner takes its lane plan where it fits
D_QK = 576
D_V = 512
MAX_VOCAB = 262144
MAX_BLOCK_TOKENS = 128
MAX_SCALED_KV = 2 ** 31 - 512
MAX_BEAMS = 16
MAX_BEAM_KEEP = 32

EXPORTS = (
    "verify_attn_mla_plan", "verify_attn_mla_workspace_size", "verify_attn_mla", "verify_attn_mla_simt",
    "verify_attn_mla_merge", "verify_attn_mla_tree_mask", "verify_attn_mla_check",
    "verify_attn_mla_host_buffer_size", "verify_attn_mla_host", "verify_attn_mla_status_string",
    "verify_attn_mla_version", "verify_attn_mla_timing_enable", "verify_attn_mla_timing_read",
    "verify_attn_mla_simt_static", "verify_attn_mla_device_plan_workspace_size", "verify_attn_mla_device_plan",
    "verify_attn_mla_tree_accept", "verify_attn_mla_defrag", "verify_attn_mla_runs",
    "verify_attn_mla_runs_workspace_size", "verify_attn_mla_test_fault", "verify_attn_mla_fp8",
    "verify_attn_mla_simt_static_check", "verify_attn_mla_defrag_append",
    "verify_attn_mla_runs_device_plan_workspace_size", "verify_attn_mla_runs_device_plan",
    "verify_attn_mla_append", "verify_attn_mla_shared", "verify_attn_mla_shared_workspace_size",
    "verify_attn_mla_sample", "verify_attn_mla_append_scaled", "verify_attn_mla_scaled",
    "verify_attn_mla_scaled_workspace_size", "verify_attn_mla_step_tables", "verify_attn_mla_beam_select",
    "verify_attn_mla_beam_select_workspace_size", "verify_attn_mla_beam_reorder",
)


class VmlaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} ({status})")


class PlanInfo(ctypes.Structure):
    _fields_ = [("num_units", ctypes.c_int32), ("max_splits", ctypes.c_int32), ("partial_rows", ctypes.c_int64),
                ("merge_rows", ctypes.c_int64), ("workspace_bytes", ctypes.c_size_t), ("lane_width", ctypes.c_int32),
                ("lane_count", ctypes.c_int32)]


def _load(path: str = LIB_PATH):
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with speculative_decoding_mla_gb300.build.build()")
    L = ctypes.CDLL(path)
    vp, i32, i64, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
    run = [vp, vp, i64, vp, vp, vp, vp, vp, vp, vp, i32, i32, f32, i32, vp, vp, vp, sz, vp]
    sig = {
        "verify_attn_mla_plan": [i32, i32, i32, vp, vp, i32, i32, ctypes.POINTER(PlanInfo), vp],
        "verify_attn_mla_workspace_size": [i32, i32, vp, vp, i32, ctypes.POINTER(sz)],
        "verify_attn_mla": run,
        "verify_attn_mla_simt": run,
        "verify_attn_mla_merge": [vp, vp, i32, i64, vp, vp, vp],
        "verify_attn_mla_tree_mask": [vp, vp, i32, i32, vp, vp, vp],
        "verify_attn_mla_check": [vp, vp],
        "verify_attn_mla_host_buffer_size": [i32, i32, vp, vp, i32, i32, i32, ctypes.POINTER(sz)],
        "verify_attn_mla_host": [vp, vp, i64, vp, vp, vp, vp, vp, i32, i32, f32, i32, vp, vp, vp, sz, vp],
        "verify_attn_mla_status_string": [i32],
        "verify_attn_mla_version": [],
        "verify_attn_mla_timing_enable": [i32],
        "verify_attn_mla_timing_read": [vp, vp, vp, i32, ctypes.POINTER(i32)],
        "verify_attn_mla_simt_static": [vp, vp, i64, vp, vp, vp, vp, vp, vp, vp, i32, i32, f32, i32, vp, vp, vp],
        "verify_attn_mla_simt_static_check": [vp],
        "verify_attn_mla_device_plan_workspace_size": [i32, i32, i64, i64, i32, ctypes.POINTER(sz)],
        "verify_attn_mla_device_plan": [vp, vp, i64, vp, vp, vp, vp, vp, i32, i32, i64, i64, f32, i32, vp, vp, vp,
                                        sz, vp],
        "verify_attn_mla_runs_device_plan_workspace_size": [i32, i32, i64, i64, i32, ctypes.POINTER(sz)],
        "verify_attn_mla_runs_device_plan": [vp, vp, i64, vp, vp, vp, vp, vp, i32, i32, i64, i64, f32, i32, vp, vp,
                                             vp, sz, vp],
        "verify_attn_mla_tree_accept": [vp, vp, vp, vp, vp, i32, i32, vp, vp, vp, vp, vp],
        "verify_attn_mla_defrag": [vp, i64, vp, vp, vp, i32, vp, i64, vp, vp, vp],
        "verify_attn_mla_defrag_append": [vp, i64, vp, vp, vp, i32, vp, i64, vp, vp, i64, vp, vp],
        "verify_attn_mla_append": [vp, i64, vp, i64, vp, i64, i64, vp, vp, vp, i64, i32, i64, i32, vp, i64, f32, vp, vp,
                                   vp],
        "verify_attn_mla_shared": [vp, vp, i64, f32, vp, i64, vp, vp, vp, vp, vp, vp, vp, i32, i32, f32, i32, vp, vp, vp,
                                   sz, vp],
        "verify_attn_mla_shared_workspace_size": [i32, i32, i64, vp, vp, i32, ctypes.POINTER(sz)],
        "verify_attn_mla_sample": [vp, i32, i64, i64, i32, vp, vp, vp, vp, vp, vp, vp, vp],
        "verify_attn_mla_append_scaled": [vp, i64, vp, i64, vp, i64, i64, vp, vp, vp, i64, i32, i64, i32, vp, i64, vp,
                                          i32, vp, vp, vp],
        "verify_attn_mla_scaled": [vp, vp, i64, vp, i32, vp, vp, vp, vp, vp, i32, i32, i64, i64, f32, vp, vp, vp, sz, vp],
        "verify_attn_mla_scaled_workspace_size": [i32, i32, i64, i64, ctypes.POINTER(sz)],
        "verify_attn_mla_step_tables": [vp, vp, i32, i32, vp, i64, i64, vp, i64, vp, vp, vp, i64, i64, vp, vp, vp, vp, vp,
                                        vp, vp],
        "verify_attn_mla_beam_select": [vp, i32, i64, i64, i32, i32, i32, vp, vp, i32, vp, vp, vp, vp, sz, vp],
        "verify_attn_mla_beam_select_workspace_size": [i64, i32, i32, ctypes.POINTER(sz)],
        "verify_attn_mla_beam_reorder": [vp, i64, vp, i64, i64, i64, i32, i32, vp, vp, vp, vp, vp],
        "verify_attn_mla_runs": run,
        "verify_attn_mla_runs_workspace_size": [i32, i32, vp, vp, i32, ctypes.POINTER(sz)],
        "verify_attn_mla_test_fault": [i32, i64],
        "verify_attn_mla_fp8": [vp, vp, i64, f32, vp, vp, vp, vp, vp, vp, vp, i32, i32, f32, i32, vp, vp, vp, sz, vp],
    }
    for name, args in sig.items():
        f = getattr(L, name)
        f.argtypes = args
        f.restype = ctypes.c_char_p if name == "verify_attn_mla_status_string" else ctypes.c_int
    return L


_lib = _load()


def lib():
    return _lib


def status_string(status: int) -> str:
    return _lib.verify_attn_mla_status_string(int(status)).decode()


def _check(rc: int, where: str):
    if rc != VMLA_OK:
        raise VmlaError(rc, where)


def _arg(t, itemsize: int, name: str, on_device: bool) -> Optional[int]:
    """Pointer of an array argument after the checks the C ABI cannot make from a bare pointer:
    contiguous storage, the element size of the type the entry point reads (0: any) and device or
    host memory as the entry point expects.  Raises ValueError before any call."""
    if t is None:
        return None
    if isinstance(t, np.ndarray):
        if on_device:
            raise ValueError(f"{name}: device memory expected, got a numpy array")
        if not t.flags.c_contiguous:
            raise ValueError(f"{name}: not contiguous")
        if itemsize and t.itemsize != itemsize:
            raise ValueError(f"{name}: {itemsize}-byte elements expected, got {t.dtype}")
        return t.ctypes.data
    if not t.is_contiguous():
        raise ValueError(f"{name}: not contiguous")
    if itemsize and t.element_size() != itemsize:
        raise ValueError(f"{name}: {itemsize}-byte elements expected, got {t.dtype}")
    if bool(t.is_cuda) != on_device:
        raise ValueError(f"{name}: {'device' if on_device else 'host'} memory expected, got {t.device}")
    return t.data_ptr()


def _d(t, itemsize: int, name: str) -> Optional[int]:
    return _arg(t, itemsize, name, True)


def _h(t, itemsize: int, name: str) -> Optional[int]:
    return _arg(t, itemsize, name, False)


def _rows(t, itemsize: int, name: str, shape) -> int:
    """Pointer of a device array whose last dimension is contiguous and whose other strides the entry
    point takes as arguments.  shape: expected sizes (None: any)."""
    if isinstance(t, np.ndarray) or not t.is_cuda:
        raise ValueError(f"{name}: device memory expected")
    _shape(t, name, shape)
    if t.element_size() != itemsize:
        raise ValueError(f"{name}: {itemsize}-byte elements expected, got {t.dtype}")
    if t.numel() and t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: last dimension not contiguous")
    return t.data_ptr()


def _shape(t, name: str, shape):
    if len(t.shape) != len(shape) or any(w is not None and int(n) != int(w) for n, w in zip(t.shape, shape)):
        raise ValueError(f"{name}: shape {tuple(shape)} expected, got {tuple(t.shape)}")


def _same_device(**tensors):
    """Every given tensor lies on the current device, where the kernels are launched."""
    tensors = {name: t for name, t in tensors.items() if getattr(t, "is_cuda", False)}
    if not tensors:
        return  # host memory is refused where the pointers are taken
    import torch
    cur = torch.cuda.current_device()
    for name, t in tensors.items():
        if t.device.index != cur:
            raise ValueError(f"{name}: on {t.device}, but the current device is cuda:{cur}")


def _host_i32(a) -> np.ndarray:
    if hasattr(a, "cpu"):
        a = a.cpu().numpy()
    return np.ascontiguousarray(a, dtype=np.int32)


def _host_pair(batch_from, other, names):
    """Both host offset arrays; the call takes the batch from the first and reads as many entries of the second."""
    a, b = _host_i32(batch_from), _host_i32(other)
    if len(a) > len(b):
        raise ValueError(f"{names}: batch + 1 entries each expected, got {len(a)} and {len(b)}")
    return a, b


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def verify_attn_mla_plan(kernel: int, qo_indptr_host, kv_indptr_host, num_heads: int, splits: int = 0,
                         num_sms: int = 152):
    """Host-only split plan: (PlanInfo, splits per sequence)."""
    qo, kv = _host_pair(qo_indptr_host, kv_indptr_host, "qo_indptr_host, kv_indptr_host")
    B = len(qo) - 1
    info = PlanInfo()
    per = np.zeros(max(B, 1), dtype=np.int32)
    _check(_lib.verify_attn_mla_plan(kernel, B, num_heads, qo.ctypes.data, kv.ctypes.data, splits, num_sms,
                                     ctypes.byref(info), per.ctypes.data), "verify_attn_mla_plan")
    return info, per[:B]


def verify_attn_mla_workspace_size(qo_indptr_host, kv_indptr_host, num_heads: int, splits: int = 0) -> int:
    qo, kv = _host_pair(qo_indptr_host, kv_indptr_host, "qo_indptr_host, kv_indptr_host")
    n = ctypes.c_size_t(0)
    _check(_lib.verify_attn_mla_workspace_size(len(qo) - 1, num_heads, qo.ctypes.data, kv.ctypes.data, splits,
                                               ctypes.byref(n)), "verify_attn_mla_workspace_size")
    return int(n.value)


class Prepared:
    """One entry-point call whose arguments were checked and marshalled once.  Calling it repeats
    the C call on the same buffers: their contents (and the host indptr arrays' contents) may change
    between calls, their shapes and addresses may not.  It keeps a reference to every array it was
    built from.  Per call this saves the Python checks (about 20 us on the GPU host), which would
    otherwise delay the first kernel of a call made from an idle GPU."""

    __slots__ = ("_fn", "_name", "_args", "_keep")

    def __init__(self, fn, name: str, args, keep):
        self._fn = fn
        self._name = name
        self._args = tuple(t(v) for t, v in zip(fn.argtypes, args))
        self._keep = keep

    def __call__(self):
        rc = self._fn(*self._args)
        if rc != VMLA_OK:
            raise VmlaError(rc, self._name)


def _run_args(q, kv_pool, kv_indptr, kv_indices, qo_indptr, kv_indptr_host, qo_indptr_host, out, lse, workspace,
              sm_scale, draft_mask=None, parent=None, splits=0, stream=None, num_heads=None, pool_slots=None):
    kvh, qoh = _host_pair(kv_indptr_host, qo_indptr_host, "kv_indptr_host, qo_indptr_host")
    H = int(num_heads if num_heads is not None else q.shape[1])
    S = int(pool_slots if pool_slots is not None else kv_pool.shape[0])
    args = (_d(q, 2, "q"), _d(kv_pool, 2, "kv_pool"), S, _d(kv_indptr, 4, "kv_indptr"),
            _d(kv_indices, 4, "kv_indices"), _d(qo_indptr, 4, "qo_indptr"), _d(draft_mask, 8, "draft_mask"),
            _d(parent, 4, "parent"), kvh.ctypes.data, qoh.ctypes.data, len(kvh) - 1, H, float(sm_scale), int(splits),
            _d(out, 2, "out"), _d(lse, 4, "lse"), _d(workspace, 0, "workspace"),
            workspace.numel() * workspace.element_size(), _stream(stream))
    return args, (q, kv_pool, kv_indptr, kv_indices, qo_indptr, kvh, qoh, out, lse, workspace, draft_mask, parent)


def _run(fn, name, *a, **k):
    args, _ = _run_args(*a, **k)
    _check(fn(*args), name)


def prepare_verify_attn_mla(q, kv_pool, kv_indptr, kv_indices, qo_indptr, kv_indptr_host, qo_indptr_host, out, lse,
                            workspace, sm_scale, draft_mask=None, parent=None, splits=0, stream=None,
                            kernel: str = "tc") -> Prepared:
    """verify_attn_mla (kernel "tc") or verify_attn_mla_simt ("simt") with its arguments checked and
    marshalled once; call the result to run it."""
    name = "verify_attn_mla" if kernel == "tc" else "verify_attn_mla_simt"
    args, keep = _run_args(q, kv_pool, kv_indptr, kv_indices, qo_indptr, kv_indptr_host, qo_indptr_host, out, lse,
                           workspace, sm_scale, draft_mask, parent, splits, stream)
    return Prepared(getattr(_lib, name), name, args, keep)


def verify_attn_mla(q, kv_pool, kv_indptr, kv_indices, qo_indptr, kv_indptr_host, qo_indptr_host, out, lse,
                    workspace, sm_scale, draft_mask=None, parent=None, splits=0, stream=None):
    """Tensor-core verify attention into `out` [T,H,512] bf16 and `lse` [T,H] fp32."""
    _run(_lib.verify_attn_mla, "verify_attn_mla", q, kv_pool, kv_indptr, kv_indices, qo_indptr, kv_indptr_host,
         qo_indptr_host, out, lse, workspace, sm_scale, draft_mask, parent, splits, stream)


def _dplan_ws(fn, name, batch, num_heads, max_total_q, max_total_kv, splits):
    n = ctypes.c_size_t(0)
    _check(fn(int(batch), int(num_heads), int(max_total_q), int(max_total_kv), int(splits), ctypes.byref(n)), name)
    return int(n.value)


def verify_attn_mla_device_plan_workspace_size(batch: int, num_heads: int, max_total_q: int, max_total_kv: int,
                                               splits: int = 0) -> int:
    return _dplan_ws(_lib.verify_attn_mla_device_plan_workspace_size, "verify_attn_mla_device_plan_workspace_size",
                     batch, num_heads, max_total_q, max_total_kv, splits)


def verify_attn_mla_runs_device_plan_workspace_size(batch: int, num_heads: int, max_total_q: int, max_total_kv: int,
                                                    splits: int = 0) -> int:
    return _dplan_ws(_lib.verify_attn_mla_runs_device_plan_workspace_size,
                     "verify_attn_mla_runs_device_plan_workspace_size", batch, num_heads, max_total_q, max_total_kv,
                     splits)


def _dplan_call(fn, name, q, kv_pool, kv_indptr, rows, rows_name, qo_indptr, batch, max_total_q, max_total_kv, out,
                lse, workspace, sm_scale, draft_mask, parent, splits, stream, num_heads, pool_slots):
    H = int(num_heads if num_heads is not None else q.shape[1])
    S = int(pool_slots if pool_slots is not None else kv_pool.shape[0])
    rc = fn(_d(q, 2, "q"), _d(kv_pool, 2, "kv_pool"), S, _d(kv_indptr, 4, "kv_indptr"), _d(rows, 4, rows_name),
            _d(qo_indptr, 4, "qo_indptr"), _d(draft_mask, 8, "draft_mask"), _d(parent, 4, "parent"), int(batch), H,
            int(max_total_q), int(max_total_kv), float(sm_scale), int(splits), _d(out, 2, "out"), _d(lse, 4, "lse"),
            _d(workspace, 0, "workspace"), workspace.numel() * workspace.element_size(), _stream(stream))
    _check(rc, name)


def verify_attn_mla_device_plan(q, kv_pool, kv_indptr, kv_indices, qo_indptr, batch: int, max_total_q: int,
                                max_total_kv: int, out, lse, workspace, sm_scale, draft_mask=None, parent=None,
                                splits=0, stream=None, num_heads=None, pool_slots=None):
    """Stream-capture-safe verify attention: the plan is built on the device from the device indptr arrays."""
    _dplan_call(_lib.verify_attn_mla_device_plan, "verify_attn_mla_device_plan", q, kv_pool, kv_indptr, kv_indices,
                "kv_indices", qo_indptr, batch, max_total_q, max_total_kv, out, lse, workspace, sm_scale, draft_mask,
                parent, splits, stream, num_heads, pool_slots)


def verify_attn_mla_runs_device_plan(q, kv_pool, kv_indptr, run_base, qo_indptr, batch: int, max_total_q: int,
                                     max_total_kv: int, out, lse, workspace, sm_scale, draft_mask=None, parent=None,
                                     splits=0, stream=None, num_heads=None, pool_slots=None):
    """verify_attn_mla_runs with the plan built on the device (capture-safe; rows read from their pool runs)."""
    _dplan_call(_lib.verify_attn_mla_runs_device_plan, "verify_attn_mla_runs_device_plan", q, kv_pool, kv_indptr,
                run_base, "run_base", qo_indptr, batch, max_total_q, max_total_kv, out, lse, workspace, sm_scale,
                draft_mask, parent, splits, stream, num_heads, pool_slots)


def verify_attn_mla_defrag(src_pool, kv_indptr, kv_indices, kv_indptr_host, dst_pool, run_base, status_word=None,
                           stream=None):
    """Copies every sequence's rows into its run of dst_pool (runs start at run_base) and zeroes each run's tail."""
    kvh = _host_i32(kv_indptr_host)
    rc = _lib.verify_attn_mla_defrag(_d(src_pool, 2, "src_pool"), int(src_pool.shape[0]),
                                     _d(kv_indptr, 4, "kv_indptr"), _d(kv_indices, 4, "kv_indices"),
                                     kvh.ctypes.data, len(kvh) - 1, _d(dst_pool, 2, "dst_pool"),
                                     int(dst_pool.shape[0]), _d(run_base, 4, "run_base"),
                                     _d(status_word, 4, "status_word"), _stream(stream))
    _check(rc, "verify_attn_mla_defrag")


def _append_args(src_pool, kv_indptr, kv_indices, kv_indptr_host, dst_pool, run_base, first_row, status_word=None,
                 stream=None, max_new_rows=0):
    kvh = _host_i32(kv_indptr_host)
    args = (_d(src_pool, 2, "src_pool"), int(src_pool.shape[0]), _d(kv_indptr, 4, "kv_indptr"),
            _d(kv_indices, 4, "kv_indices"), kvh.ctypes.data, len(kvh) - 1, _d(dst_pool, 2, "dst_pool"),
            int(dst_pool.shape[0]), _d(run_base, 4, "run_base"), _d(first_row, 4, "first_row"), int(max_new_rows),
            _d(status_word, 4, "status_word"), _stream(stream))
    return args, (src_pool, kv_indptr, kv_indices, kvh, dst_pool, run_base, first_row, status_word)


def verify_attn_mla_defrag_append(src_pool, kv_indptr, kv_indices, kv_indptr_host, dst_pool, run_base, first_row,
                                  status_word=None, stream=None, max_new_rows=0):
    """The defragmentation for a decode loop: rows below first_row[b] are already in sequence b's run
    (max_new_rows: a bound on the new rows per sequence, or 0)."""
    args, _ = _append_args(src_pool, kv_indptr, kv_indices, kv_indptr_host, dst_pool, run_base, first_row,
                           status_word, stream, max_new_rows)
    _check(_lib.verify_attn_mla_defrag_append(*args), "verify_attn_mla_defrag_append")


def prepare_verify_attn_mla_defrag_append(*a, **k) -> Prepared:
    """verify_attn_mla_defrag_append with its arguments checked and marshalled once."""
    args, keep = _append_args(*a, **k)
    return Prepared(_lib.verify_attn_mla_defrag_append, "verify_attn_mla_defrag_append", args, keep)


def _step(t, dim: int, least: int) -> int:
    """Stride of a dimension, or `least` where its size makes the stride immaterial."""
    return int(t.stride(dim)) if int(t.shape[dim]) > 1 else least


def _cache_append_args(latent, k_rope, positions, slots, cos_sin, kv_pool, q_rope=None, q=None, kv_scale=0.0,
                       interleaved=True, status_word=None, stream=None, pool_args=None):
    T = int(latent.shape[0])
    R = D_QK - D_V
    fp8 = float(kv_scale) != 0.0 or pool_args is not None
    if (q_rope is None) != (q is None):
        raise ValueError("q_rope and q are given together")
    H = int(q.shape[1]) if q is not None else 0
    lat = _rows(latent, 2, "latent", (T, D_V))
    rope = _rows(k_rope, 2, "k_rope", (T, R))
    qr = _rows(q_rope, 2, "q_rope", (T, H, R)) if q is not None else None
    if q is not None:
        _shape(q, "q", (T, H, D_QK))
    _shape(positions, "positions", (T,))
    _shape(slots, "slots", (T,))
    _shape(cos_sin, "cos_sin", (None, R))
    _shape(kv_pool, "kv_pool", (None, D_QK))
    if status_word is not None and status_word.numel() < 2:
        raise ValueError("status_word: two words expected")
    _same_device(latent=latent, k_rope=k_rope, positions=positions, slots=slots, cos_sin=cos_sin, kv_pool=kv_pool,
                 q_rope=q_rope, q=q, status_word=status_word)
    args = (lat, _step(latent, 0, D_V), rope, _step(k_rope, 0, R), qr, _step(q_rope, 0, R) if H else 0,
            _step(q_rope, 1, R) if H else 0, _d(positions, 4, "positions"), _d(slots, 4, "slots"),
            _d(cos_sin, 4, "cos_sin"), int(cos_sin.shape[0]), int(bool(interleaved)), T, H,
            _d(kv_pool, 1 if fp8 else 2, "kv_pool"), int(kv_pool.shape[0]),
            *(pool_args or (float(kv_scale),)), _d(q, 2, "q"), _d(status_word, 4, "status_word"), _stream(stream))
    return args, (latent, k_rope, positions, slots, cos_sin, kv_pool, q_rope, q, status_word)


def verify_attn_mla_append(*a, **k):
    """Writes new tokens' rows into the pool (bf16, or e4m3 codes with kv_scale > 0), the last 64 columns turned by
    the tokens' positions, and with q_rope / q the queries' last 64 columns likewise.  latent [T, 512], k_rope
    [T, 64], q_rope [T, H, 64] may be strided; interleaved: pairs (2i, 2i + 1), else (i, i + 32); slot -1: padding."""
    args, _ = _cache_append_args(*a, **k)
    _check(_lib.verify_attn_mla_append(*args), "verify_attn_mla_append")


def prepare_verify_attn_mla_append(*a, **k) -> Prepared:
    """verify_attn_mla_append with its arguments checked and marshalled once."""
    args, keep = _cache_append_args(*a, **k)
    return Prepared(_lib.verify_attn_mla_append, "verify_attn_mla_append", args, keep)


def _append_scaled_args(latent, k_rope, positions, slots, cos_sin, kv_pool, kv_scales, block_tokens=1, q_rope=None,
                        q=None, interleaved=True, status_word=None, stream=None):
    _scales(kv_pool, kv_scales, block_tokens)
    args, keep = _cache_append_args(latent, k_rope, positions, slots, cos_sin, kv_pool, q_rope, q, 0.0, interleaved,
                                    status_word, stream, (_d(kv_scales, 4, "kv_scales"), int(block_tokens)))
    return args, (*keep, kv_scales)


def _scales(kv_pool, kv_scales, block_tokens):
    """A pool of e4m3 codes and its scales, one per block of slots."""
    _shape(kv_pool, "kv_pool", (None, D_QK))
    if int(block_tokens) < 1 or int(kv_pool.shape[0]) % int(block_tokens):
        raise ValueError(f"block_tokens: {block_tokens} does not divide the pool's {int(kv_pool.shape[0])} slots")
    _shape(kv_scales, "kv_scales", (int(kv_pool.shape[0]) // int(block_tokens),))
    if not str(kv_scales.dtype).endswith("float32"):
        raise ValueError(f"kv_scales: float32 expected, got {kv_scales.dtype}")
    _same_device(kv_scales=kv_scales)


def verify_attn_mla_append_scaled(*a, **k):
    """Writes new tokens' rows as e4m3 codes into a pool with one fp32 scale (a power of two) per block of
    block_tokens slots, setting or raising the blocks' scales; rotation, queries and padding as in
    verify_attn_mla_append.  Tokens of one block stand together, slots ascending."""
    args, _ = _append_scaled_args(*a, **k)
    _check(_lib.verify_attn_mla_append_scaled(*args), "verify_attn_mla_append_scaled")


def prepare_verify_attn_mla_append_scaled(*a, **k) -> Prepared:
    """verify_attn_mla_append_scaled with its arguments checked and marshalled once."""
    args, keep = _append_scaled_args(*a, **k)
    return Prepared(_lib.verify_attn_mla_append_scaled, "verify_attn_mla_append_scaled", args, keep)


def verify_attn_mla_scaled_workspace_size(batch: int, num_heads: int, max_total_q: int, max_total_kv: int) -> int:
    n = ctypes.c_size_t(0)
    _check(_lib.verify_attn_mla_scaled_workspace_size(int(batch), int(num_heads), int(max_total_q), int(max_total_kv),
                                                      ctypes.byref(n)), "verify_attn_mla_scaled_workspace_size")
    return int(n.value)


def _scaled_args(q, kv_pool, kv_scales, kv_indptr, kv_indices, qo_indptr, out, lse, workspace, sm_scale,
                 block_tokens=1, draft_mask=None, parent=None, stream=None):
    if len(q.shape) != 3:
        raise ValueError(f"q: three dimensions expected, got {tuple(q.shape)}")
    T, H, N, B = int(q.shape[0]), int(q.shape[1]), int(kv_indices.shape[0]), int(kv_indptr.shape[0]) - 1
    _scales(kv_pool, kv_scales, block_tokens)
    for t, name, shape in ((q, "q", (T, H, D_QK)), (out, "out", (T, H, D_V)), (lse, "lse", (T, H)),
                           (kv_indices, "kv_indices", (N,)), (kv_indptr, "kv_indptr", (None,)),
                           (qo_indptr, "qo_indptr", (B + 1,))):
        _shape(t, name, shape)
    if B < 0:
        raise ValueError("kv_indptr: batch + 1 entries expected")
    for t, name in ((draft_mask, "draft_mask"), (parent, "parent")):
        if t is not None:
            _shape(t, name, (T,))
    _same_device(q=q, kv_pool=kv_pool, kv_indptr=kv_indptr, kv_indices=kv_indices, qo_indptr=qo_indptr, out=out, lse=lse,
                 workspace=workspace, draft_mask=draft_mask, parent=parent)
    args = (_d(q, 2, "q"), _d(kv_pool, 1, "kv_pool"), int(kv_pool.shape[0]), _d(kv_scales, 4, "kv_scales"),
            int(block_tokens), _d(kv_indptr, 4, "kv_indptr"), _d(kv_indices, 4, "kv_indices"),
            _d(qo_indptr, 4, "qo_indptr"), _d(draft_mask, 8, "draft_mask"), _d(parent, 4, "parent"), B, H, T, N,
            float(sm_scale), _d(out, 2, "out"), _d(lse, 4, "lse"), _d(workspace, 0, "workspace"),
            workspace.numel() * workspace.element_size(), _stream(stream))
    return args, (q, kv_pool, kv_scales, kv_indptr, kv_indices, qo_indptr, out, lse, workspace, draft_mask, parent)


def verify_attn_mla_scaled(*a, **k):
    """Attention over a pool of e4m3 codes with one scale per block of block_tokens slots: single tokens, drafts or
    trees.  The lengths are read on the device; q [T, heads, 576], out, lse and kv_indices may have room for more
    rows than qo_indptr and kv_indptr use."""
    args, _ = _scaled_args(*a, **k)
    _check(_lib.verify_attn_mla_scaled(*args), "verify_attn_mla_scaled")


def prepare_verify_attn_mla_scaled(*a, **k) -> Prepared:
    """verify_attn_mla_scaled with its arguments checked and marshalled once."""
    args, keep = _scaled_args(*a, **k)
    return Prepared(_lib.verify_attn_mla_scaled, "verify_attn_mla_scaled", args, keep)


def _tables_args(cached, added, block_table, free_blocks, free_count, free_left, scratch, kv_indptr, qo_indptr,
                 kv_indices, positions, slots, block_tokens=1, status_word=None, stream=None):
    B, N, T = int(cached.shape[0]), int(kv_indices.shape[0]), int(slots.shape[0])
    for t, name, shape in ((cached, "cached", (None,)), (added, "added", (B,)), (block_table, "block_table", (B, None)),
                           (free_blocks, "free_blocks", (None,)), (free_count, "free_count", (1,)),
                           (free_left, "free_left", (1,)), (scratch, "scratch", (1,)), (kv_indptr, "kv_indptr", (B + 1,)),
                           (qo_indptr, "qo_indptr", (B + 1,)), (kv_indices, "kv_indices", (None,)),
                           (positions, "positions", (T,)), (slots, "slots", (None,))):
        _shape(t, name, shape)
    if status_word is not None and status_word.numel() < 2:
        raise ValueError("status_word: two words expected")
    _same_device(cached=cached, added=added, block_table=block_table, free_blocks=free_blocks, free_count=free_count,
                 free_left=free_left, scratch=scratch, kv_indptr=kv_indptr, qo_indptr=qo_indptr, kv_indices=kv_indices,
                 positions=positions, slots=slots, status_word=status_word)
    width = int(block_table.shape[1])
    args = (_d(cached, 4, "cached"), _d(added, 4, "added"), B, int(block_tokens),
            _rows(block_table, 4, "block_table", (B, width)), _step(block_table, 0, width), width,
            _d(free_blocks, 4, "free_blocks"), int(free_blocks.shape[0]), _d(free_count, 4, "free_count"),
            _d(free_left, 4, "free_left"), _d(scratch, 4, "scratch"), T, N, _d(kv_indptr, 4, "kv_indptr"),
            _d(qo_indptr, 4, "qo_indptr"), _d(kv_indices, 4, "kv_indices"), _d(positions, 4, "positions"),
            _d(slots, 4, "slots"), _d(status_word, 4, "status_word"), _stream(stream))
    return args, (cached, added, block_table, free_blocks, free_count, free_left, scratch, kv_indptr, qo_indptr,
                  kv_indices, positions, slots, status_word)


def verify_attn_mla_step_tables(*a, **k):
    """kv_indptr, qo_indptr, kv_indices, positions and slots of a step from the requests' cached and added lengths
    (int32 device arrays), growing block_table [batch, width] by blocks from the free list's end."""
    args, _ = _tables_args(*a, **k)
    _check(_lib.verify_attn_mla_step_tables(*args), "verify_attn_mla_step_tables")


def prepare_verify_attn_mla_step_tables(*a, **k) -> Prepared:
    """verify_attn_mla_step_tables with its arguments checked and marshalled once."""
    args, keep = _tables_args(*a, **k)
    return Prepared(_lib.verify_attn_mla_step_tables, "verify_attn_mla_step_tables", args, keep)


def verify_attn_mla_beam_select_workspace_size(rows: int, vocab: int, keep: int) -> int:
    n = ctypes.c_size_t(0)
    _check(_lib.verify_attn_mla_beam_select_workspace_size(int(rows), int(vocab), int(keep), ctypes.byref(n)),
           "verify_attn_mla_beam_select_workspace_size")
    return int(n.value)


def _beam_select_args(logits, score, parent, token, new_score, workspace, beams, finished=None, pad_token=0, stream=None):
    if len(logits.shape) != 2:
        raise ValueError(f"logits: two dimensions expected, got {tuple(logits.shape)}")
    rows, V = (int(n) for n in logits.shape)
    size = 0 if isinstance(logits, np.ndarray) else logits.element_size()
    if size not in (2, 4) or not str(logits.dtype).endswith(("bfloat16", "float32")):
        raise ValueError(f"logits: device memory of bfloat16 or float32 expected, got {logits.dtype}")
    if int(beams) < 1 or rows % int(beams):
        raise ValueError(f"beams: {beams} does not divide the {rows} rows of logits")
    R = rows // int(beams)
    _shape(parent, "parent", (R, None))
    K = int(parent.shape[1])
    for t, name, shape in ((score, "score", (rows,)), (token, "token", (R, K)), (new_score, "new_score", (R, K)),
                           (finished, "finished", (rows,))):
        if t is not None:
            _shape(t, name, shape)
    _same_device(logits=logits, score=score, finished=finished, parent=parent, token=token, new_score=new_score,
                 workspace=workspace)
    args = (_rows(logits, size, "logits", (rows, V)), int(size == 4), _step(logits, 0, V), R, int(beams), K, V,
            _d(score, 4, "score"), _d(finished, 4, "finished"), int(pad_token), _d(parent, 4, "parent"),
            _d(token, 4, "token"), _d(new_score, 4, "new_score"), _d(workspace, 0, "workspace"),
            workspace.numel() * workspace.element_size(), _stream(stream))
    return args, (logits, score, finished, parent, token, new_score, workspace)


def verify_attn_mla_beam_select(*a, **k):
    """The best parent.shape[1] continuations per request over `beams` beams and the vocabulary: logits [requests x
    beams, vocab] bf16 or fp32 (rows may be strided) and scores in, parent, token and new_score [requests, keep] out."""
    args, _ = _beam_select_args(*a, **k)
    _check(_lib.verify_attn_mla_beam_select(*args), "verify_attn_mla_beam_select")


def prepare_verify_attn_mla_beam_select(*a, **k) -> Prepared:
    """verify_attn_mla_beam_select with its arguments checked and marshalled once."""
    args, keep = _beam_select_args(*a, **k)
    return Prepared(_lib.verify_attn_mla_beam_select, "verify_attn_mla_beam_select", args, keep)


def _beam_reorder_args(src, dst, parent, beams, length=None, new_length=None, status_word=None, stream=None):
    if len(src.shape) != 2 or len(parent.shape) != 2:
        raise ValueError("src, parent: two dimensions expected")
    R, K = (int(n) for n in parent.shape)
    _shape(src, "src", (R * int(beams), None))
    _shape(dst, "dst", (R * K, int(src.shape[1])))
    for t, name, shape in ((length, "length", (R * int(beams),)), (new_length, "new_length", (R * K,))):
        if t is not None:
            _shape(t, name, shape)
    if status_word is not None and status_word.numel() < 2:
        raise ValueError("status_word: two words expected")
    _same_device(src=src, dst=dst, parent=parent, length=length, new_length=new_length, status_word=status_word)
    size, to = (t.element_size() if getattr(t, "is_cuda", False) else 0 for t in (src, dst))
    if size not in (2, 4, 8) or to != size:
        raise ValueError("src, dst: device memory of the same type, of 2, 4 or 8 bytes, expected")
    words = int(src.shape[1]) * size
    steps = [_step(src, 0, int(src.shape[1])) * size, _step(dst, 0, int(dst.shape[1])) * size]
    if words % 4 or any(s % 4 for s in steps):
        raise ValueError("src, dst: rows and strides of whole 32-bit words expected")
    if length is not None and size != 4:
        raise ValueError("length: counts 32-bit words, so rows of 4-byte elements are expected with it")
    args = (_rows(src, size, "src", tuple(src.shape)), steps[0] // 4, _rows(dst, size, "dst", tuple(dst.shape)),
            steps[1] // 4, words // 4, R, int(beams), K, _d(parent, 4, "parent"), _d(length, 4, "length"),
            _d(new_length, 4, "new_length"), _d(status_word, 4, "status_word"), _stream(stream))
    return args, (src, dst, parent, length, new_length, status_word)


def verify_attn_mla_beam_reorder(*a, **k):
    """Row r keep + k of dst gets row r beams + parent[r, k] of src (rows of 32-bit words, `length` of each)."""
    args, _ = _beam_reorder_args(*a, **k)
    _check(_lib.verify_attn_mla_beam_reorder(*args), "verify_attn_mla_beam_reorder")


def prepare_verify_attn_mla_beam_reorder(*a, **k) -> Prepared:
    """verify_attn_mla_beam_reorder with its arguments checked and marshalled once."""
    args, keep = _beam_reorder_args(*a, **k)
    return Prepared(_lib.verify_attn_mla_beam_reorder, "verify_attn_mla_beam_reorder", args, keep)


def verify_attn_mla_shared_workspace_size(shared_rows: int, qo_indptr_host, kv_indptr_host, num_heads: int,
                                          splits: int = 0) -> int:
    qo, kv = _host_pair(qo_indptr_host, kv_indptr_host, "qo_indptr_host, kv_indptr_host")
    n = ctypes.c_size_t(0)
    _check(_lib.verify_attn_mla_shared_workspace_size(len(qo) - 1, num_heads, int(shared_rows), qo.ctypes.data,
                                                      kv.ctypes.data, splits, ctypes.byref(n)),
           "verify_attn_mla_shared_workspace_size")
    return int(n.value)


def _shared_args(q, kv_pool, shared_indices, kv_indptr, kv_indices, qo_indptr, kv_indptr_host, qo_indptr_host, out,
                 lse, workspace, sm_scale, kv_scale=0.0, draft_mask=None, parent=None, splits=0, stream=None):
    kvh, qoh = _host_pair(kv_indptr_host, qo_indptr_host, "kv_indptr_host, qo_indptr_host")
    if len(kvh) != len(qoh) or len(kvh) < 1:
        raise ValueError("kv_indptr_host and qo_indptr_host: batch + 1 entries each expected")
    T, H, N = int(qoh[-1]), int(q.shape[1]), int(kvh[-1])
    for t, name, shape in ((q, "q", (T, H, D_QK)), (out, "out", (T, H, D_V)), (lse, "lse", (T, H)),
                           (kv_pool, "kv_pool", (None, D_QK)), (shared_indices, "shared_indices", (None,)),
                           (kv_indices, "kv_indices", (N,)), (kv_indptr, "kv_indptr", (len(kvh),)),
                           (qo_indptr, "qo_indptr", (len(kvh),))):
        _shape(t, name, shape)
    for t, name in ((draft_mask, "draft_mask"), (parent, "parent")):
        if t is not None:
            _shape(t, name, (T,))
    _same_device(q=q, kv_pool=kv_pool, shared_indices=shared_indices, kv_indptr=kv_indptr, kv_indices=kv_indices,
                 qo_indptr=qo_indptr, out=out, lse=lse, workspace=workspace, draft_mask=draft_mask, parent=parent)
    args = (_d(q, 2, "q"), _d(kv_pool, 1 if float(kv_scale) != 0.0 else 2, "kv_pool"), int(kv_pool.shape[0]),
            float(kv_scale), _d(shared_indices, 4, "shared_indices"), int(shared_indices.shape[0]),
            _d(kv_indptr, 4, "kv_indptr"), _d(kv_indices, 4, "kv_indices"), _d(qo_indptr, 4, "qo_indptr"),
            _d(draft_mask, 8, "draft_mask"), _d(parent, 4, "parent"), kvh.ctypes.data, qoh.ctypes.data, len(kvh) - 1,
            H, float(sm_scale), int(splits), _d(out, 2, "out"), _d(lse, 4, "lse"), _d(workspace, 0, "workspace"),
            workspace.numel() * workspace.element_size(), _stream(stream))
    return args, (q, kv_pool, shared_indices, kv_indptr, kv_indices, qo_indptr, kvh, qoh, out, lse, workspace,
                  draft_mask, parent)


def verify_attn_mla_shared(*a, **k):
    """Verify attention of a batch whose sequences share their first rows (shared_indices); kv_indptr and kv_indices
    hold each sequence's own rows.  The pool is bf16, or e4m3 codes with kv_scale > 0."""
    args, _ = _shared_args(*a, **k)
    _check(_lib.verify_attn_mla_shared(*args), "verify_attn_mla_shared")


def prepare_verify_attn_mla_shared(*a, **k) -> Prepared:
    """verify_attn_mla_shared with its arguments checked and marshalled once."""
    args, keep = _shared_args(*a, **k)
    return Prepared(_lib.verify_attn_mla_shared, "verify_attn_mla_shared", args, keep)


def _sample_args(logits, uniform, token, temperature=None, top_k=None, top_p=None, min_p=None, status_word=None,
                 stream=None):
    R, V = (int(n) for n in logits.shape) if len(logits.shape) == 2 else (None, None)
    if R is None:
        raise ValueError(f"logits: two dimensions expected, got {tuple(logits.shape)}")
    size = 0 if isinstance(logits, np.ndarray) else logits.element_size()
    if size not in (2, 4) or not str(logits.dtype).endswith(("bfloat16", "float32")):
        raise ValueError(f"logits: device memory of bfloat16 or float32 expected, got {logits.dtype}")
    for t, name in ((uniform, "uniform"), (token, "token"), (temperature, "temperature"), (top_k, "top_k"),
                    (top_p, "top_p"), (min_p, "min_p")):
        if t is not None:
            _shape(t, name, (R,))
    if status_word is not None and status_word.numel() < 2:
        raise ValueError("status_word: two words expected")
    _same_device(logits=logits, uniform=uniform, token=token, temperature=temperature, top_k=top_k, top_p=top_p,
                 min_p=min_p, status_word=status_word)
    args = (_rows(logits, size, "logits", (R, V)), int(size == 4), _step(logits, 0, V), R, V,
            _d(temperature, 4, "temperature"), _d(top_k, 4, "top_k"), _d(top_p, 4, "top_p"), _d(min_p, 4, "min_p"),
            _d(uniform, 4, "uniform"), _d(token, 4, "token"), _d(status_word, 4, "status_word"), _stream(stream))
    return args, (logits, uniform, token, temperature, top_k, top_p, min_p, status_word)


def verify_attn_mla_sample(*a, **k):
    """Draws one token per row of logits ([rows, vocab] bf16 or fp32, rows may be strided) into `token` [rows] int32
    with the random numbers `uniform` [rows]; temperature, top_k, top_p and min_p are per-row arrays or None."""
    args, _ = _sample_args(*a, **k)
    _check(_lib.verify_attn_mla_sample(*args), "verify_attn_mla_sample")


def prepare_verify_attn_mla_sample(*a, **k) -> Prepared:
    """verify_attn_mla_sample with its arguments checked and marshalled once."""
    args, keep = _sample_args(*a, **k)
    return Prepared(_lib.verify_attn_mla_sample, "verify_attn_mla_sample", args, keep)


def verify_attn_mla_runs_workspace_size(qo_indptr_host, kv_indptr_host, num_heads: int, splits: int = 0) -> int:
    qo, kv = _host_pair(qo_indptr_host, kv_indptr_host, "qo_indptr_host, kv_indptr_host")
    n = ctypes.c_size_t(0)
    _check(_lib.verify_attn_mla_runs_workspace_size(len(qo) - 1, num_heads, qo.ctypes.data, kv.ctypes.data, splits,
                                                    ctypes.byref(n)), "verify_attn_mla_runs_workspace_size")
    return int(n.value)


def verify_attn_mla_runs(q, kv_pool, kv_indptr, run_base, qo_indptr, kv_indptr_host, qo_indptr_host, out, lse,
                         workspace, sm_scale, draft_mask=None, parent=None, splits=0, stream=None):
    """Tensor-core verify attention on rows that lie in per-sequence runs of the pool (no gather)."""
    _run(_lib.verify_attn_mla_runs, "verify_attn_mla_runs", q, kv_pool, kv_indptr, run_base, qo_indptr,
         kv_indptr_host, qo_indptr_host, out, lse, workspace, sm_scale, draft_mask, parent, splits, stream)


def prepare_verify_attn_mla_runs(q, kv_pool, kv_indptr, run_base, qo_indptr, kv_indptr_host, qo_indptr_host, out,
                                 lse, workspace, sm_scale, draft_mask=None, parent=None, splits=0,
                                 stream=None) -> Prepared:
    """verify_attn_mla_runs with its arguments checked and marshalled once."""
    args, keep = _run_args(q, kv_pool, kv_indptr, run_base, qo_indptr, kv_indptr_host, qo_indptr_host, out, lse,
                           workspace, sm_scale, draft_mask, parent, splits, stream)
    return Prepared(_lib.verify_attn_mla_runs, "verify_attn_mla_runs", args, keep)


def _fp8_args(q, kv_pool_e4m3, kv_scale, kv_indptr, kv_indices, qo_indptr, kv_indptr_host, qo_indptr_host, out, lse,
              workspace, sm_scale, draft_mask=None, parent=None, splits=0, stream=None):
    kvh, qoh = _host_pair(kv_indptr_host, qo_indptr_host, "kv_indptr_host, qo_indptr_host")
    args = (_d(q, 2, "q"), _d(kv_pool_e4m3, 1, "kv_pool_e4m3"), int(kv_pool_e4m3.shape[0]), float(kv_scale),
            _d(kv_indptr, 4, "kv_indptr"), _d(kv_indices, 4, "kv_indices"), _d(qo_indptr, 4, "qo_indptr"),
            _d(draft_mask, 8, "draft_mask"), _d(parent, 4, "parent"), kvh.ctypes.data, qoh.ctypes.data, len(kvh) - 1,
            int(q.shape[1]), float(sm_scale), int(splits), _d(out, 2, "out"), _d(lse, 4, "lse"),
            _d(workspace, 0, "workspace"), workspace.numel() * workspace.element_size(), _stream(stream))
    return args, (q, kv_pool_e4m3, kv_indptr, kv_indices, qo_indptr, kvh, qoh, out, lse, workspace, draft_mask, parent)


def verify_attn_mla_fp8(q, kv_pool_e4m3, kv_scale, kv_indptr, kv_indices, qo_indptr, kv_indptr_host, qo_indptr_host,
                        out, lse, workspace, sm_scale, draft_mask=None, parent=None, splits=0, stream=None):
    """verify_attn_mla on an e4m3 latent pool ([S, 576] uint8 codes) with one scale."""
    args, _ = _fp8_args(q, kv_pool_e4m3, kv_scale, kv_indptr, kv_indices, qo_indptr, kv_indptr_host, qo_indptr_host,
                        out, lse, workspace, sm_scale, draft_mask, parent, splits, stream)
    _check(_lib.verify_attn_mla_fp8(*args), "verify_attn_mla_fp8")


def prepare_verify_attn_mla_fp8(*a, **k) -> Prepared:
    """verify_attn_mla_fp8 with its arguments checked and marshalled once."""
    args, keep = _fp8_args(*a, **k)
    return Prepared(_lib.verify_attn_mla_fp8, "verify_attn_mla_fp8", args, keep)


def verify_attn_mla_test_fault(fault: int, wait_cycles: int = 0):
    """Failure test only: fault 1 makes the next tensor-core calls on this thread time out; 0 restores."""
    _check(_lib.verify_attn_mla_test_fault(int(fault), int(wait_cycles)), "verify_attn_mla_test_fault")


def verify_attn_mla_tree_accept(qo_indptr, parent, draft_token, target_token, root_token, accept_len, accept_path,
                                next_token, status_word=None, stream=None):
    """Greedy acceptance of the verified draft tree (device int32 arrays; parent None = chain)."""
    batch = int(qo_indptr.numel()) - 1
    rc = _lib.verify_attn_mla_tree_accept(_d(qo_indptr, 4, "qo_indptr"), _d(parent, 4, "parent"),
                                          _d(draft_token, 4, "draft_token"), _d(target_token, 4, "target_token"),
                                          _d(root_token, 4, "root_token"), batch, int(draft_token.numel()),
                                          _d(accept_len, 4, "accept_len"), _d(accept_path, 4, "accept_path"),
                                          _d(next_token, 4, "next_token"), _d(status_word, 4, "status_word"),
                                          _stream(stream))
    _check(rc, "verify_attn_mla_tree_accept")


def verify_attn_mla_simt(q, kv_pool, kv_indptr, kv_indices, qo_indptr, kv_indptr_host, qo_indptr_host, out, lse,
                         workspace, sm_scale, draft_mask=None, parent=None, splits=0, stream=None):
    """Same operation on the CUDA-core kernel."""
    _run(_lib.verify_attn_mla_simt, "verify_attn_mla_simt", q, kv_pool, kv_indptr, kv_indices, qo_indptr,
         kv_indptr_host, qo_indptr_host, out, lse, workspace, sm_scale, draft_mask, parent, splits, stream)


def verify_attn_mla_merge(o_parts, lse_parts, out, lse, stream=None):
    S, R = int(o_parts.shape[0]), int(o_parts.shape[1])
    _check(_lib.verify_attn_mla_merge(_d(o_parts, 4, "o_parts"), _d(lse_parts, 4, "lse_parts"), S, R,
                                      _d(out, 2, "out"), _d(lse, 4, "lse"), _stream(stream)), "verify_attn_mla_merge")


def verify_attn_mla_tree_mask(parent, qo_indptr, mask_out, status_word=None, stream=None):
    B = int(qo_indptr.shape[0]) - 1
    T = int(parent.shape[0])
    _check(_lib.verify_attn_mla_tree_mask(_d(parent, 4, "parent"), _d(qo_indptr, 4, "qo_indptr"), B, T,
                                          _d(mask_out, 8, "mask_out"), _d(status_word, 4, "status_word"),
                                          _stream(stream)), "verify_attn_mla_tree_mask")


def verify_attn_mla_check(workspace, stream=None) -> int:
    """Device status of the last call on `workspace` (synchronises the stream)."""
    return int(_lib.verify_attn_mla_check(_d(workspace, 0, "workspace"), _stream(stream)))


def verify_attn_mla_host_buffer_size(qo_indptr_host, kv_indptr_host, num_heads: int, splits: int = 0,
                                     has_mask: bool = False, has_parent: bool = False) -> int:
    qo, kv = _host_pair(qo_indptr_host, kv_indptr_host, "qo_indptr_host, kv_indptr_host")
    n = ctypes.c_size_t(0)
    _check(_lib.verify_attn_mla_host_buffer_size(len(qo) - 1, num_heads, qo.ctypes.data, kv.ctypes.data, splits,
                                                 int(has_mask), int(has_parent), ctypes.byref(n)),
           "verify_attn_mla_host_buffer_size")
    return int(n.value)


def _host_args(q_host, kv_pool, kv_indptr_host, kv_indices_host, qo_indptr_host, out_host, lse_host, device_buffer,
               sm_scale, draft_mask_host=None, parent_host=None, splits=0, stream=None, num_heads=None):
    kvh, qoh = _host_pair(kv_indptr_host, qo_indptr_host, "kv_indptr_host, qo_indptr_host")
    H = int(num_heads if num_heads is not None else q_host.shape[1])
    args = (_h(q_host, 2, "q_host"), _d(kv_pool, 2, "kv_pool"), int(kv_pool.shape[0]), kvh.ctypes.data,
            _h(kv_indices_host, 4, "kv_indices_host"), qoh.ctypes.data, _h(draft_mask_host, 8, "draft_mask_host"),
            _h(parent_host, 4, "parent_host"), len(kvh) - 1, H, float(sm_scale), int(splits),
            _h(out_host, 2, "out_host"), _h(lse_host, 4, "lse_host"), _d(device_buffer, 0, "device_buffer"),
            device_buffer.numel() * device_buffer.element_size(), _stream(stream))
    return args, (q_host, kv_pool, kvh, kv_indices_host, qoh, out_host, lse_host, device_buffer, draft_mask_host,
                  parent_host)


def verify_attn_mla_host(*a, **k):
    """Host-memory inputs/outputs, device-resident kv_pool; returns after the stream has finished."""
    args, _ = _host_args(*a, **k)
    _check(_lib.verify_attn_mla_host(*args), "verify_attn_mla_host")


def prepare_verify_attn_mla_host(*a, **k) -> Prepared:
    """verify_attn_mla_host with its arguments checked and marshalled once; call the result to run it."""
    args, keep = _host_args(*a, **k)
    return Prepared(_lib.verify_attn_mla_host, "verify_attn_mla_host", args, keep)


def verify_attn_mla_version() -> int:
    return int(_lib.verify_attn_mla_version())


def verify_attn_mla_timing_enable(capacity: int):
    _check(_lib.verify_attn_mla_timing_enable(int(capacity)), "verify_attn_mla_timing_enable")


def verify_attn_mla_timing_read(capacity: int):
    """(gather_ms, verify_ms, merge_ms) arrays of the recorded calls, in launch order."""
    g = np.zeros(max(capacity, 1), np.float32)
    v = np.zeros(max(capacity, 1), np.float32)
    m = np.zeros(max(capacity, 1), np.float32)
    n = ctypes.c_int(0)
    _check(_lib.verify_attn_mla_timing_read(g.ctypes.data, v.ctypes.data, m.ctypes.data, int(capacity),
                                            ctypes.byref(n)), "verify_attn_mla_timing_read")
    return g[: n.value].copy(), v[: n.value].copy(), m[: n.value].copy()


STATIC_SCRATCH_BYTES = 32 << 20


def verify_attn_mla_simt_static(q, kv_pool, kv_indptr, kv_indices, qo_indptr, kv_indptr_host, qo_indptr_host, out,
                                lse, sm_scale, draft_mask=None, parent=None, splits=0, stream=None):
    """CUDA-core verify with the library's fixed scratch array instead of a workspace (no allocation)."""
    kvh, qoh = _host_pair(kv_indptr_host, qo_indptr_host, "kv_indptr_host, qo_indptr_host")
    rc = _lib.verify_attn_mla_simt_static(_d(q, 2, "q"), _d(kv_pool, 2, "kv_pool"), int(kv_pool.shape[0]),
                                          _d(kv_indptr, 4, "kv_indptr"), _d(kv_indices, 4, "kv_indices"),
                                          _d(qo_indptr, 4, "qo_indptr"), _d(draft_mask, 8, "draft_mask"),
                                          _d(parent, 4, "parent"),
                                          kvh.ctypes.data, qoh.ctypes.data, len(kvh) - 1, int(q.shape[1]),
                                          float(sm_scale), int(splits), _d(out, 2, "out"), _d(lse, 4, "lse"),
                                          _stream(stream))
    _check(rc, "verify_attn_mla_simt_static")


def verify_attn_mla_simt_static_check(stream=None) -> int:
    """Synchronises the stream and returns the status word the static-scratch calls left (0 = ok)."""
    return int(_lib.verify_attn_mla_simt_static_check(_stream(stream)))
