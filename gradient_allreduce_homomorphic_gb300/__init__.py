"""Python binding of libgar.so, the GB300 gradient-averaging library.

Argument marshalling only: every step of the path runs in the library's CUDA
kernels.  PyTorch supplies device memory and streams.  The functions carry
the names of the C entry points declared in ``include/gar.h``; they take
torch tensors (and lists of them) in place of raw pointers, enqueue on the
current CUDA stream unless ``stream`` is given, and raise ``GarError`` on a
non-zero status.  There is no fallback: if the library is not built, or the
tensors are not on a CUDA device, the call fails.
"""
from __future__ import annotations

import ctypes as C
import os
import struct
import threading
from dataclasses import dataclass

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libgar.so")

GAR_OK, GAR_EINVAL, GAR_EDTYPE, GAR_EALIGN, GAR_EOVERFLOW, GAR_ECUDA = 0, -1, -2, -3, -4, -5
GAR_F32, GAR_BF16 = 0, 1
GAR_F8E4M3, GAR_F8E5M2 = 0, 1
GAR_SUM, GAR_AVG = 0, 1
GAR_MAX_WORKERS = 64


class GarError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"gar status {status}: {message}")
        self.status = status


class gar_seg(C.Structure):
    _fields_ = [("buffer", C.c_int32), ("reserved", C.c_int32), ("offset", C.c_int64), ("numel", C.c_int64)]


_lock = threading.Lock()
_lib = None
_bound = {}  # entry point -> its ctypes function, once the library is loaded

_vp, _pp = C.c_void_p, C.POINTER(C.c_void_p)
_i32, _i64, _u64 = C.c_int32, C.c_int64, C.c_uint64
_SIGNATURES = {
    "gar_version": (C.c_int, []),
    "gar_last_error": (C.c_char_p, []),
    "gar_launch_count": (C.c_uint64, []),
    "gar_sync_status": (C.c_int, [_vp, _vp, _i32]),
    "gar_checksum": (C.c_int, [_vp, _i64, _vp, _vp]),
    "gar_fusion_plan": (C.c_int, [_vp, _vp, _i32, _i64, _i32, _vp, C.POINTER(_i32), _vp]),
    "gar_fusion_pack": (C.c_int, [_pp, _vp, _vp, _i32, _i32, _vp, _i64, _vp]),
    "gar_fusion_unpack": (C.c_int, [_vp, _vp, _vp, _i32, _i32, _pp, _vp]),
    "gar_fused_allreduce": (C.c_int, [_pp, _pp, _i32, _vp, _vp, _i32, _vp, _i32, _i32, _vp]),
    "gar_fusion_pack_all": (C.c_int, [_pp, _i32, _vp, _vp, _i32, _pp, _vp, _i32, _vp, _vp]),
    "gar_fused_allreduce_range": (C.c_int, [_pp, _pp, _i32, _vp, _vp, _i32, _vp, _i32, _i32, _vp, _vp]),
    "gar_ring_allreduce_sim": (C.c_int, [_pp, _i32, _i64, _i32, _i32, _vp]),
    "gar_ring_allreduce_sim_out": (C.c_int, [_pp, _i32, _i64, _i32, _i32, _pp, _i32, _vp]),
    "gar_ring_allreduce_bidir": (C.c_int, [_pp, _i32, _i64, _i32, _i32, _vp]),
    "gar_ring_allreduce_steps": (C.c_int, [_pp, _i32, _i64, _i32, C.POINTER(_i32), _vp, _vp]),
    "gar_dbtree_allreduce": (C.c_int, [_pp, _i32, _i64, _i32, _i32, _vp]),
    "gar_dbtree_parents": (C.c_int, [_i32, _i32, _vp]),
    "gar_thc_words": (_i64, [_i64, _i32]),
    "gar_thc_range": (C.c_int, [_pp, _i32, _i64, _vp, _vp]),
    "gar_thc_encode": (C.c_int, [_vp, _i64, _vp, _i32, _u64, _i32, _vp, _vp]),
    "gar_thc_aggregate": (C.c_int, [_pp, _i32, _i64, _i32, _vp, _vp]),
    "gar_thc_decode": (C.c_int, [_vp, _i64, _vp, _i32, _i32, _vp, _vp]),
    "gar_thc_allreduce_fused": (C.c_int, [_pp, _i32, _i64, _i32, _u64, _vp, _vp, _pp, _vp]),
    "gar_thc_allreduce_fused_masked": (C.c_int, [_pp, _i32, _u64, _i64, _i32, _u64, _vp, _vp, _pp, _vp]),
    "gar_thc_allreduce_fused_plan": (C.c_int, [_pp, _i32, _vp, _vp, _i32, _vp, _i32, _i32, _u64, _vp, _pp, _pp,
                                               _vp]),
    "gar_thc_plan_nmse_workspace_bytes": (C.c_size_t, [_vp, _i32, _i32, _i32]),
    "gar_thc_allreduce_fused_plan_nmse": (C.c_int, [_pp, _i32, _vp, _vp, _i32, _vp, _i32, _i32, _u64, _vp, _pp,
                                                    _pp, _pp, _vp, _vp, C.c_size_t, _vp]),
    "gar_nuhc_encode": (C.c_int, [_vp, _i64, _vp, _i32, _i32, _vp, _u64, _i32, _vp, _vp]),
    "gar_nuhc_aggregate": (C.c_int, [_pp, _i32, _i64, _i32, _vp, _vp, _vp]),
    "gar_nuhc_decode": (C.c_int, [_vp, _i64, _vp, _i32, _i32, _vp, _vp]),
    "gar_nuhc_allreduce_fused": (C.c_int, [_pp, _i32, _i64, _i32, _i32, _vp, _u64, _vp, _vp, _pp, _vp]),
    "gar_nuhc_allreduce_fused_masked": (C.c_int, [_pp, _i32, _u64, _i64, _i32, _i32, _vp, _u64, _vp, _vp, _pp,
                                                  _vp]),
    "gar_rht": (C.c_int, [_vp, _vp, _i64, _u64, _i32, _vp]),
    "gar_rht_norm_range_workspace_bytes": (C.c_size_t, [_i32, _i64]),
    "gar_rht_norm_range": (C.c_int, [_pp, _i32, _i64, C.c_double, _vp, _vp, C.c_size_t, _vp]),
    "gar_rht_tiles": (_i64, [_i64]),
    "gar_rht_ef_forward": (C.c_int, [_vp, _vp, _vp, _i64, _u64, _vp, _vp]),
    "gar_rht_norm_range_from_sums": (C.c_int, [_pp, _i32, _i64, C.c_double, _vp, _vp]),
    "gar_rht_ef_update": (C.c_int, [_vp, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _i64, _u64, _vp]),
    "gar_ef_apply": (C.c_int, [_vp, _vp, _vp, _i64, _vp]),
    "gar_ef_update": (C.c_int, [_vp, _vp, _vp, _i64, _vp]),
    "gar_nmse_workspace_bytes": (C.c_size_t, [_i64]),
    "gar_nmse": (C.c_int, [_vp, _vp, _i64, _vp, _vp, C.c_size_t, _vp]),
    "gar_nmse_noalloc": (C.c_int, [_vp, _vp, _i64, _vp, _vp]),
    "gar_nmse_sums": (C.c_int, [_vp, _vp, _i64, _vp, _vp, C.c_size_t, _vp]),
    "gar_nmse_combine": (C.c_int, [_vp, _i32, _vp, _vp]),
    "gar_fp8_scale_bytes": (_i64, [_i64, _i64]),
    "gar_fp8_quantize": (C.c_int, [_vp, _i32, _i64, _i64, _i64, _i32, _i32, _vp, _i64, _vp, _vp, _i64, _vp, _vp]),
    "gar_fp8_matmul": (C.c_int, [_vp, _i64, _vp, _i32, _vp, _i64, _vp, _i32, _i64, _i64, _i64, _vp, _i64, _vp, _i64,
                                 _i32, _vp]),
    "gar_distill_loss": (C.c_int, [_vp, _i32, _i64, _i64, _i64, _vp, _vp, _i32, C.c_float, _vp, _vp, _vp, _vp, _i64,
                                   _vp]),
    "gar_distill_grad": (C.c_int, [_vp, _i32, _i64, _i64, _i64, _vp, _vp, _i32, C.c_float, _vp, _vp, _vp, _i64, _vp]),
    "gar_balance_workspace_bytes": (C.c_size_t, [_i32]),
    "gar_balance_loss": (C.c_int, [_vp, _i32, _i64, _i32, _i64, _i32, _i32, _vp, C.c_float, _vp, _vp, _vp, _vp, _i64,
                                   _vp, C.c_size_t, _vp]),
    "gar_vocab_workspace_bytes": (C.c_size_t, [_i64, _i64, _i64, _i32]),
    "gar_vocab_loss": (C.c_int, [_vp, _i64, _vp, _i64, _i32, _vp, _vp, _i64, _i64, _i64, _vp, _vp, _vp, C.c_size_t, _vp]),
    "gar_vocab_grad": (C.c_int, [_vp, _i64, _vp, _i64, _i32, _vp, _vp, _i64, _i64, _i64, _vp, _vp, _i64, _vp, _i64, _vp,
                                 _i64, _i32, _vp, C.c_size_t, _vp]),
    "gar_vocab_grad_with_loss": (C.c_int, [_vp, _i64, _vp, _i64, _i32, _vp, _vp, _i64, _i64, _i64, _vp, _vp, _vp, _i64, _vp,
                                           _i64, _vp, _i64, _i32, _i32, _vp, C.c_size_t, _vp]),
    "gar_expert_rows": (_i64, [_i32, _i64, _i32, _i32, _i32, _i32]),
    "gar_expert_workspace_bytes": (C.c_size_t, [_i32, _i64, _i32, _i32]),
    "gar_expert_sort": (C.c_int, [_vp, _i32, _i64, _i32, _i32, _i32, _i32, _vp, _vp, _i64, _vp, _vp, C.c_size_t, _vp]),
    "gar_expert_gather": (C.c_int, [_vp, _i32, _i64, _i64, _i64, _i32, _i32, _vp, _vp, _i64, _vp, _vp, _i64, _vp]),
    "gar_expert_combine": (C.c_int, [_vp, _i64, _i64, _i32, _i64, _i64, _i32, _i32, _vp, _vp, _vp, _i64, _vp, _i64, _vp]),
    "gar_expert_combine_grad": (C.c_int, [_vp, _i64, _vp, _i64, _i32, _i64, _i64, _i32, _i32, _vp, _vp, _i64, _vp, _vp, _i64,
                                          _vp, _vp]),
    "gar_expert_weights": (C.c_int, [_vp, _i32, _i64, _i32, _i64, _i32, _i32, _vp, _vp, _vp]),
    "gar_expert_weights_grad": (C.c_int, [_vp, _vp, _i32, _i64, _i32, _i32, _vp, _vp, _i64, _i32, _i32, _vp]),
    "gar_grad_workspace_bytes": (C.c_size_t, [_i32, _i32]),
    "gar_grad_norm": (C.c_int, [_vp, _i32, _vp, _vp, _i32, _vp, _vp, C.c_size_t, _vp]),
    "gar_grad_clip": (C.c_int, [_vp, _vp, _i32, _vp, _vp, _i32, _i32, C.c_float, _vp, _vp, C.c_size_t, _vp]),
}


def load(path: str = LIB_PATH):
    """Load libgar.so (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(path):
                raise RuntimeError(
                    f"{path} is missing: build it with gradient_allreduce_homomorphic_gb300.build.build() "
                    "(there is no CPU fallback)")
            lib = C.CDLL(path)
            for name, (res, args) in _SIGNATURES.items():
                fn = getattr(lib, name)
                fn.restype = res
                fn.argtypes = args
                _bound[name] = fn
            _lib = lib
    return _lib


class _StreamArg(C.c_void_p):
    """The cudaStream_t argument of a device call (marks the call for the timeline)."""


class Timeline:
    """Horovod-Timeline-like trace of the library's device calls ([H]
    "Horovod Timeline"): with the environment variable GAR_TIMELINE set to a
    path, every call that enqueues device work is bracketed by a pair of CUDA
    events on its own stream, and at exit (or on ``dump()``) the calls are
    written as Chrome Trace Event JSON (chrome://tracing): one complete event
    per call, named after the entry point, timestamps in microseconds from
    the first call, one track per stream.  Events cost a few microseconds of
    host time per call, so the timeline is off unless asked for."""

    def __init__(self, path: str):
        import atexit

        self.path = path
        self.records = []  # (name, stream handle, start event, end event)
        self._lock = threading.Lock()
        atexit.register(self.dump)

    def begin(self, name, stream_handle):
        import torch

        ext = torch.cuda.ExternalStream(stream_handle) if stream_handle else torch.cuda.default_stream()
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record(ext)
        return (name, stream_handle or 0, start, end, ext)

    def end(self, token):
        name, handle, start, end, ext = token
        end.record(ext)
        with self._lock:
            self.records.append((name, handle, start, end))

    def events(self):
        """The recorded calls as Chrome trace events (synchronises the device)."""
        import torch

        with self._lock:
            recs = list(self.records)
        if not recs:
            return []
        torch.cuda.synchronize()
        t0 = recs[0][2]
        tracks = {}
        out = []
        for name, handle, start, end in recs:
            tid = tracks.setdefault(handle, len(tracks))
            out.append({"name": name, "cat": "gar", "ph": "X", "pid": 0, "tid": tid,
                        "ts": round(t0.elapsed_time(start) * 1e3, 3), "dur": round(start.elapsed_time(end) * 1e3, 3),
                        "args": {"stream": hex(handle)}})
        return out

    def dump(self):
        import json

        try:
            ev = self.events()
        except Exception:  # the CUDA context may be gone at interpreter exit
            return
        with open(self.path, "w") as f:
            json.dump({"traceEvents": ev, "displayTimeUnit": "ms"}, f)


_timeline = Timeline(os.environ["GAR_TIMELINE"]) if os.environ.get("GAR_TIMELINE") else None


def timeline():
    """The active Timeline, or None when GAR_TIMELINE is not set."""
    return _timeline


def _call(name, *args):
    token = None
    if _timeline is not None and args and isinstance(args[-1], _StreamArg):
        token = _timeline.begin(name, args[-1].value)
    rc = (_bound.get(name) or getattr(load(), name))(*args)
    if token is not None:
        _timeline.end(token)
    if rc != GAR_OK:
        raise GarError(rc, load().gar_last_error().decode(errors="replace"))


_current_stream = None  # () -> handle of the current stream of the current device


def _find_current_stream():
    """The current stream's handle without building torch's stream object
    (3 us of a call's host time) where this torch can say it directly."""
    import torch

    global _current_stream
    raw, device = getattr(torch._C, "_cuda_getCurrentRawStream", None), getattr(torch._C, "_cuda_getDevice", None)
    if raw is None or device is None:
        _current_stream = lambda: torch.cuda.current_stream().cuda_stream  # noqa: E731
    else:
        torch.cuda.init()
        _current_stream = lambda: raw(device())  # noqa: E731
    return _current_stream


def _stream(stream):
    if stream is None:
        handle = (_current_stream or _find_current_stream())()
    else:
        handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    return handle if _timeline is None else _StreamArg(handle)


def _dev(t):
    if not t.is_cuda:
        raise GarError(GAR_EINVAL, "tensor is not on a CUDA device (the library has no CPU path)")
    return t.data_ptr()


class PtrTable:
    """A host array of device pointers built once from a list of tensors, so
    that repeated calls skip the per-call marshalling.  Keeps the tensors
    alive; numel and dtype describe the first tensor."""

    def __init__(self, tensors, allow_none: bool = False):
        self.tensors = list(tensors)
        if allow_none:
            ptrs = [_dev(t) if t is not None else None for t in self.tensors]
        else:
            ptrs = [t.data_ptr() if t.is_cuda else _dev(t) for t in self.tensors]
        self.array = (C.c_void_p * len(ptrs))(*ptrs)
        first = next((t for t in self.tensors if t is not None), None)
        self.numel = first.numel() if first is not None else 0
        self.first = first
        self.checked = {}  # (shape, dtype) that every tensor was found to have -> their stride
        self.last = None   # (P, shape, dtype) asked of them last, and what _workers said
        self.size = tuple(first.shape) if first is not None and first.dim() == 2 else None

    def __len__(self):
        return len(self.tensors)


def pointer_table(tensors, allow_none: bool = False) -> PtrTable:
    return tensors if isinstance(tensors, PtrTable) else PtrTable(tensors, allow_none)


def _ptr_array(tensors):
    return pointer_table(tensors).array


def _dtype_code(t) -> int:
    import torch

    if t.dtype == torch.float32:
        return GAR_F32
    if t.dtype == torch.bfloat16:
        return GAR_BF16
    raise GarError(GAR_EDTYPE, f"unsupported dtype {t.dtype}")


def gar_version() -> int:
    return int(load().gar_version())


def gar_last_error() -> str:
    return load().gar_last_error().decode(errors="replace")


def gar_launch_count() -> int:
    return int(load().gar_launch_count())


# ------------------------------------------------------------ Tensor Fusion
@dataclass
class FusionPlan:
    segs: C.Array           # gar_seg[count]
    dtype: np.ndarray       # int32[count]
    buf_numel: np.ndarray   # int64[n_buffers]

    @property
    def count(self) -> int:
        return len(self.dtype)

    @property
    def n_buffers(self) -> int:
        return len(self.buf_numel)

    def buffers(self) -> np.ndarray:
        return np.array([s.buffer for s in self.segs], np.int32)

    def offsets(self) -> np.ndarray:
        return np.array([s.offset for s in self.segs], np.int64)

    def subplan(self, first: int, count: int) -> "FusionPlan":
        """The plan restricted to tensors first .. first+count-1 (a view of the
        same segments; buffer ids and buffer lengths unchanged)."""
        segs = (gar_seg * max(count, 1)).from_address(C.addressof(self.segs) + first * C.sizeof(gar_seg))
        sub = FusionPlan(segs, self.dtype[first:first + count].copy(), self.buf_numel)
        sub._parent = self  # keep the segment storage alive
        return sub

    def buffer_tensors(self, buffer: int):
        """(first, count) of the tensors of one buffer (contiguous in plan order)."""
        ids = np.nonzero(self.buffers() == buffer)[0]
        return (int(ids[0]), int(ids.size)) if ids.size else (0, 0)


def gar_fusion_plan(numel, dtype, capacity_bytes: int = 64 << 20, align_bytes: int = 16) -> FusionPlan:
    numel = np.ascontiguousarray(numel, np.int64)
    dtype = np.ascontiguousarray(dtype, np.int32)
    count = int(numel.size)
    segs = (gar_seg * max(count, 1))()
    bn = np.zeros(max(count, 1), np.int64)
    nb = _i32(0)
    _call("gar_fusion_plan", numel.ctypes.data, dtype.ctypes.data, count, capacity_bytes, align_bytes,
          C.addressof(segs), C.byref(nb), bn.ctypes.data)
    return FusionPlan(segs, dtype, bn[:nb.value].copy())


def gar_fusion_pack(src, plan: FusionPlan, buffer: int, fusion_buf, stream=None):
    """src: one worker's tensors (list or PtrTable; entries of other buffers may be None)."""
    ptrs = pointer_table(src, allow_none=True).array
    _call("gar_fusion_pack", ptrs, C.addressof(plan.segs), plan.dtype.ctypes.data, plan.count, buffer,
          _dev(fusion_buf), int(plan.buf_numel[buffer]), _stream(stream))


def gar_fusion_unpack(fusion_buf, plan: FusionPlan, buffer: int, dst, stream=None):
    ptrs = pointer_table(dst, allow_none=True).array
    _call("gar_fusion_unpack", _dev(fusion_buf), C.addressof(plan.segs), plan.dtype.ctypes.data, plan.count,
          buffer, ptrs, _stream(stream))


def gar_fusion_pack_all(src, plan: FusionPlan, fusion_bufs, d_mM=None, stream=None, tables=None):
    """Pack every worker's tensors into its fusion buffers in one pass.

    src[w][i]: worker w's tensor i; fusion_bufs[w][b]: worker w's buffer b;
    d_mM (optional, fp32 plans): [n_buffers, 2] per-buffer min/max output."""
    if tables is None:
        tables = pack_all_tables(src, fusion_bufs)
    s, f = tables
    P = len(s) // max(plan.count, 1)
    _call("gar_fusion_pack_all", s.array, P, C.addressof(plan.segs), plan.dtype.ctypes.data, plan.count, f.array,
          plan.buf_numel.ctypes.data, plan.n_buffers, _dev(d_mM) if d_mM is not None else None, _stream(stream))


def pack_all_tables(src, fusion_bufs):
    """Host pointer tables for gar_fusion_pack_all (reuse them across steps)."""
    return (PtrTable([t for row in src for t in row]), PtrTable([t for row in fusion_bufs for t in row]))


def fused_pointer_tables(src, dst):
    """Host pointer tables for gar_fused_allreduce (reuse them across steps)."""
    return (PtrTable([t for row in src for t in row]), PtrTable([t for row in dst for t in row]))


def gar_fused_allreduce(src, dst, plan: FusionPlan, op: int = GAR_AVG, stream=None, tables=None):
    """src[w][i], dst[w][i]: worker w's tensor i (dst may be src)."""
    P = len(src)
    s, d = tables if tables is not None else fused_pointer_tables(src, dst)
    _call("gar_fused_allreduce", s.array, d.array, P, C.addressof(plan.segs), plan.dtype.ctypes.data, plan.count,
          plan.buf_numel.ctypes.data, plan.n_buffers, op, _stream(stream))


def gar_fused_allreduce_range(src, dst, plan: FusionPlan, d_mM, op: int = GAR_AVG, stream=None, tables=None):
    """gar_fused_allreduce that also writes each buffer's THC range [m, M]
    (d_mM: [n_buffers, 2] fp32 device tensor) from the same reads."""
    P = len(src)
    s, d = tables if tables is not None else fused_pointer_tables(src, dst)
    _call("gar_fused_allreduce_range", s.array, d.array, P, C.addressof(plan.segs), plan.dtype.ctypes.data,
          plan.count, plan.buf_numel.ctypes.data, plan.n_buffers, op, _dev(d_mM), _stream(stream))


GAR_STATUS_NONFINITE = 1
GAR_STATUS_TIMEOUT = 2


def gar_checksum(words, d_out, stream=None):
    """(s2 << 32) | s1 of the 32-bit words (a CUDA tensor of 4-byte elements)
    into d_out (one int64/uint64 element on the device)."""
    n = words.numel() * words.element_size() // 4
    _call("gar_checksum", _dev(words), n, _dev(d_out), _stream(stream))


def gar_sync_status(stream=None, clear: bool = True) -> int:
    """Wait for `stream`, then return the device status word (GAR_STATUS_*
    bits: conditions the kernels found on the device), clearing it if asked."""
    out = C.c_uint32(0)
    _call("gar_sync_status", _stream(stream), C.byref(out), 1 if clear else 0)
    return int(out.value)


# ----------------------------------------------------------- ring all-reduce
def gar_ring_allreduce_sim(bufs, op: int = GAR_AVG, stream=None):
    t = pointer_table(bufs)
    _call("gar_ring_allreduce_sim", t.array, len(t), t.numel, _dtype_code(t.first), op, _stream(stream))


def gar_ring_allreduce_bidir(bufs, op: int = GAR_AVG, stream=None):
    """Bidirectional dual ring (in place): first half clockwise, second half counter-clockwise."""
    t = pointer_table(bufs)
    _call("gar_ring_allreduce_bidir", t.array, len(t), t.numel, _dtype_code(t.first), op, _stream(stream))


def gar_dbtree_allreduce(bufs, op: int = GAR_AVG, stream=None):
    """Double-binary-tree all-reduce (in place): first half over tree 1, the rest over tree 2."""
    t = pointer_table(bufs)
    _call("gar_dbtree_allreduce", t.array, len(t), t.numel, _dtype_code(t.first), op, _stream(stream))


def gar_dbtree_parents(P: int, tree: int):
    """Host only: parent rank of every rank in tree 0 or 1 (-1: the root)."""
    out = np.zeros(P, np.int32)
    _call("gar_dbtree_parents", P, tree, out.ctypes.data)
    return out


def gar_ring_allreduce_sim_out(bufs, out, op: int = GAR_AVG, stream=None):
    t, o = pointer_table(bufs), pointer_table(out)
    _call("gar_ring_allreduce_sim_out", t.array, len(t), t.numel, _dtype_code(t.first), op,
          o.array, len(o), _stream(stream))


def gar_ring_allreduce_steps(bufs, op: int = GAR_AVG, stream=None):
    """Literal schedule (fp32, in place); returns (steps, sent_elems[P])."""
    P = len(bufs)
    steps = _i32(0)
    sent = np.zeros(P, np.int64)
    _call("gar_ring_allreduce_steps", _ptr_array(bufs), P, bufs[0].numel(), op, C.byref(steps),
          sent.ctypes.data, _stream(stream))
    return steps.value, sent


# --------------------------------------------------------------------- THC
def gar_thc_words(N: int, b: int) -> int:
    return int(load().gar_thc_words(N, b))


def gar_thc_range(x, d_mM, stream=None):
    t = pointer_table(x)
    _call("gar_thc_range", t.array, len(t), t.numel, _dev(d_mM), _stream(stream))


def gar_thc_encode(x, d_mM, b: int, seed: int, worker: int, packed, stream=None):
    _call("gar_thc_encode", _dev(x), x.numel(), _dev(d_mM), b, seed, worker, _dev(packed), _stream(stream))


def gar_thc_aggregate(packed, N: int, b: int, sums, stream=None):
    t = pointer_table(packed)
    _call("gar_thc_aggregate", t.array, len(t), N, b, _dev(sums), _stream(stream))


def gar_thc_decode(sums, d_mM, b: int, P: int, avg, stream=None):
    _call("gar_thc_decode", _dev(sums), sums.numel(), _dev(d_mM), b, P, _dev(avg), _stream(stream))


def gar_thc_allreduce_fused(x, b: int, seed: int, d_mM, avg, packed=None, stream=None):
    t = pointer_table(x)
    pk = pointer_table(packed).array if packed is not None else None
    _call("gar_thc_allreduce_fused", t.array, len(t), t.numel, b, seed, _dev(d_mM), _dev(avg), pk,
          _stream(stream))


def gar_thc_allreduce_fused_masked(x, arrived: int, b: int, seed: int, d_mM, avg, packed=None, stream=None):
    """THC round over the workers whose bit is set in `arrived` (stragglers
    dropped); x[w] / packed[w] of the others may be None."""
    xt = pointer_table(x, allow_none=True)
    pk = pointer_table(packed, allow_none=True).array if packed is not None else None
    _call("gar_thc_allreduce_fused_masked", xt.array, len(xt), arrived, xt.numel, b, seed, _dev(d_mM), _dev(avg),
          pk, _stream(stream))


def thc_plan_tables(src, out, packed=None):
    """Host pointer tables for gar_thc_allreduce_fused_plan (reuse them across steps):
    src[w][i] worker w's tensor i, out[i] output tensor i, packed[w][b] or None."""
    return (PtrTable([t for row in src for t in row]), PtrTable(out),
            PtrTable([t for row in packed for t in row]) if packed is not None else None)


def gar_thc_allreduce_fused_plan(src, plan: FusionPlan, b: int, seed: int, d_mM, out, packed=None, stream=None,
                                 tables=None):
    """Uniform THC of every fusion buffer of `plan`, reading the workers'
    tensors src[w][i] directly and writing the average to out[i]; d_mM is the
    [n_buffers, 2] per-buffer range; packed[w][b] optionally receives worker
    w's indices of buffer b."""
    s, o, pk = tables if tables is not None else thc_plan_tables(src, out, packed)
    P = len(s) // max(plan.count, 1)
    _call("gar_thc_allreduce_fused_plan", s.array, P, C.addressof(plan.segs), plan.dtype.ctypes.data, plan.count,
          plan.buf_numel.ctypes.data, plan.n_buffers, b, seed, _dev(d_mM), o.array,
          pk.array if pk is not None else None, _stream(stream))


def gar_thc_plan_nmse_workspace_bytes(plan: FusionPlan, b: int) -> int:
    return int(load().gar_thc_plan_nmse_workspace_bytes(plan.buf_numel.ctypes.data, plan.n_buffers, plan.count, b))


def gar_thc_allreduce_fused_plan_nmse(src, plan: FusionPlan, b: int, seed: int, d_mM, out, ref, d_pair, workspace,
                                      packed=None, stream=None, tables=None, ref_table=None):
    """gar_thc_allreduce_fused_plan that also writes d_pair (2 fp64, device) =
    (sum (ref - avg)^2, sum ref^2) over the call's tensors; ref[i] is the
    reference tensor of tensor i (e.g. the ring average)."""
    s, o, pk = tables if tables is not None else thc_plan_tables(src, out, packed)
    r = ref_table if ref_table is not None else PtrTable(ref)
    P = len(s) // max(plan.count, 1)
    nbytes = workspace.numel() * workspace.element_size()
    _call("gar_thc_allreduce_fused_plan_nmse", s.array, P, C.addressof(plan.segs), plan.dtype.ctypes.data, plan.count,
          plan.buf_numel.ctypes.data, plan.n_buffers, b, seed, _dev(d_mM), o.array,
          pk.array if pk is not None else None, r.array, _dev(d_pair), _dev(workspace), nbytes, _stream(stream))


# --------------------------------------------------------- non-uniform THC
def _table(table):
    t = np.ascontiguousarray(table, np.uint16)
    return t, t.ctypes.data


def gar_nuhc_encode(x, d_mM, b: int, g: int, table, seed: int, worker: int, packed, stream=None):
    t, tp = _table(table)
    _call("gar_nuhc_encode", _dev(x), x.numel(), _dev(d_mM), b, g, tp, seed, worker, _dev(packed), _stream(stream))


def gar_nuhc_aggregate(packed, N: int, b: int, table, sums, stream=None):
    t, tp = _table(table)
    pt = pointer_table(packed)
    _call("gar_nuhc_aggregate", pt.array, len(pt), N, b, tp, _dev(sums), _stream(stream))


def gar_nuhc_decode(sums, d_mM, g: int, P: int, avg, stream=None):
    _call("gar_nuhc_decode", _dev(sums), sums.numel(), _dev(d_mM), g, P, _dev(avg), _stream(stream))


def gar_nuhc_allreduce_fused(x, b: int, g: int, table, seed: int, d_mM, avg, packed=None, stream=None):
    t, tp = _table(table)
    xt = pointer_table(x)
    pk = pointer_table(packed).array if packed is not None else None
    _call("gar_nuhc_allreduce_fused", xt.array, len(xt), xt.numel, b, g, tp, seed, _dev(d_mM), _dev(avg), pk,
          _stream(stream))


def gar_nuhc_allreduce_fused_masked(x, arrived: int, b: int, g: int, table, seed: int, d_mM, avg, packed=None,
                                    stream=None):
    """Non-uniform THC round over the workers whose bit is set in `arrived`
    (stragglers dropped); x[w] / packed[w] of the others may be None."""
    t, tp = _table(table)
    xt = pointer_table(x, allow_none=True)
    pk = pointer_table(packed, allow_none=True).array if packed is not None else None
    _call("gar_nuhc_allreduce_fused_masked", xt.array, len(xt), arrived, xt.numel, b, g, tp, seed, _dev(d_mM),
          _dev(avg), pk, _stream(stream))


# ------------------------------------------- RHT, range and error feedback
def gar_rht(x, out, seed: int, inverse: bool = False, stream=None):
    """out = (1/sqrt n) H D x, or (1/sqrt n) D H x with inverse=True; out may be x."""
    _call("gar_rht", _dev(x), _dev(out), x.numel(), seed, int(bool(inverse)), _stream(stream))


def gar_rht_norm_range_workspace_bytes(P: int, n: int) -> int:
    return int(load().gar_rht_norm_range_workspace_bytes(P, n))


def gar_rht_norm_range(x, t_p: float, d_mM, workspace, stream=None):
    t = pointer_table(x)
    nbytes = workspace.numel() * workspace.element_size()
    _call("gar_rht_norm_range", t.array, len(t), t.numel, float(t_p), _dev(d_mM), _dev(workspace), nbytes,
          _stream(stream))


def gar_rht_tiles(n: int) -> int:
    return int(load().gar_rht_tiles(n))


def gar_rht_ef_forward(grad, e, y, seed: int, sumsq=None, stream=None):
    """y = (1/sqrt n) H D (grad + e); sumsq (fp64, gar_rht_tiles(n)) receives
    the per-tile sums of squares of grad + e if given."""
    _call("gar_rht_ef_forward", _dev(grad), _dev(e), _dev(y), grad.numel(), seed,
          _dev(sumsq) if sumsq is not None else None, _stream(stream))


def gar_rht_norm_range_from_sums(sumsq, n: int, t_p: float, d_mM, stream=None):
    """The norm-based range from the workers' per-tile sums (a list of fp64 tensors)."""
    t = pointer_table(sumsq)
    _call("gar_rht_norm_range_from_sums", t.array, len(t), n, float(t_p), _dev(d_mM), _stream(stream))


def gar_rht_ef_update(packed, b: int, steps: int, table, d_mM, grad, e, tmp, seed: int, stream=None):
    """e = (grad + e) - (1/sqrt n) D H decode(packed); table None for uniform THC (steps = 2^b - 1)."""
    tp = None
    if table is not None:
        t, tp = _table(table)
    _call("gar_rht_ef_update", _dev(packed), b, steps, tp, _dev(d_mM), _dev(grad), _dev(e), _dev(tmp), e.numel(),
          seed, _stream(stream))


def gar_ef_apply(grad, e, x, stream=None):
    _call("gar_ef_apply", _dev(grad), _dev(e), _dev(x), grad.numel(), _stream(stream))


def gar_ef_update(e, x, x_hat, stream=None):
    _call("gar_ef_update", _dev(e), _dev(x), _dev(x_hat), e.numel(), _stream(stream))


# -------------------------------------------------------------------- NMSE
def gar_nmse_workspace_bytes(N: int) -> int:
    return int(load().gar_nmse_workspace_bytes(N))


def gar_nmse(x, x_hat, d_out, workspace, stream=None):
    nbytes = workspace.numel() * workspace.element_size()
    _call("gar_nmse", _dev(x), _dev(x_hat), x.numel(), _dev(d_out), _dev(workspace), nbytes, _stream(stream))


def gar_nmse_sums(x, x_hat, d_pair, workspace, stream=None):
    """(sum (x - x_hat)^2, sum x^2) of one range into d_pair (2 fp64, device)."""
    nbytes = workspace.numel() * workspace.element_size()
    _call("gar_nmse_sums", _dev(x), _dev(x_hat), x.numel(), _dev(d_pair), _dev(workspace), nbytes, _stream(stream))


def gar_nmse_combine(d_pairs, d_out, stream=None):
    """NMSE from the pairs of gar_nmse_sums (d_pairs: [n, 2] fp64, device)."""
    _call("gar_nmse_combine", _dev(d_pairs), d_pairs.numel() // 2, _dev(d_out), _stream(stream))


def gar_nmse_noalloc(x, x_hat, d_out, stream=None):
    """NMSE without a workspace, for callers that may not allocate device
    memory: partial sums go to a fixed array inside the library (see gar.h)."""
    _call("gar_nmse_noalloc", _dev(x), _dev(x_hat), x.numel(), _dev(d_out), _stream(stream))


# ------------------------------------- a worker's products and losses: 8-bit
def fp8_matrix(rows: int, cols: int, dtype=None, device="cuda"):
    """(codes, scales) of a rows x cols block-scaled 8-bit matrix, uninitialised:
    codes are a [rows, cols] view (torch.float8_e4m3fn unless ``dtype`` is
    float8_e5m2) whose rows start on 16 bytes, scales uint8 [ceil(cols / 512),
    rows, 4]."""
    import torch

    ld = (cols + 15) // 16 * 16
    codes = torch.empty((rows, ld), dtype=torch.uint8, device=device).view(dtype or torch.float8_e4m3fn)[:, :cols]
    return codes, torch.empty(((cols + 511) // 512, rows, 4), dtype=torch.uint8, device=device)


# torch's types by what the library calls them; filled on first use, so that the package imports without torch
_FLOATS, _FP8S, _INT32, _FLOAT32, _UINT8 = {}, {}, None, None, None


def _types():
    import torch

    global _INT32, _FLOAT32, _UINT8
    _INT32, _FLOAT32, _UINT8 = torch.int32, torch.float32, torch.uint8
    _FP8S.update({torch.float8_e4m3fn: GAR_F8E4M3, torch.float8_e5m2: GAR_F8E5M2})
    _FLOATS.update({torch.float32: GAR_F32, torch.bfloat16: GAR_BF16})


def _code(t, table, name):
    if not _FLOATS:
        _types()
    code = table.get(t.dtype)
    if code is None:
        raise GarError(GAR_EDTYPE, f"{name} is {t.dtype}, not one of {', '.join(map(str, table))}")
    return code


def _matrix(t, name, rows, cols):
    """(pointer, row stride) of a rows x cols CUDA tensor whose rows are contiguous."""
    if t.shape != (rows, cols):
        raise GarError(GAR_EINVAL, f"{name} has shape {tuple(t.shape)}, not {(rows, cols)}")
    ld, inner = t.stride()
    if inner != 1 and cols > 1:
        raise GarError(GAR_EINVAL, f"{name}: the elements of a row are not contiguous")
    # the stride of a single row means nothing: one that the library accepts
    return _dev(t), ld if rows > 1 else (cols + 15) // 16 * 16


def _vector(t, name, dtype, n):
    if t.dtype != dtype:
        raise GarError(GAR_EDTYPE, f"{name} is {t.dtype}, not {dtype}")
    if t.numel() != n or not t.is_contiguous():
        raise GarError(GAR_EINVAL, f"{name} is not a contiguous tensor of {n} elements")
    return _dev(t)


def _two_dims(t, name):
    if t.dim() != 2:
        raise GarError(GAR_EINVAL, f"{name} has {t.dim()} dimensions, not two")
    return t.shape


def gar_fp8_scale_bytes(rows: int, cols: int) -> int:
    return int(load().gar_fp8_scale_bytes(rows, cols))


def gar_fp8_quantize(x, q, scale, qt=None, scale_t=None, square: bool = False, stream=None):
    """Codes and scales of x [rows, cols] (fp32 or bf16): q [rows, cols] with
    ``scale``, and/or qt [cols, rows], the transpose's, with ``scale_t`` (see
    fp8_matrix; either pair may be None).  square: 128 x 128 blocks instead of
    128 along the summed axis."""
    dtype = _code(x, _FLOATS, "x")
    rows, cols = _two_dims(x, "x")
    fmt = qp = sp = qtp = stp = None
    ldq = ldqt = 0
    if q is not None:
        fmt = _code(q, _FP8S, "q")
    if qt is not None:
        f = _code(qt, _FP8S, "qt")
        if fmt is not None and f != fmt:
            raise GarError(GAR_EDTYPE, "q and qt have different formats")
        fmt = f
    xp, ldx = _matrix(x, "x", rows, cols)
    if q is not None:
        qp, ldq = _matrix(q, "q", rows, cols)
        sp = _vector(scale, "scale", _UINT8, (cols + 511) // 512 * rows * 4) if scale is not None else None
    if qt is not None:
        qtp, ldqt = _matrix(qt, "qt", cols, rows)
        stp = _vector(scale_t, "scale_t", _UINT8, (rows + 511) // 512 * cols * 4) if scale_t is not None else None
    _call("gar_fp8_quantize", xp, dtype, rows, cols, ldx, fmt or 0, 1 if square else 0, qp, ldq, sp, qtp, ldqt, stp,
          _stream(stream))


def gar_fp8_matmul(a, a_scale, b, b_scale, d, c=None, stream=None):
    """d = a b^T (+ c): a [M, K] and b [N, K] codes with their scales, d [M, N]
    fp32 or bf16, c of d's type (it may be d)."""
    fmt_a, fmt_b, dtype = _code(a, _FP8S, "a"), _code(b, _FP8S, "b"), _code(d, _FLOATS, "d")
    M, K = _two_dims(a, "a")
    N = _two_dims(b, "b")[0]
    ap, lda = _matrix(a, "a", M, K)
    bp, ldb = _matrix(b, "b", N, K)
    dp, ldd = _matrix(d, "d", M, N)
    words = (K + 511) // 512 * 4
    asp = _vector(a_scale, "a_scale", _UINT8, words * M)
    bsp = _vector(b_scale, "b_scale", _UINT8, words * N)
    cp, ldc = None, 0
    if c is not None:
        if c.dtype != d.dtype:
            raise GarError(GAR_EDTYPE, f"c is {c.dtype}, d {d.dtype}")
        cp, ldc = _matrix(c, "c", M, N)
    _call("gar_fp8_matmul", ap, lda, asp, fmt_a, bp, ldb, bsp, fmt_b, M, N, K, cp, ldc, dp, ldd, dtype, _stream(stream))


def _distill_args(z, index, teacher, tau, weight, dz):
    dtype = _code(z, _FLOATS, "z")
    rows, vocab = _two_dims(z, "z")
    k = index.shape[-1] if index.dim() else 0
    zp, ldz = _matrix(z, "z", rows, vocab)
    dzp, lddz = None, 0
    if dz is not None:
        if dz.dtype != z.dtype:
            raise GarError(GAR_EDTYPE, f"dz is {dz.dtype}, z {z.dtype}")
        dzp, lddz = _matrix(dz, "dz", rows, vocab)
    head = (zp, dtype, rows, vocab, ldz, _vector(index, "index", _INT32, rows * k),
            _vector(teacher, "teacher", _FLOAT32, rows * k), k, tau,
            None if weight is None else _vector(weight, "weight", _FLOAT32, rows))
    return rows, head, dzp, lddz


def gar_distill_loss(z, index, teacher, tau: float, loss, lse, dz=None, weight=None, stream=None):
    """Distillation loss of student logits z [rows, vocab] against the teacher's
    top logits (index, teacher [rows, k]) at temperature tau: loss and lse
    [rows], and the gradient dz (z's type; may be z) under the rows' weights."""
    rows, head, dzp, lddz = _distill_args(z, index, teacher, tau, weight, dz)
    _call("gar_distill_loss", *head, _vector(loss, "loss", _FLOAT32, rows), _vector(lse, "lse", _FLOAT32, rows), dzp, lddz,
          _stream(stream))


def gar_distill_grad(z, index, teacher, tau: float, lse, dz, weight=None, stream=None):
    """The gradient of gar_distill_loss alone, from its lse."""
    rows, head, dzp, lddz = _distill_args(z, index, teacher, tau, weight, dz)
    _call("gar_distill_grad", *head, _vector(lse, "lse", _FLOAT32, rows), dzp, lddz, _stream(stream))


def gar_balance_workspace_bytes(P: int) -> int:
    return int(load().gar_balance_workspace_bytes(P))


def _worker_fits(t, name, shape, stride, dtype):
    """Whether one worker's tensor is as asked; what _workers' quick comparison turned down may still be."""
    if t is None:
        raise GarError(GAR_EINVAL, f"{name} lacks a worker's tensor")
    if not t.is_cuda:
        _dev(t)
    if t.dtype != dtype and not (dtype is _UINT8 and t.element_size() == 1):
        raise GarError(GAR_EDTYPE, f"{name} is {t.dtype}, not {dtype}")
    # one token's row stride means nothing, the stride of its elements does
    if t.shape != shape or (t.stride() != stride if shape[0] > 1 else t.stride()[-1] != 1 and shape[-1] > 1):
        raise GarError(GAR_EINVAL, f"{name} has a tensor of shape {tuple(t.shape)}, not {shape}, or of another stride")


def _workers(given, name, P, shape, dtype):
    """(pointers, row stride) of one tensor per worker, each of the given shape
    and type and all of one row stride.  A PtrTable's tensors are looked at once
    for each shape and type asked of them."""
    table = isinstance(given, PtrTable)
    if table and given.last is not None and given.last[0] == (P, shape, dtype):
        return given.last[1]
    tensors = given.tensors if table else given
    if len(tensors) != P:
        raise GarError(GAR_EINVAL, f"{name} has {len(tensors)} tensors, not {P}")
    stride = given.checked.get((shape, dtype)) if table else None
    if stride is None:
        if tensors[0] is None:
            _worker_fits(None, name, shape, None, dtype)
        stride, ptrs = tensors[0].stride(), []
        for t in tensors:
            if t is None or t.dtype is not dtype or t.shape != shape or not t.is_cuda or t.stride() != stride:
                _worker_fits(t, name, shape, stride, dtype)
            ptrs.append(t.data_ptr())
        if table:
            given.checked[shape, dtype] = stride
    if stride[-1] != 1 and shape[-1] > 1 and shape[0] > 0:
        raise GarError(GAR_EINVAL, f"{name}: the elements of a row are not contiguous")
    found = given.array if table else struct.pack(f"{P}Q", *ptrs), stride[0] if shape[0] > 1 else max(shape[-1], 1)
    if table:
        given.last = (P, shape, dtype), found
    return found


def gar_balance_loss(z, k: int, alpha: float, choice, counts, loss, workspace, dz=None, valid=None, stream=None):
    """A router's choices, counts and balance loss over P workers.  z[w]
    [tokens, experts] logits, choice[w] [tokens, k] int32 out, counts [P,
    experts] int32 out, loss one fp32 out, dz[w] of z's type out (may be z[w]),
    valid[w] [tokens] uint8 or bool.  Lists or PtrTables."""
    first = z.first if isinstance(z, PtrTable) else z[0] if len(z) else None
    if first is None:
        raise GarError(GAR_EINVAL, "z has no worker's tensor")
    dtype = _code(first, _FLOATS, "z")
    P, (tokens, experts) = len(z), _two_dims(first, "z[0]")
    za, ldz = _workers(z, "z", P, (tokens, experts), first.dtype)
    ca, ldc = _workers(choice, "choice", P, (tokens, k), _INT32)
    da, lddz = _workers(dz, "dz", P, (tokens, experts), first.dtype) if dz is not None else (None, 0)
    va = _workers(valid, "valid", P, (tokens,), _UINT8)[0] if valid is not None else None
    if ldc != k:
        raise GarError(GAR_EINVAL, "choice has to be contiguous")
    _call("gar_balance_loss", za, P, tokens, experts, ldz, dtype, k, va, alpha, ca,
          _vector(counts, "counts", _INT32, P * experts), _vector(loss, "loss", _FLOAT32, 1), da, lddz, _dev(workspace),
          workspace.numel() * workspace.element_size(), _stream(stream))


# --------------------------------- the vocabulary layer's cross entropy
def gar_vocab_workspace_bytes(rows: int, vocab: int, hidden: int, dw_dtype=None) -> int:
    """Bytes for gar_vocab_loss and gar_vocab_grad; dw_dtype: torch.float32 or
    bfloat16 (None: bfloat16)."""
    if not _FLOATS:
        _types()
    if dw_dtype is not None and dw_dtype not in _FLOATS:
        raise GarError(GAR_EDTYPE, f"dw is {dw_dtype}, not one of {', '.join(map(str, _FLOATS))}")
    return int(load().gar_vocab_workspace_bytes(rows, vocab, hidden, GAR_BF16 if dw_dtype is None else _FLOATS[dw_dtype]))


def _vocab_args(x, w, target, weight):
    dtype = _code(x, _FLOATS, "x")
    if w.dtype != x.dtype:
        raise GarError(GAR_EDTYPE, f"w is {w.dtype}, x {x.dtype}")
    rows, hidden = _two_dims(x, "x")
    vocab = _two_dims(w, "w")[0]
    xp, ldx = _matrix(x, "x", rows, hidden)
    wp, ldw = _matrix(w, "w", vocab, hidden)
    return rows, vocab, hidden, (xp, ldx, wp, ldw, dtype, _vector(target, "target", _INT32, rows),
                                 None if weight is None else _vector(weight, "weight", _FLOAT32, rows), rows, vocab, hidden)


def gar_vocab_loss(x, w, target, loss, lse, workspace, weight=None, stream=None):
    """Cross entropy of a vocabulary layer, logits x w^T, without its logits: x
    [rows, hidden] and w [vocab, hidden] bf16, target [rows] int32; loss and lse
    [rows] fp32.  Rows with a target outside the vocabulary or weight 0 do not
    count (0)."""
    rows, _, _, head = _vocab_args(x, w, target, weight)
    _call("gar_vocab_loss", *head, _vector(loss, "loss", _FLOAT32, rows), _vector(lse, "lse", _FLOAT32, rows),
          _dev(workspace), workspace.numel() * workspace.element_size(), _stream(stream))


def _vocab_outputs(x, dx, dw, addend, rows, vocab, hidden, workspace, stream):
    dxp = dwp = ap = None
    lddx = lddw = lda = 0
    dw_type = GAR_BF16
    if dx is not None:
        if dx.dtype != x.dtype:
            raise GarError(GAR_EDTYPE, f"dx is {dx.dtype}, x {x.dtype}")
        dxp, lddx = _matrix(dx, "dx", rows, hidden)
    if dw is not None:
        dw_type = _code(dw, _FLOATS, "dw")
        dwp, lddw = _matrix(dw, "dw", vocab, hidden)
    if addend is not None:
        if dw is None or addend.dtype != dw.dtype:
            raise GarError(GAR_EDTYPE, f"addend is {addend.dtype}, dw {None if dw is None else dw.dtype}")
        ap, lda = _matrix(addend, "addend", vocab, hidden)
    return (dxp, lddx, ap, lda, dwp, lddw, dw_type), (_dev(workspace), workspace.numel() * workspace.element_size(), _stream(stream))


def gar_vocab_grad(x, w, target, lse, dx, dw, workspace, weight=None, addend=None, stream=None):
    """The gradient of sum(weight * loss) from the lse of gar_vocab_loss: dx
    [rows, hidden] bf16 and dw [vocab, hidden] fp32 or bf16 (either may be None);
    addend, of dw's type, is added to dw (it may be dw).  lse alone does not hold
    the share of a target that is all but sure (gar_vocab_grad_with_loss)."""
    rows, vocab, hidden, head = _vocab_args(x, w, target, weight)
    out, tail = _vocab_outputs(x, dx, dw, addend, rows, vocab, hidden, workspace, stream)
    _call("gar_vocab_grad", *head, _vector(lse, "lse", _FLOAT32, rows), *out, *tail)


def gar_vocab_grad_with_loss(x, w, target, loss, lse, dx, dw, workspace, weight=None, addend=None, parts: int = 0, stream=None):
    """The same gradient from the loss and lse of gar_vocab_loss: each target's share
    keeps its digits, however small its loss.  parts=2: dx and a bf16 dw too from
    all of g's bits, at twice their products' cost (the workspace of an fp32 dw)."""
    rows, vocab, hidden, head = _vocab_args(x, w, target, weight)
    out, tail = _vocab_outputs(x, dx, dw, addend, rows, vocab, hidden, workspace, stream)
    _call("gar_vocab_grad_with_loss", *head, _vector(loss, "loss", _FLOAT32, rows), _vector(lse, "lse", _FLOAT32, rows), *out, parts,
          *tail)


# ------------------------------------------- tokens to experts and back
def gar_expert_rows(P: int, tokens: int, k: int, experts: int, align: int = 1, capacity: int = 0) -> int:
    """Rows of the experts' buffer that any choices of P workers' tokens fit in."""
    rows = int(load().gar_expert_rows(P, tokens, k, experts, align, capacity))
    if rows < 0:
        raise GarError(GAR_EINVAL, f"P={P} tokens={tokens} k={k} experts={experts} align={align} capacity={capacity}")
    return rows


def gar_expert_workspace_bytes(P: int, tokens: int, k: int, experts: int) -> int:
    return int(load().gar_expert_workspace_bytes(P, tokens, k, experts))


def _first(given, name):
    """The first worker's tensor, of two dimensions."""
    if isinstance(given, PtrTable):
        if given.size is not None:
            return given.first, *given.size
        t = given.first
    else:
        t = given[0] if len(given) else None
    if t is None:
        raise GarError(GAR_EINVAL, f"{name} has no worker's tensor")
    return t, *_two_dims(t, name)


def _per_choice(given, name, P, tokens, k, dtype):
    """The pointers of one [tokens, k] tensor per worker, contiguous."""
    table, ld = _workers(given, name, P, (tokens, k), dtype)
    if ld != k:
        raise GarError(GAR_EINVAL, f"{name} has to be contiguous")
    return table


def gar_expert_sort(choice, experts: int, position, source, offsets, workspace, align: int = 1, capacity: int = 0, stream=None):
    """Rows of the pairs (worker, token, choice) sorted by expert: choice[w]
    [tokens, k] int32 in, position[w] [tokens, k] int32, source [rows] int32 and
    offsets [experts + 1] int32 out.  Each expert's rows are filled up to a
    multiple of align, or are capacity rows, what is over them dropped."""
    if not _FLOATS:
        _types()
    _, tokens, k = _first(choice, "choice")
    P, rows = len(choice), source.numel()
    _call("gar_expert_sort", _per_choice(choice, "choice", P, tokens, k, _INT32), P, tokens, k, experts, align, capacity,
          _per_choice(position, "position", P, tokens, k, _INT32), _vector(source, "source", _INT32, rows), rows,
          _vector(offsets, "offsets", _INT32, experts + 1), _dev(workspace), workspace.numel() * workspace.element_size(),
          _stream(stream))


def gar_expert_gather(x, position, source, y, weight=None, stream=None):
    """y[position[w][t, j]] = x[w][t] (times weight[w][t, j]); an expert's rows
    without a token become 0.  x[w] [tokens, hidden], y [rows, hidden]."""
    first, tokens, hidden = _first(x, "x")
    dtype, P, rows, k = _code(first, _FLOATS, "x"), len(x), source.numel(), _first(position, "position")[2]
    if y.dtype != first.dtype:
        raise GarError(GAR_EDTYPE, f"y is {y.dtype}, x {first.dtype}")
    xa, ldx = _workers(x, "x", P, (tokens, hidden), first.dtype)
    yp, ldy = _matrix(y, "y", rows, hidden)
    wa = _per_choice(weight, "weight", P, tokens, k, _FLOAT32) if weight is not None else None
    _call("gar_expert_gather", xa, P, tokens, hidden, ldx, dtype, k, _per_choice(position, "position", P, tokens, k, _INT32),
          _vector(source, "source", _INT32, rows), rows, wa, yp, ldy, _stream(stream))


def gar_expert_combine(y, position, out, weight=None, addend=None, stream=None):
    """out[w][t] = addend[w][t] + sum_j weight[w][t, j] y[position[w][t, j]] (weight
    None: 1; addend None: 0; it may be out)."""
    first, tokens, hidden = _first(out, "out")
    dtype, P, k = _code(first, _FLOATS, "out"), len(out), _first(position, "position")[2]
    if y.dtype != first.dtype:
        raise GarError(GAR_EDTYPE, f"y is {y.dtype}, out {first.dtype}")
    rows = _two_dims(y, "y")[0]
    yp, ldy = _matrix(y, "y", rows, hidden)
    oa, ldo = _workers(out, "out", P, (tokens, hidden), first.dtype)
    aa, lda = _workers(addend, "addend", P, (tokens, hidden), first.dtype) if addend is not None else (None, 0)
    wa = _per_choice(weight, "weight", P, tokens, k, _FLOAT32) if weight is not None else None
    _call("gar_expert_combine", yp, ldy, rows, P, tokens, hidden, dtype, k,
          _per_choice(position, "position", P, tokens, k, _INT32), wa, aa, lda, oa, ldo, _stream(stream))


def gar_expert_combine_grad(dout, y, position, source, weight, dy, dweight, stream=None):
    """The gradient of gar_expert_combine: dy[position] = weight dout (rows without
    a token 0), dweight[w][t, j] = <dout[w][t], y[position[w][t, j]]>; dy may be y."""
    first, tokens, hidden = _first(dout, "dout")
    dtype, P, rows, k = _code(first, _FLOATS, "dout"), len(dout), source.numel(), _first(position, "position")[2]
    if y.dtype != first.dtype or dy.dtype != first.dtype:
        raise GarError(GAR_EDTYPE, f"y is {y.dtype}, dy {dy.dtype}, dout {first.dtype}")
    da, ldd = _workers(dout, "dout", P, (tokens, hidden), first.dtype)
    yp, ldy = _matrix(y, "y", rows, hidden)
    gp, ldg = _matrix(dy, "dy", rows, hidden)
    _call("gar_expert_combine_grad", da, ldd, yp, ldy, P, tokens, hidden, dtype, k,
          _per_choice(position, "position", P, tokens, k, _INT32), _vector(source, "source", _INT32, rows), rows,
          _per_choice(weight, "weight", P, tokens, k, _FLOAT32), gp, ldg,
          _per_choice(dweight, "dweight", P, tokens, k, _FLOAT32), _stream(stream))


def gar_expert_weights(z, choice, weight, stream=None):
    """weight[w][t, j]: the softmax over the token's chosen logits z[w][t, choice]
    (a choice of -1 has weight 0)."""
    first, tokens, experts = _first(z, "z")
    dtype, P, k = _code(first, _FLOATS, "z"), len(z), _first(choice, "choice")[2]
    za, ldz = _workers(z, "z", P, (tokens, experts), first.dtype)
    _call("gar_expert_weights", za, P, tokens, experts, ldz, dtype, k, _per_choice(choice, "choice", P, tokens, k, _INT32),
          _per_choice(weight, "weight", P, tokens, k, _FLOAT32), _stream(stream))


def gar_expert_weights_grad(weight, dweight, choice, dz, accumulate: bool = False, stream=None):
    """The gradient of gar_expert_weights over the router's logits: dz[w] [tokens,
    experts], 0 where an expert was not chosen; accumulate: added to dz."""
    first, tokens, experts = _first(dz, "dz")
    dtype, P, k = _code(first, _FLOATS, "dz"), len(dz), _first(choice, "choice")[2]
    da, ldd = _workers(dz, "dz", P, (tokens, experts), first.dtype)
    _call("gar_expert_weights_grad", _per_choice(weight, "weight", P, tokens, k, _FLOAT32),
          _per_choice(dweight, "dweight", P, tokens, k, _FLOAT32), P, tokens, experts, k,
          _per_choice(choice, "choice", P, tokens, k, _INT32), da, ldd, dtype, 1 if accumulate else 0, _stream(stream))


# ------------------------------------------------- gradient norm, clipping
class GradTables:
    """Host tables of P workers' gradient tensors, built once: grads[w][i], and the
    tensors that the clipped ones go to (the same ones unless given).  Building them
    takes the host about half a microsecond a tensor, more than clipping does where they
    are small: kept, as long as the gradients stay where they are.  With norm_only
    they go nowhere (gar_grad_norm), and a tensor may stand in the lists more than once."""

    def __init__(self, grads, out=None, norm_only: bool = False):
        self.P = len(grads)
        self.count = len(grads[0]) if self.P else 0
        self.src = self._table(grads, "grads")
        self.dst = None if norm_only else self.src if out is None else self._table(out, "out")
        first = self.src.tensors[:self.count]
        types, sizes = [t.dtype for t in first], [t.numel() for t in first]
        self.dtype = np.array([_dtype_code(t) for t in first], np.int32)
        self.numel = np.array(sizes, np.int64)
        self.host = self.numel.ctypes.data, self.dtype.ctypes.data
        for name, table in (("grads", self.src),) if out is None else (("grads", self.src), ("out", self.dst)):
            if [t.dtype for t in table.tensors] != types * self.P:
                raise GarError(GAR_EDTYPE, f"{name}: a tensor is not of the type of the first worker's")
            if [t.numel() for t in table.tensors] != sizes * self.P or not all([t.is_contiguous() for t in table.tensors]):
                raise GarError(GAR_EINVAL, f"{name}: a tensor is not contiguous, or not of the size of the first worker's")
        places = [] if norm_only else [p for p, n in zip(self.dst.array, sizes * self.P) if n]
        if len(set(places)) < len(places):
            raise GarError(GAR_EINVAL, "the same tensor stands twice in the lists: it would be scaled twice")

    def _table(self, rows, name):
        if not 1 <= self.P <= GAR_MAX_WORKERS or len(rows) != self.P or any(len(r) != self.count for r in rows):
            raise GarError(GAR_EINVAL, f"{name}: {len(rows)} workers' lists, not all of {self.count} tensors")
        return PtrTable([t for r in rows for t in r])


def grad_tables(grads, out=None, norm_only: bool = False) -> GradTables:
    if out is not None and (norm_only or isinstance(grads, GradTables)):
        raise GarError(GAR_EINVAL, "out is for lists of tensors to be clipped: tables say where theirs go, a norm writes none")
    return grads if isinstance(grads, GradTables) else GradTables(grads, out, norm_only)


def gar_grad_workspace_bytes(grads) -> int:
    t = grad_tables(grads, norm_only=True)
    return int(load().gar_grad_workspace_bytes(t.P, t.count))


def gar_grad_norm(grads, norm, workspace, stream=None):
    """norm[w] = the 2-norm of worker w's gradient tensors grads[w][i] (lists, or
    grad_tables), [P] fp32.  A tensor that stands twice counts twice."""
    t = grad_tables(grads, norm_only=True)
    _call("gar_grad_norm", t.src.array, t.P, *t.host, t.count,
          _vector(norm, "norm", _float32(), t.P), _dev(workspace), workspace.numel() * workspace.element_size(),
          _stream(stream))


def gar_grad_clip(grads, max_norm: float, norm, workspace, out=None, shared: bool = False, stream=None):
    """Each worker's gradients times min(1, max_norm / norm[w]), in place or to
    out[w][i] (tables: to what they were built with); shared: by the norm of the
    first worker's, norm [1].  A norm that is not finite leaves them as they are."""
    t = grad_tables(grads, out)
    if t.dst is None:
        raise GarError(GAR_EINVAL, "the tables are for the norm alone")
    _call("gar_grad_clip", t.src.array, t.dst.array, t.P, *t.host, t.count,
          1 if shared else 0, max_norm, _vector(norm, "norm", _float32(), 1 if shared else t.P), _dev(workspace),
          workspace.numel() * workspace.element_size(), _stream(stream))


def _float32():
    if _FLOAT32 is None:
        _types()
    return _FLOAT32


__all__ = [n for n in dir() if n.startswith(("gar_", "GAR_"))] + ["GarError", "FusionPlan", "PtrTable", "load",
                                                                    "pointer_table", "fused_pointer_tables", "thc_plan_tables",
                                                                    "fp8_matrix", "GradTables", "grad_tables",
                                                                    "Timeline", "timeline"]
