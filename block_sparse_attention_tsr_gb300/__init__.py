"""GB300 block-sparse attention forward -- Python binding of ``libtsr_gb300.so``.

Argument marshalling only: every step (planning, permutation, attention) runs
in the library's CUDA kernels, reached through the C ABI of ``include/tsr.h``.
There is no CPU path; without the built library every call raises.

The names follow the C ABI:

    mask = make_mask(kind, B, H, N, d, blocks=..., bq=64, bk=64)   # device tensors
    plan = tsr_plan(mask)                                            # physical tile plan
    out, lse = tsr_bsa_forward(q, k, v, plan)                        # bf16 O, fp32 lse
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import struct
from typing import Optional

import torch

from . import _build

__all__ = [
    "TsrError", "build", "lib", "make_mask", "Mask", "Plan", "tsr_plan", "tsr_plan_update",
    "tsr_bsa_forward",
    "tsr_bsa_forward_batch", "tsr_plan_device_status", "tsr_temporal_permute", "tsr_svg_route",
    "tsr_rope", "tsr_rope_backward", "tsr_block_select",
    "BackwardPlan", "tsr_backward_plan", "tsr_backward_plan_update", "tsr_bsa_backward",
    "tsr_attention_host",
    "tsr_regime_load",
    "tsr_regime_lookup", "tsr_abi_version", "UNIFORM", "SEGMENTS", "SVG", "KEYLIST",
    "ORIENT_ROWS", "ORIENT_KEYS",
    "PLAN_SYNC_CHECK", "PLAN_NO_LPT", "PLAN_TEST_STALL", "PLAN_DEBUG_CHECKS",
    "PLAN_TEMPORAL_TILES",
]

UNIFORM, SEGMENTS, SVG, KEYLIST = 0, 1, 2, 3
ORIENT_ROWS, ORIENT_KEYS = 1, 2
PLAN_SYNC_CHECK, PLAN_NO_LPT, PLAN_TEST_STALL, PLAN_DEBUG_CHECKS = 1, 2, 4, 8
PLAN_TEMPORAL_TILES = 16
_STATUS = {0: "ok", 1: "invalid argument", 2: "unsupported", 3: "CUDA error", 4: "out of memory",
           5: "device wait timed out", 6: "internal error"}

REGIME_TABLE = os.path.join(os.path.dirname(os.path.abspath(__file__)), "regimes_gb300.txt")


class TsrError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{_STATUS.get(status, status)}: {message}")
        self.status = status


class _Mask(ctypes.Structure):
    _fields_ = [
        ("kind", ctypes.c_int32),
        ("B", ctypes.c_int32), ("H", ctypes.c_int32), ("N", ctypes.c_int32), ("d", ctypes.c_int32),
        ("bq", ctypes.c_int32), ("bk", ctypes.c_int32),
        ("n_qseg", ctypes.c_int32), ("n_kseg", ctypes.c_int32),
        ("q_bounds", ctypes.c_void_p), ("k_bounds", ctypes.c_void_p),
        ("blocks", ctypes.c_void_p),
        ("n_frames", ctypes.c_int32), ("frame_size", ctypes.c_int32),
        ("head_kind", ctypes.c_void_p),
        ("slice_m", ctypes.c_int32),
        ("indptr", ctypes.c_void_p), ("indices", ctypes.c_void_p),
        ("temporal_radius", ctypes.c_int32),
    ]


class _RopeDesc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("N", ctypes.c_int32), ("d", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("n_axes", ctypes.c_int32),
                ("axis_dim", ctypes.c_int32 * 4), ("halves", ctypes.c_int32),
                ("inverse", ctypes.c_int32), ("theta", ctypes.c_double),
                ("positions", ctypes.c_void_p), ("positions_per_batch", ctypes.c_int32),
                ("grid", ctypes.c_int32 * 4)]


class _RopeTensor(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("out", ctypes.c_void_p), ("H", ctypes.c_int32),
                ("x_stride", ctypes.c_int64 * 3), ("out_stride", ctypes.c_int64 * 3)]


class _SelectDesc(ctypes.Structure):
    _fields_ = [(f, ctypes.c_int32) for f in ("B", "H", "N", "d", "bq", "bk", "keep", "first", "diagonal")]


# The same layouts as packed bytes, which the calls below pass (filling a ctypes
# structure field by field takes longer than the kernels of a small call).
_ROPE_DESC = struct.Struct("@5i4i2idPi4i4x")
_ROPE_TENSOR = struct.Struct("@PPi3q3q")
_SELECT_DESC = struct.Struct("@9i")
for _packed, _fields in ((_ROPE_DESC, _RopeDesc), (_ROPE_TENSOR, _RopeTensor), (_SELECT_DESC, _SelectDesc)):
    assert _packed.size == ctypes.sizeof(_fields)


class _Request(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("plan", ctypes.c_void_p), ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p)]


class _Opts(ctypes.Structure):
    _fields_ = [("bn", ctypes.c_int32), ("stages", ctypes.c_int32),
                ("ctas_per_sm", ctypes.c_int32), ("flags", ctypes.c_int32),
                ("orient", ctypes.c_int32), ("kv_split", ctypes.c_int32)]


class _Stats(ctypes.Structure):
    _fields_ = [("bm", ctypes.c_int32), ("bn", ctypes.c_int32), ("stages", ctypes.c_int32),
                ("ctas_per_sm", ctypes.c_int32), ("gathered", ctypes.c_int32),
                ("n_temporal_heads", ctypes.c_int32), ("n_items", ctypes.c_int64),
                ("n_entries", ctypes.c_int64), ("n_boundary", ctypes.c_int64),
                ("n_logical_on", ctypes.c_int64), ("n_logical_total", ctypes.c_int64),
                ("max_item_len", ctypes.c_int64), ("regime_id", ctypes.c_int32),
                ("orient", ctypes.c_int32), ("kv_split", ctypes.c_int32),
                ("temporal_band", ctypes.c_int32)]


class _Regime(ctypes.Structure):
    _fields_ = [("bn", ctypes.c_int32), ("stages", ctypes.c_int32),
                ("ctas_per_sm", ctypes.c_int32), ("id", ctypes.c_int32), ("orient", ctypes.c_int32)]


_LIB = None
EXPORTS = ("tsr_abi_version", "tsr_status_string", "tsr_last_error", "tsr_plan", "tsr_plan_update",
           "tsr_bsa_forward", "tsr_bsa_forward_batch", "tsr_plan_device_status", "tsr_plan_destroy", "tsr_plan_get_stats",
           "tsr_plan_export", "tsr_temporal_permute", "tsr_svg_route", "tsr_rope",
           "tsr_block_select_workspace", "tsr_block_select", "tsr_backward_plan",
           "tsr_backward_plan_update", "tsr_backward_plan_destroy", "tsr_backward_plan_device_status",
           "tsr_backward_plan_test_stall",
           "tsr_bsa_backward_workspace", "tsr_bsa_backward", "tsr_attention_host",
           "tsr_release_host_buffers", "tsr_regime_load", "tsr_regime_lookup")


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile the CUDA library in-tree (sm_103a) and return its path."""
    return _build.build(force=force, verbose=verbose)


def lib_path() -> str:
    return _build.LIB


def lib():
    """The loaded library.  Raises if it has not been built."""
    global _LIB
    if _LIB is not None:
        return _LIB
    if not os.path.exists(_build.LIB):
        raise RuntimeError(f"the CUDA library is not built ({_build.LIB} missing): "
                           "call block_sparse_attention_tsr_gb300.build() first")
    L = ctypes.CDLL(_build.LIB)
    P, I32, I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    sig = {
        "tsr_abi_version": ([], I32),
        "tsr_status_string": ([ctypes.c_int], ctypes.c_char_p),
        "tsr_last_error": ([], ctypes.c_char_p),
        "tsr_plan": ([P, P, P, P], ctypes.c_int),
        "tsr_plan_update": ([P, P, P], ctypes.c_int),
        "tsr_bsa_forward": ([P, P, P, P, P, P, P], ctypes.c_int),
        "tsr_bsa_forward_batch": ([P, I32, P], ctypes.c_int),
        "tsr_plan_device_status": ([P, P], ctypes.c_int),
        "tsr_plan_destroy": ([P], ctypes.c_int),
        "tsr_plan_get_stats": ([P, P], ctypes.c_int),
        "tsr_plan_export": ([P, P, P], ctypes.c_int),
        "tsr_temporal_permute": ([P, P, I32, I32, I32, I32, I32, P, I32, P], ctypes.c_int),
        "tsr_svg_route": ([P, P, P, I32, I32, I32, I32, I32, I32, P, I32, P, P, P], ctypes.c_int),
        "tsr_rope": ([P, P, I32, P], ctypes.c_int),
        "tsr_block_select_workspace": ([P, P], ctypes.c_int),
        "tsr_block_select": ([P, P, P, P, P, ctypes.c_size_t, P], ctypes.c_int),
        "tsr_backward_plan": ([P, P, P], ctypes.c_int),
        "tsr_backward_plan_update": ([P, P, P], ctypes.c_int),
        "tsr_backward_plan_destroy": ([P], ctypes.c_int),
        "tsr_backward_plan_device_status": ([P, P], ctypes.c_int),
        "tsr_backward_plan_test_stall": ([P, I32], ctypes.c_int),
        "tsr_bsa_backward_workspace": ([P, P], ctypes.c_int),
        "tsr_bsa_backward": ([P] * 11 + [ctypes.c_size_t, P], ctypes.c_int),
        "tsr_attention_host": ([P, P, P, P, P, P, P], ctypes.c_int),
        "tsr_release_host_buffers": ([], None),
        "tsr_regime_load": ([ctypes.c_char_p], ctypes.c_int),
        "tsr_regime_lookup": ([I32, I32, I32, I32, ctypes.c_double, P], ctypes.c_int),
    }
    for name, (args, res) in sig.items():
        f = getattr(L, name)
        f.argtypes = args
        f.restype = res
    _LIB = L
    if os.path.exists(REGIME_TABLE):
        _check(L.tsr_regime_load(REGIME_TABLE.encode()))
    return _LIB


def _check(status: int) -> None:
    if status != 0:
        msg = _LIB.tsr_last_error().decode(errors="replace") if _LIB is not None else ""
        raise TsrError(status, msg)


def _stream_ptr(stream) -> int:
    if stream is None:
        # the current stream's handle, without a Stream object for it
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _dptr(t: Optional[torch.Tensor]) -> int:
    if t is None:
        return 0
    if not t.is_cuda:
        raise ValueError("mask and tensor arguments must be CUDA tensors")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


def _on_device(*tensors) -> None:
    """CUDA tensors of the current device: the library launches there."""
    current = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.get_device() != current:
            raise ValueError(f"tensor on {t.device}: arguments must be CUDA tensors of the current device, "
                             f"cuda:{current}")


def _allocating_on(stream):
    """Context in which new tensors belong to the stream that the call runs on, so
    that a workspace freed on return is not reused before the call's kernels end."""
    if stream is None:
        return contextlib.nullcontext()
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream))
    return torch.cuda.stream(stream)


class Mask:
    """A tsr_mask struct plus the device tensors it points into (kept alive)."""

    def __init__(self, kind: int, B: int, H: int, N: int, d: int, *, bq: int = 0, bk: int = 0,
                 blocks=None, q_bounds=None, k_bounds=None, head_kind=None, n_frames: int = 0,
                 frame_size: int = 0, slice_m: int = 0, indptr=None, indices=None,
                 temporal_radius: int = 0):
        self.tensors = dict(blocks=blocks, q_bounds=q_bounds, k_bounds=k_bounds,
                            head_kind=head_kind, indptr=indptr, indices=indices)
        s = _Mask()
        s.kind, s.B, s.H, s.N, s.d = kind, B, H, N, d
        s.bq, s.bk = bq, bk
        s.blocks = _dptr(blocks)
        s.q_bounds, s.k_bounds = _dptr(q_bounds), _dptr(k_bounds)
        s.n_qseg = q_bounds.numel() - 1 if q_bounds is not None else 0
        s.n_kseg = k_bounds.numel() - 1 if k_bounds is not None else 0
        s.head_kind = _dptr(head_kind)
        s.n_frames, s.frame_size = n_frames, frame_size
        s.slice_m = slice_m
        s.indptr, s.indices = _dptr(indptr), _dptr(indices)
        s.temporal_radius = int(temporal_radius)
        self.struct = s
        self.kind, self.B, self.H, self.N, self.d = kind, B, H, N, d


def make_mask(kind: int, B: int, H: int, N: int, d: int, **kw) -> Mask:
    return Mask(kind, B, H, N, d, **kw)


class Plan:
    """Owner of a tsr_plan_t; released by destroy() or garbage collection."""

    def __init__(self, handle: int, mask: Mask):
        self.handle = handle
        self.mask = mask
        self.B, self.H, self.N, self.d = mask.B, mask.H, mask.N, mask.d

    def update(self, mask: "Mask", stream=None) -> "Plan":
        """Re-plan for a new mask of the same shape, reusing the plan's storage."""
        _check(lib().tsr_plan_update(self.handle, ctypes.byref(mask.struct), _stream_ptr(stream)))
        self.mask = mask
        return self

    def stats(self) -> dict:
        st = _Stats()
        _check(lib().tsr_plan_get_stats(self.handle, ctypes.byref(st)))
        return {f: getattr(st, f) for f, _ in st._fields_}

    def export(self) -> bytes:
        n = ctypes.c_size_t(0)
        _check(lib().tsr_plan_export(self.handle, None, ctypes.byref(n)))
        buf = (ctypes.c_uint8 * n.value)()
        _check(lib().tsr_plan_export(self.handle, buf, ctypes.byref(n)))
        return bytes(buf)[: n.value]

    def destroy(self) -> None:
        if self.handle:
            lib().tsr_plan_destroy(self.handle)
            self.handle = 0

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass


def _opts(opts) -> Optional[_Opts]:
    if opts is None:
        return None
    unknown = set(opts) - {"bn", "stages", "ctas_per_sm", "flags", "orient", "kv_split"}
    if unknown:
        raise ValueError(f"unknown plan option(s): {sorted(unknown)}")
    o = _Opts()
    o.bn = int(opts.get("bn", 0))
    o.stages = int(opts.get("stages", 0))
    o.ctas_per_sm = int(opts.get("ctas_per_sm", 0))
    o.flags = int(opts.get("flags", 0))
    o.orient = int(opts.get("orient", 0))
    o.kv_split = int(opts.get("kv_split", 0))
    return o


def tsr_plan(mask: Mask, opts: Optional[dict] = None, stream=None) -> Plan:
    """Physical tile plan of `mask` (see tsr_plan in include/tsr.h)."""
    L = lib()
    h = ctypes.c_void_p(0)
    o = _opts(opts)
    _check(L.tsr_plan(ctypes.byref(mask.struct), ctypes.byref(o) if o is not None else None,
                      ctypes.byref(h), _stream_ptr(stream)))
    return Plan(h.value, mask)


def tsr_plan_update(plan: Plan, mask: Mask, stream=None) -> Plan:
    return plan.update(mask, stream)


def tsr_bsa_forward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, plan: Plan,
                    out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                    stream=None):
    """Attention over `plan`: returns (out bf16 [B,H,N,d], lse fp32 [B,H,N])."""
    shape = (plan.B, plan.H, plan.N, plan.d)
    for t in (q, k, v):
        if t.dtype != torch.bfloat16 or t.shape != shape:
            raise ValueError(f"q, k, v must be bf16 of shape {shape}")
    if out is None:
        out = torch.empty(shape, dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty(shape[:3], dtype=torch.float32, device=q.device)
    _check(lib().tsr_bsa_forward(_dptr(q), _dptr(k), _dptr(v), plan.handle, _dptr(out),
                                 _dptr(lse), _stream_ptr(stream)))
    return out, lse


def tsr_plan_device_status(plan: Plan, stream=None) -> None:
    _check(lib().tsr_plan_device_status(plan.handle, _stream_ptr(stream)))


class BackwardPlan:
    """Owner of a tsr_backward_plan_t; released by destroy() or garbage collection."""

    def __init__(self, handle: int, mask: Mask):
        self.handle = handle
        self.mask = mask
        self.B, self.H, self.N, self.d = mask.B, mask.H, mask.N, mask.d
        need = ctypes.c_size_t(0)
        _check(lib().tsr_bsa_backward_workspace(handle, ctypes.byref(need)))
        self.workspace_bytes = need.value

    def update(self, mask: Mask, stream=None) -> "BackwardPlan":
        """Re-plan for a new mask of the same shape, reusing the plan's storage."""
        _check(lib().tsr_backward_plan_update(self.handle, ctypes.byref(mask.struct), _stream_ptr(stream)))
        self.mask = mask
        return self

    def device_status(self, stream=None) -> None:
        _check(lib().tsr_backward_plan_device_status(self.handle, _stream_ptr(stream)))

    def test_stall(self, where: int) -> None:
        """Test only: see tsr_backward_plan_test_stall in include/tsr.h."""
        _check(lib().tsr_backward_plan_test_stall(self.handle, int(where)))

    def destroy(self) -> None:
        if self.handle:
            lib().tsr_backward_plan_destroy(self.handle)
            self.handle = 0

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass


def tsr_backward_plan(mask: Mask, stream=None) -> BackwardPlan:
    """The tiles of a UNIFORM or SEGMENTS mask by query and by key, for
    tsr_bsa_backward (see include/tsr.h)."""
    h = ctypes.c_void_p(0)
    _check(lib().tsr_backward_plan(ctypes.byref(mask.struct), ctypes.byref(h), _stream_ptr(stream)))
    return BackwardPlan(h.value, mask)


def tsr_backward_plan_update(plan: BackwardPlan, mask: Mask, stream=None) -> BackwardPlan:
    return plan.update(mask, stream)


def tsr_bsa_backward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor,
                     lse: torch.Tensor, dout: torch.Tensor, plan: BackwardPlan,
                     dq: Optional[torch.Tensor] = None, dk: Optional[torch.Tensor] = None,
                     dv: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                     stream=None):
    """Gradients of tsr_bsa_forward: returns (dq, dk, dv), bf16 [B, H, N, d].  ``out``
    and ``lse`` are the forward's over the plan's mask.  ``workspace``: uint8, at
    least plan.workspace_bytes; default: one allocated for the call."""
    shape = (plan.B, plan.H, plan.N, plan.d)
    for t in (q, k, v, out, dout, dq, dk, dv):
        if t is not None and (t.dtype != torch.bfloat16 or t.shape != shape):
            raise ValueError(f"q, k, v, out, dout and the gradients must be bf16 of shape {shape}")
    if lse.dtype != torch.float32 or lse.shape != shape[:3]:
        raise ValueError(f"lse must be fp32 of shape {shape[:3]}")
    _on_device(q, k, v, out, lse, dout, dq, dk, dv, workspace)
    if dq is None or dk is None or dv is None or workspace is None:
        with _allocating_on(stream):
            dq, dk, dv = (torch.empty(shape, dtype=torch.bfloat16, device=q.device) if t is None else t
                          for t in (dq, dk, dv))
            if workspace is None:
                workspace = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device=q.device)
    _check(lib().tsr_bsa_backward(_dptr(q), _dptr(k), _dptr(v), _dptr(out), _dptr(lse), _dptr(dout),
                                  plan.handle, _dptr(dq), _dptr(dk), _dptr(dv), _dptr(workspace),
                                  workspace.numel() * workspace.element_size(), _stream_ptr(stream)))
    return dq, dk, dv


def tsr_temporal_permute(src: torch.Tensor, dst: torch.Tensor, n_frames: int, frame_size: int,
                         head_kind=None, inverse: bool = False, stream=None) -> torch.Tensor:
    """Temporal-major permutation of [B, H, F*S, row] tensors (see include/tsr.h)."""
    B, H, N = src.shape[:3]
    row_bytes = src[0, 0, 0].numel() * src.element_size()
    hk = None
    if head_kind is not None:
        hk_arr = (ctypes.c_int8 * H)(*[int(x) for x in head_kind])
        hk = ctypes.cast(hk_arr, ctypes.c_void_p)
    _check(lib().tsr_temporal_permute(_dptr(src), _dptr(dst), B, H, n_frames, frame_size,
                                      row_bytes, hk, 1 if inverse else 0, _stream_ptr(stream)))
    return dst


def tsr_bsa_forward_batch(requests, stream=None):
    """Several requests in one launch (see include/tsr.h).  ``requests``: a
    sequence of (q, k, v, plan) or (q, k, v, plan, out, lse); returns the list
    of (out, lse)."""
    n = len(requests)
    arr = (_Request * max(1, n))()
    outs = []
    for i, rq in enumerate(requests):
        q, k, v, plan = rq[:4]
        out = rq[4] if len(rq) > 4 and rq[4] is not None else torch.empty_like(q)
        lse = (rq[5] if len(rq) > 5 and rq[5] is not None else
               torch.empty(q.shape[:3], dtype=torch.float32, device=q.device))
        arr[i].q, arr[i].k, arr[i].v = _dptr(q), _dptr(k), _dptr(v)
        arr[i].plan = plan.handle
        arr[i].out, arr[i].lse = _dptr(out), _dptr(lse)
        outs.append((out, lse))
    _check(lib().tsr_bsa_forward_batch(ctypes.cast(arr, ctypes.c_void_p), n, _stream_ptr(stream)))
    return outs


def tsr_svg_route(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, n_frames: int,
                  frame_size: int, samples, temporal_radius: int = 0, stats=None,
                  head_kind=None, stream=None):
    """Route each head to the spatial or temporal SVG pattern from sampled query
    rows (see include/tsr.h).  Returns (stats fp32 [B, H, 3], head_kind int8 [H]),
    both on q's device; ``samples`` is a host sequence of row indices."""
    B, H, N, d = q.shape
    if N != n_frames * frame_size or k.shape != q.shape or v.shape != q.shape:
        raise ValueError("q, k, v must be [B, H, n_frames * frame_size, d] alike")
    if stats is None:
        stats = torch.empty((B, H, 3), dtype=torch.float32, device=q.device)
    if head_kind is None:
        head_kind = torch.empty((H,), dtype=torch.int8, device=q.device)
    smp = [int(x) for x in samples]
    arr = (ctypes.c_int32 * max(1, len(smp)))(*smp)
    _check(lib().tsr_svg_route(_dptr(q), _dptr(k), _dptr(v), B, H, n_frames, frame_size, d,
                               temporal_radius, ctypes.cast(arr, ctypes.c_void_p), len(smp),
                               _dptr(stats), _dptr(head_kind), _stream_ptr(stream)))
    return stats, head_kind


_ROPE_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


def tsr_rope(x, axis_dims, *, grid=None, positions: Optional[torch.Tensor] = None,
             theta: float = 10000.0, halves: bool = False, inverse: bool = False, out=None,
             stream=None):
    """Rotary positions over several axes (see include/tsr.h).

    ``x``: a tensor [B, H, N, d] (bf16, fp16 or fp32; any strides, d contiguous:
    a [B, N, H, d] projection goes in as ``x.transpose(1, 2)``), or a sequence of
    up to four that differ in H and strides only (Q and K), rotated in one launch.
    ``axis_dims``: channels per axis.  ``grid``: tokens per axis, in row-major
    order, or ``positions``: int32 [N, axes] or [B, N, axes].  ``out``: like x
    (x itself: in place); default contiguous [B, H, N, d].  Returns out."""
    one = isinstance(x, torch.Tensor)
    xs = (x,) if one else tuple(x)
    if not 1 <= len(xs) <= 4:
        raise ValueError("one to four tensors per call")
    if (grid is None) == (positions is None):
        raise ValueError("give grid or positions")
    first = xs[0]
    if first.dim() != 4:
        raise ValueError("the tensors are [B, H, N, d]")
    B, _, N, d = first.shape
    dtype = first.dtype
    code = _ROPE_DTYPES.get(dtype)
    if code is None:
        raise ValueError("the tensors are bf16, fp16 or fp32")
    dims = [int(a) for a in axis_dims]
    axes = len(dims)
    if not 1 <= axes <= 4:
        raise ValueError("one to four axes")
    for t in xs:
        if t.dim() != 4 or t.dtype != dtype or t.shape[::2] != (B, N) or t.shape[3] != d:
            raise ValueError("the tensors of one call are [B, H, N, d] with the same B, N, d and dtype")
    if out is None:
        _on_device(*xs, positions)
        with _allocating_on(stream):
            outs = [torch.empty(t.shape, dtype=dtype, device=t.device) for t in xs]
    else:
        outs = (out,) if isinstance(out, torch.Tensor) else tuple(out)
        if len(outs) != len(xs):
            raise ValueError("as many outputs as tensors")
        _on_device(*xs, *outs, positions)
    tensors = b""
    for t, o in zip(xs, outs):
        xb, xh, xn, x_last = t.stride()
        ob, oh, on, o_last = o.stride()
        if out is not None and (o.shape != t.shape or o.dtype != dtype):
            raise ValueError("out must have x's shape and dtype")
        if x_last != 1 or o_last != 1:
            raise ValueError("the last dimension must be contiguous")
        tensors += _ROPE_TENSOR.pack(t.data_ptr(), o.data_ptr(), t.shape[1], xb, xh, xn, ob, oh, on)
    pad = (0,) * (4 - axes)
    if positions is not None:
        if positions.dtype != torch.int32 or positions.shape not in ((N, axes), (B, N, axes)):
            raise ValueError("positions must be int32 [N, axes] or [B, N, axes]")
        where = (_dptr(positions), positions.dim() == 3, 0, 0, 0, 0)
    else:
        cells = [int(g) for g in grid]
        if len(cells) != axes:
            raise ValueError("grid needs one size per axis")
        where = (0, 0, *cells, *pad)
    desc = _ROPE_DESC.pack(B, N, d, code, axes, *dims, *pad, bool(halves), bool(inverse), theta, *where)
    _check(lib().tsr_rope(desc, tensors, len(xs), _stream_ptr(stream)))
    return outs[0] if one else list(outs)


def tsr_rope_backward(dout, axis_dims, **kw):
    """The gradient of tsr_rope's input from its output's: the inverse rotation,
    same arguments (``out``: where the gradient goes)."""
    return tsr_rope(dout, axis_dims, inverse=not kw.pop("inverse", False), **kw)


def tsr_block_select(q: torch.Tensor, k: torch.Tensor, keep: int, *, bq: int = 64, bk: int = 64,
                     first: int = 0, diagonal: bool = False, out: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The key blocks each query block keeps, as a UNIFORM mask's ``blocks``: uint8
    [B, H, ceil(N / bq), ceil(N / bk)] (see tsr_block_select in include/tsr.h).
    ``workspace``: uint8, at least tsr_block_select_workspace() bytes; default: one
    allocated for the call."""
    if q.dim() != 4 or k.shape != q.shape or q.dtype != torch.bfloat16 or k.dtype != torch.bfloat16:
        raise ValueError("q, k must be bf16 [B, H, N, d] alike")
    _on_device(q, k, out, workspace)
    B, H, N, d = q.shape
    bq, bk = int(bq), int(bk)
    desc = _SELECT_DESC.pack(B, H, N, d, bq, bk, int(keep), int(first), bool(diagonal))
    L = lib()
    need = ctypes.c_size_t(0)
    _check(L.tsr_block_select_workspace(desc, ctypes.byref(need)))
    shape = (B, H, -(-N // bq), -(-N // bk))
    if out is None or workspace is None:
        with _allocating_on(stream):
            if out is None:
                out = torch.empty(shape, dtype=torch.uint8, device=q.device)
            if workspace is None:
                workspace = torch.empty(need.value, dtype=torch.uint8, device=q.device)
    if out.shape != shape or out.dtype != torch.uint8:
        raise ValueError(f"out must be uint8 of shape {shape}")
    _check(L.tsr_block_select(desc, _dptr(q), _dptr(k), _dptr(out), _dptr(workspace),
                              workspace.numel() * workspace.element_size(), _stream_ptr(stream)))
    return out


def tsr_attention_host(kind: int, B: int, H: int, N: int, d: int, q, k, v, out, lse,
                       opts: Optional[dict] = None, **mask_arrays):
    """One whole call from host memory.  q, k, v, out: CPU bf16 tensors (pinned for
    speed), lse: CPU fp32; mask arrays are CPU tensors / NumPy arrays."""
    import numpy as np
    keep = []

    def hptr(x):
        if x is None:
            return 0
        if isinstance(x, torch.Tensor):
            if x.is_cuda or not x.is_contiguous():
                raise ValueError("host tensors must be contiguous CPU tensors")
            keep.append(x)
            return x.data_ptr()
        a = np.ascontiguousarray(x)
        keep.append(a)
        return a.ctypes.data

    s = _Mask()
    s.kind, s.B, s.H, s.N, s.d = kind, B, H, N, d
    s.bq, s.bk = mask_arrays.get("bq", 0), mask_arrays.get("bk", 0)
    s.blocks = hptr(mask_arrays.get("blocks"))
    qb, kb = mask_arrays.get("q_bounds"), mask_arrays.get("k_bounds")
    s.q_bounds, s.k_bounds = hptr(qb), hptr(kb)
    s.n_qseg = len(qb) - 1 if qb is not None else 0
    s.n_kseg = len(kb) - 1 if kb is not None else 0
    s.head_kind = hptr(mask_arrays.get("head_kind"))
    s.n_frames, s.frame_size = mask_arrays.get("n_frames", 0), mask_arrays.get("frame_size", 0)
    s.slice_m = mask_arrays.get("slice_m", 0)
    s.indptr, s.indices = hptr(mask_arrays.get("indptr")), hptr(mask_arrays.get("indices"))
    s.temporal_radius = int(mask_arrays.get("temporal_radius", 0))
    o = _opts(opts)
    _check(lib().tsr_attention_host(ctypes.byref(s), ctypes.byref(o) if o is not None else None,
                                    hptr(q), hptr(k), hptr(v), hptr(out), hptr(lse)))
    return out, lse


def tsr_regime_load(path: Optional[str]) -> None:
    _check(lib().tsr_regime_load(path.encode() if path else None))


def tsr_regime_lookup(kind: int, bq: int, bk: int, N: int, density: float) -> dict:
    r = _Regime()
    _check(lib().tsr_regime_lookup(kind, bq, bk, N, density, ctypes.byref(r)))
    return {"bn": r.bn, "stages": r.stages, "ctas_per_sm": r.ctas_per_sm, "id": r.id,
            "orient": r.orient}


def tsr_abi_version() -> int:
    return int(lib().tsr_abi_version())
