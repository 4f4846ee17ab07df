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
    "tsr_rope", "tsr_rope_backward", "tsr_norm_rope", "tsr_norm_rope_backward", "tsr_block_select",
    "tsr_linear", "tsr_linear_backward", "tsr_linear_device_status",
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


class _NormRopeTensor(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("weight", ctypes.c_void_p), ("dout", ctypes.c_void_p),
                ("out", ctypes.c_void_p), ("dweight", ctypes.c_void_p), ("H", ctypes.c_int32),
                ("weight_dtype", ctypes.c_int32), ("x_stride", ctypes.c_int64 * 3),
                ("dout_stride", ctypes.c_int64 * 3), ("out_stride", ctypes.c_int64 * 3)]


class _LinearDesc(ctypes.Structure):
    _fields_ = [(f, ctypes.c_int32) for f in ("B", "N", "in_heads", "in_dim", "out_heads", "out_dim", "dtype",
                                              "activation")]


class _LinearArgs(ctypes.Structure):
    _fields_ = ([(f, ctypes.c_void_p) for f in ("x", "weight", "bias", "residual", "out", "pre")]
                + [(f + "_stride", ctypes.c_int64 * 3) for f in ("x", "residual", "out", "pre")])


class _LinearGrads(ctypes.Structure):
    _fields_ = ([(f, ctypes.c_void_p) for f in ("dout", "x", "weight", "pre", "dx", "dweight", "dbias")]
                + [(f + "_stride", ctypes.c_int64 * 3) for f in ("dout", "x", "pre", "dx")])


class _SelectDesc(ctypes.Structure):
    _fields_ = [(f, ctypes.c_int32) for f in ("B", "H", "N", "d", "bq", "bk", "keep", "first", "diagonal")]


# The same layouts as packed bytes, which the calls below pass (filling a ctypes
# structure field by field takes longer than the kernels of a small call).
_ROPE_DESC = struct.Struct("@5i4i2idPi4i4x")
_ROPE_TENSOR = struct.Struct("@PPi3q3q")
_NORM_ROPE_TENSOR = struct.Struct("@PPPPP2i3q3q3q")
_LINEAR_DESC = struct.Struct("@8i")
_LINEAR_ARGS = struct.Struct("@6P12q")
_LINEAR_GRADS = struct.Struct("@7P12q")
_SELECT_DESC = struct.Struct("@9i")
for _packed, _fields in ((_ROPE_DESC, _RopeDesc), (_ROPE_TENSOR, _RopeTensor), (_SELECT_DESC, _SelectDesc),
                         (_NORM_ROPE_TENSOR, _NormRopeTensor), (_LINEAR_DESC, _LinearDesc),
                         (_LINEAR_ARGS, _LinearArgs), (_LINEAR_GRADS, _LinearGrads)):
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
           "tsr_plan_export", "tsr_temporal_permute", "tsr_svg_route", "tsr_rope", "tsr_norm_rope",
           "tsr_norm_rope_backward_workspace", "tsr_norm_rope_backward", "tsr_linear_workspace", "tsr_linear",
           "tsr_linear_backward_workspace", "tsr_linear_backward", "tsr_linear_device_status",
           "tsr_linear_test_stall", "tsr_block_select_workspace", "tsr_block_select", "tsr_backward_plan",
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
        "tsr_norm_rope": ([P, ctypes.c_double, P, I32, P], ctypes.c_int),
        "tsr_norm_rope_backward_workspace": ([P, I32, P], ctypes.c_int),
        "tsr_norm_rope_backward": ([P, ctypes.c_double, P, I32, P, ctypes.c_size_t, P], ctypes.c_int),
        "tsr_linear_workspace": ([P, P], ctypes.c_int),
        "tsr_linear": ([P, P, P, ctypes.c_size_t, P], ctypes.c_int),
        "tsr_linear_backward_workspace": ([P, P], ctypes.c_int),
        "tsr_linear_backward": ([P, P, P, ctypes.c_size_t, P], ctypes.c_int),
        "tsr_linear_device_status": ([P], ctypes.c_int),
        "tsr_linear_test_stall": ([I32], ctypes.c_int),
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


_ready = torch.cuda.is_initialized


def _device() -> int:
    """The current device.  torch.cuda.current_device() where CUDA is not set up yet, or must
    not be (in a forked child): it does that, or says so; else without its steps (1 us a call)."""
    return torch._C._cuda_getDevice() if _ready() else torch.cuda.current_device()


def _stream_ptr(stream) -> int:
    if stream is None:
        # the current stream's handle, without a Stream object for it
        return torch._C._cuda_getCurrentRawStream(_device())
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
    current = _device()
    for t in tensors:
        if t is not None and t.get_device() != current:
            raise ValueError(f"tensor on {t.device}: arguments must be CUDA tensors of the current device, "
                             f"cuda:{current}")


_HERE = contextlib.nullcontext()


def _allocating_on(stream):
    """Context in which new tensors belong to the stream that the call runs on, so
    that a workspace freed on return is not reused before the call's kernels end."""
    if stream is None:
        return _HERE
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


def _heads_list(x):
    return (x,) if isinstance(x, torch.Tensor) else tuple(x)


def _heads_call(xs, axis_dims, grid, positions, theta, halves, inverse=False):
    """What the calls that rotate heads share: the tensors' type, channels, shapes and strides,
    and the packed tsr_rope_desc."""
    if not 1 <= len(xs) <= 4:
        raise ValueError("one to four tensors per call")
    if (grid is None) == (positions is None):
        raise ValueError("give grid or positions")
    first = xs[0]
    dtype = first.dtype
    code = _ROPE_DTYPES.get(dtype)
    if code is None:
        raise ValueError("the tensors are bf16, fp16 or fp32")
    dims = [int(a) for a in axis_dims]
    axes = len(dims)
    if not 1 <= axes <= 4:
        raise ValueError("one to four axes")
    if first.dim() != 4:
        raise ValueError("the tensors are [B, H, N, d]")
    B, _, N, d = first.shape
    rows = []
    for t in xs:
        shape = t.shape
        if len(shape) != 4 or t.dtype is not dtype or shape[0] != B or shape[2] != N or shape[3] != d:
            raise ValueError("the tensors of one call are [B, H, N, d] with the same B, N, d and dtype")
        rows.append((t, shape, t.stride()))
    pad = (0,) * (4 - axes)
    if positions is not None:
        if positions.dtype is not torch.int32 or positions.shape not in ((N, axes), (B, N, axes)):
            raise ValueError("positions must be int32 [N, axes] or [B, N, axes]")
        where = (_dptr(positions), positions.dim() == 3, 0, 0, 0, 0)
    else:
        cells = [int(g) for g in grid]
        if len(cells) != axes:
            raise ValueError("grid needs one size per axis")
        where = (0, 0, *cells, *pad)
    return dtype, d, rows, _ROPE_DESC.pack(B, N, d, code, axes, *dims, *pad, bool(halves), bool(inverse), theta, *where)


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
    xs = _heads_list(x)
    dtype, _, rows, desc = _heads_call(xs, axis_dims, grid, positions, theta, halves, inverse)
    if out is None:
        _on_device(*xs, positions)
        with _allocating_on(stream):
            outs = [torch.empty_like(t, memory_format=torch.contiguous_format) for t in xs]
    else:
        outs = _heads_list(out)
        if len(outs) != len(xs):
            raise ValueError("as many outputs as tensors")
        _on_device(*xs, *outs, positions)
    tensors = b""
    for (t, shape, (xb, xh, xn, x_last)), o in zip(rows, outs):
        if out is not None and (o.shape != shape or o.dtype != dtype):
            raise ValueError("out must have x's shape and dtype")
        ob, oh, on, o_last = o.stride()
        if x_last != 1 or o_last != 1:
            raise ValueError("the last dimension must be contiguous")
        tensors += _ROPE_TENSOR.pack(t.data_ptr(), o.data_ptr(), shape[1], xb, xh, xn, ob, oh, on)
    _check(lib().tsr_rope(desc, tensors, len(xs), _stream_ptr(stream)))
    return outs[0] if isinstance(x, torch.Tensor) else list(outs)


def tsr_rope_backward(dout, axis_dims, **kw):
    """The gradient of tsr_rope's input from its output's: the inverse rotation,
    same arguments (``out``: where the gradient goes)."""
    return tsr_rope(dout, axis_dims, inverse=not kw.pop("inverse", False), **kw)


def _weights(weight, xs, dtype, d):
    """One weight (or None) per tensor, and their type's code."""
    ws = tuple(weight) if isinstance(weight, (list, tuple)) else (weight,) * len(xs)
    if len(ws) != len(xs):
        raise ValueError("one weight (or None) for each tensor")
    kind = None
    for w in ws:
        if w is not None:
            if w.shape != (d,) or (w.dtype is not dtype and w.dtype is not torch.float32) or kind not in (None, w.dtype):
                raise ValueError("the weights are [d], all of the tensors' type or all fp32")
            kind = w.dtype
    return ws, _ROPE_DTYPES[kind or dtype]


def tsr_norm_rope(x, weight, axis_dims, *, eps: float = 1e-6, grid=None,
                  positions: Optional[torch.Tensor] = None, theta: float = 10000.0, halves: bool = False,
                  out=None, stream=None):
    """RMS norm over each head's d channels, then tsr_rope, in one pass (see
    tsr_norm_rope in include/tsr.h).  ``x``, ``out`` and the positions as for tsr_rope;
    ``weight``: [d] of x's type or fp32, or None (ones); for several tensors a sequence of
    as many (one tensor alone is shared by all).  Returns out."""
    xs = _heads_list(x)
    dtype, d, rows, desc = _heads_call(xs, axis_dims, grid, positions, theta, halves)
    ws, code = _weights(weight, xs, dtype, d)
    if out is None:
        _on_device(*xs, *ws, positions)
        with _allocating_on(stream):
            outs = [torch.empty_like(t, memory_format=torch.contiguous_format) for t in xs]
    else:
        outs = _heads_list(out)
        if len(outs) != len(xs):
            raise ValueError("as many outputs as tensors")
        _on_device(*xs, *ws, *outs, positions)
    tensors = b""
    for (t, shape, (xb, xh, xn, x_last)), w, o in zip(rows, ws, outs):
        if out is not None and (o.shape != shape or o.dtype != dtype):
            raise ValueError("out must have x's shape and dtype")
        ob, oh, on, o_last = o.stride()
        if x_last != 1 or o_last != 1:
            raise ValueError("the last dimension must be contiguous")
        tensors += _NORM_ROPE_TENSOR.pack(t.data_ptr(), 0 if w is None else _dptr(w), 0, o.data_ptr(), 0, shape[1], code,
                                          xb, xh, xn, 0, 0, 0, ob, oh, on)
    _check(lib().tsr_norm_rope(desc, eps, tensors, len(xs), _stream_ptr(stream)))
    return outs[0] if isinstance(x, torch.Tensor) else list(outs)


def tsr_norm_rope_backward(dout, x, weight, axis_dims, *, eps: float = 1e-6, grid=None,
                           positions: Optional[torch.Tensor] = None, theta: float = 10000.0,
                           halves: bool = False, out=None, dweight=None,
                           workspace: Optional[torch.Tensor] = None, stream=None):
    """Gradients of tsr_norm_rope: returns (dx, dweight), lists of them for several
    tensors; dweight is None where the weight is.  ``out``: where dx goes (any strides);
    ``workspace``: uint8, at least tsr_norm_rope_backward_workspace() bytes; default: one
    allocated for the call."""
    xs, gs = _heads_list(x), _heads_list(dout)
    one = isinstance(x, torch.Tensor)
    dtype, d, rows, desc = _heads_call(xs, axis_dims, grid, positions, theta, halves)
    ws, code = _weights(weight, xs, dtype, d)
    if len(set(id(w) for w in ws if w is not None)) != sum(w is not None for w in ws):
        raise ValueError("a shared weight's gradient needs a call for each tensor")
    if len(gs) != len(xs) or any(g.shape != t.shape or g.dtype != dtype for g, t in zip(gs, xs)):
        raise ValueError("dout must have x's shapes and dtype")
    outs = None if out is None else _heads_list(out)
    dws = None if dweight is None else _heads_list(dweight)
    for given in (outs, dws):
        if given is not None and len(given) != len(xs):
            raise ValueError("as many outputs as tensors")
    _on_device(*xs, *gs, *ws, positions, workspace, *(outs or ()), *(dws or ()))
    L = lib()
    with _allocating_on(stream):
        if outs is None:
            outs = [torch.empty_like(t, memory_format=torch.contiguous_format) for t in xs]
        if dws is None:
            dws = [None if w is None else torch.empty_like(w) for w in ws]
        if workspace is None:
            need = ctypes.c_size_t(0)
            _check(L.tsr_norm_rope_backward_workspace(desc, len(xs), ctypes.byref(need)))
            workspace = torch.empty(need.value, dtype=torch.uint8, device=xs[0].device)
    tensors = b""
    for (t, shape, (xb, xh, xn, x_last)), g, w, o, dw in zip(rows, gs, ws, outs, dws):
        gb, gh, gn, g_last = g.stride()
        ob, oh, on, o_last = o.stride()
        if o.shape != shape or o.dtype != dtype:
            raise ValueError("out must have x's shape and dtype")
        if x_last != 1 or g_last != 1 or o_last != 1:
            raise ValueError("the last dimension must be contiguous")
        if (dw is None) != (w is None) or (dw is not None and (dw.shape != w.shape or dw.dtype != w.dtype)):
            raise ValueError("dweight must have the weight's shape and dtype")
        tensors += _NORM_ROPE_TENSOR.pack(t.data_ptr(), _dptr(w), g.data_ptr(), o.data_ptr(), _dptr(dw), shape[1], code,
                                          xb, xh, xn, gb, gh, gn, ob, oh, on)
    _check(L.tsr_norm_rope_backward(desc, eps, tensors, len(xs), _dptr(workspace),
                                    workspace.numel() * workspace.element_size(), _stream_ptr(stream)))
    return (outs[0], dws[0]) if one else (list(outs), list(dws))


_ACTIVATIONS = {None: 0, "gelu": 1, "gelu_tanh": 2, "silu": 3}


def _token_rows(t):
    """B, heads, N, channels per head and the b, h, n strides of [B, N, features],
    [N, features] or head-major [B, heads, N, dim]; channels contiguous."""
    shape, stride = t.shape, t.stride()
    if len(shape) == 3:
        rows = (shape[0], 1, shape[1], shape[2]), (stride[0], 0, stride[1])
    elif len(shape) == 4:
        rows = tuple(shape), stride[:3]
    elif len(shape) == 2:
        rows = (1, 1, shape[0], shape[1]), (0, 0, stride[0])
    else:
        raise ValueError("token rows are [N, features], [B, N, features] or [B, heads, N, dim]")
    if stride[-1] != 1:
        raise ValueError("the last dimension must be contiguous")
    return rows


def _linear_desc(x_rows, weight, out_heads, dtype, activation) -> bytes:
    B, in_heads, N, in_dim = x_rows
    code = _ROPE_DTYPES.get(dtype)
    if code not in (0, 1):
        raise ValueError("the tensors are bf16 or fp16")
    if activation not in _ACTIVATIONS:
        raise ValueError(f"activation: one of {list(_ACTIVATIONS)}")
    if weight.dim() != 2 or weight.dtype != dtype or weight.shape[1] != in_heads * in_dim:
        raise ValueError("weight must be [out features, in features] of x's type")
    M = weight.shape[0]
    if out_heads < 1 or M % out_heads:
        raise ValueError("heads must divide the out features")
    return _LINEAR_DESC.pack(B, N, in_heads, in_dim, out_heads, M // out_heads, code, _ACTIVATIONS[activation])


_LINEAR_WORKSPACE = {}    # bytes by entry point and packed desc (sizes only)


def _workspace(need_of, name, desc, workspace, device):
    if workspace is None:
        need = _LINEAR_WORKSPACE.get((name, desc))
        if need is None:
            n = ctypes.c_size_t(0)
            _check(need_of(desc, ctypes.byref(n)))
            if len(_LINEAR_WORKSPACE) >= 4096:
                _LINEAR_WORKSPACE.clear()
            need = _LINEAR_WORKSPACE[name, desc] = n.value
        if need == 0:
            return None, 0
        return torch.empty(need, dtype=torch.uint8, device=device), need
    return workspace, workspace.numel() * workspace.element_size()


def tsr_linear(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None, *,
               activation: Optional[str] = None, residual: Optional[torch.Tensor] = None, heads: int = 0,
               pre=None, out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
               stream=None):
    """activation(x weight^T + bias) + residual (see tsr_linear in include/tsr.h).

    ``x``: [N, K], [B, N, K] or the attention's head-major [B, H, N, d] with K = H d, any
    strides that are multiples of 8; ``weight``: [M, K].  ``heads``: 0 for an output
    [B, N, M] ([N, M]), or the heads of a head-major output [B, heads, N, M / heads].
    ``activation``: None, "gelu", "gelu_tanh" or "silu".  ``residual``, ``out``: like the
    output.  ``pre``: True, or a tensor like the output: the values before the activation,
    for tsr_linear_backward.  ``workspace``: uint8, at least tsr_linear_workspace() bytes;
    default: one allocated for the call.  Returns out, or (out, pre)."""
    rows, x_stride = _token_rows(x)
    dtype, M = x.dtype, weight.shape[0]
    out_heads = heads or 1
    desc = _linear_desc(rows, weight, out_heads, dtype, activation)
    B, _, N, _ = rows
    if heads:
        shape = (B, heads, N, M // heads)
    else:
        shape = (N, M) if x.dim() == 2 else (B, N, M)
    if bias is not None and (bias.dtype != dtype or bias.shape != (M,)):
        raise ValueError("bias must be [out features] of x's type")
    keep = pre is not None and pre is not False
    given = pre if isinstance(pre, torch.Tensor) else None
    for t in (residual, out, given):
        if t is not None and (t.shape != shape or t.dtype != dtype):
            raise ValueError(f"residual, out and pre must be {dtype} of shape {tuple(shape)}")
    _on_device(x, weight, bias, residual, out, given, workspace)
    L = lib()
    with _allocating_on(stream):
        if out is None:
            out = torch.empty(shape, dtype=dtype, device=x.device)
        if keep and given is None:
            given = torch.empty(shape, dtype=dtype, device=x.device)
        workspace, size = _workspace(L.tsr_linear_workspace, 0, desc, workspace, x.device)
    none = (0, 0, 0)
    args = _LINEAR_ARGS.pack(x.data_ptr(), _dptr(weight), _dptr(bias), 0 if residual is None else residual.data_ptr(),
                             out.data_ptr(), given.data_ptr() if keep else 0, *x_stride,
                             *(none if residual is None else _token_rows(residual)[1]), *_token_rows(out)[1],
                             *(_token_rows(given)[1] if keep else none))
    _check(L.tsr_linear(desc, args, _dptr(workspace), size, _stream_ptr(stream)))
    return (out, given) if keep else out


def tsr_linear_backward(dout: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, *,
                        activation: Optional[str] = None, pre: Optional[torch.Tensor] = None,
                        need=(True, True, True), dx: Optional[torch.Tensor] = None,
                        dweight: Optional[torch.Tensor] = None, dbias: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None, stream=None):
    """Gradients of tsr_linear from ``dout``, like its output (head-major if that was):
    returns (dx, dweight, dbias), None where ``need`` is false.  ``pre``: what the forward
    kept, for an activation.  ``dx``, ``dweight``, ``dbias``: where they go."""
    rows, x_stride = _token_rows(x)
    out_rows, g_stride = _token_rows(dout)
    dtype, M = x.dtype, weight.shape[0]
    if dout.dtype != dtype or out_rows[::2] != rows[::2] or out_rows[1] * out_rows[3] != M:
        raise ValueError("dout must be like the layer's output")
    desc = _linear_desc(rows, weight, out_rows[1], dtype, activation)
    if activation is not None and (pre is None or pre.shape != dout.shape or pre.dtype != dtype):
        raise ValueError("pre must be like the layer's output")
    if len(need) != 3:
        raise ValueError("need: whether dx, dweight and dbias are needed")
    for t, like, name in ((dx, x.shape, "dx"), (dweight, weight.shape, "dweight"), (dbias, (M,), "dbias")):
        if t is not None and (t.shape != like or t.dtype != dtype):
            raise ValueError(f"{name} must be {dtype} of shape {tuple(like)}")
    _on_device(dout, x, weight, pre, dx, dweight, dbias, workspace)
    L = lib()
    with _allocating_on(stream):
        new = lambda t, shape, wanted: None if not wanted else t if t is not None else torch.empty(
            shape, dtype=dtype, device=x.device)
        dx, dweight, dbias = new(dx, x.shape, need[0]), new(dweight, weight.shape, need[1]), new(dbias, (M,), need[2])
        workspace, size = _workspace(L.tsr_linear_backward_workspace, 1, desc, workspace, x.device)
    none = (0, 0, 0)
    args = _LINEAR_GRADS.pack(dout.data_ptr(), x.data_ptr(), _dptr(weight), 0 if activation is None else pre.data_ptr(),
                              0 if dx is None else dx.data_ptr(), _dptr(dweight), _dptr(dbias), *g_stride, *x_stride,
                              *(none if activation is None else _token_rows(pre)[1]),
                              *(none if dx is None else _token_rows(dx)[1]))
    _check(L.tsr_linear_backward(desc, args, _dptr(workspace), size, _stream_ptr(stream)))
    return dx, dweight, dbias


def tsr_linear_device_status(stream=None) -> None:
    """Raises if a wait in a linear layer's product gave up (see include/tsr.h)."""
    _check(lib().tsr_linear_device_status(_stream_ptr(stream)))


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
