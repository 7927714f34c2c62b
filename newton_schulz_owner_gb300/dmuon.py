"""ctypes binding of ``libdmuon.so`` (declared in ``include/dmuon.h``).

Argument marshalling only: every step of the Muon step runs in the library's
CUDA kernels.  PyTorch provides device memory and the CUDA stream.  Importing
this module raises ``ImportError`` if the library has not been built, so no
caller can silently fall back to another implementation.
"""
from __future__ import annotations

import ctypes
import os
from typing import List, Optional, Sequence, Tuple

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libdmuon.so")
if not os.path.exists(_LIB_PATH):
    raise ImportError(f"{_LIB_PATH} is missing: build it with "
                      "`python -m newton_schulz_owner_gb300.build_lib` (or __graft_entry__.build())")
_lib = ctypes.CDLL(_LIB_PATH)

OK, ERR_INVALID_ARG, ERR_ALIGNMENT, ERR_WORKSPACE, ERR_CUDA, ERR_TIMEOUT, ERR_UNSUPPORTED = \
    0, -1, -2, -3, -4, -5, -6
F32, BF16 = 0, 1
NS_STANDARD, NS_GRAM, NS_GRAM_ALL = 0, 1, 2
PACK_ALIGN_ELEMS = 128
DEFAULT_ABC = (3.4445, -4.7750, 2.0315)
ACT_SILU, ACT_GELU, ACT_GELU_TANH = 0, 1, 2
SAVE_NONE, SAVE_BF16, SAVE_ACT8 = 0, 1, 2
ACT8_BLOCK = 32          # columns that share a scale

EXPORTED = ("dmuon_plan", "dmuon_workspace_bytes", "dmuon_ns_variant_for", "dmuon_pack", "dmuon_ns_batched",
            "dmuon_unpack_update", "dmuon_muon_step", "dmuon_stream_status",
            "dmuon_debug_wait_timeout", "dmuon_ns_batched_noalloc", "dmuon_noalloc_status",
            "dmuon_adamw",
            "dmuon_adamw_workspace_bytes", "dmuon_act8_save", "dmuon_act8_load",
            "dmuon_ffn_workspace_bytes", "dmuon_ffn_forward", "dmuon_ffn_backward",
            "dmuon_xent_workspace_bytes", "dmuon_xent", "dmuon_status_string", "dmuon_version",
            "dmuon_launch_count", "dmuon_trace_begin", "dmuon_trace_end")
NOALLOC_SCRATCH_BYTES = 64 << 20
# largest short side m and long side n of a matrix the library accepts
MAX_M, MAX_N = 32768, 1048576


class Shape(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64)]


class FfnShape(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("hidden", ctypes.c_int64), ("ffn", ctypes.c_int64),
                ("activation", ctypes.c_int), ("save", ctypes.c_int)]


class XentShape(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("hidden", ctypes.c_int64), ("vocab", ctypes.c_int64)]


_vp, _i, _f, _sz, _i64p = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t, \
    ctypes.POINTER(ctypes.c_int64)
_ShapeP = ctypes.POINTER(Shape)
_VPP = ctypes.POINTER(ctypes.c_void_p)

_lib.dmuon_plan.argtypes = [_i, _ShapeP, _i, ctypes.POINTER(ctypes.c_int), _i64p, _i64p]
_lib.dmuon_plan.restype = _i
_lib.dmuon_workspace_bytes.argtypes = [_i, _ShapeP, _i]
_lib.dmuon_workspace_bytes.restype = _sz
_lib.dmuon_ns_variant_for.argtypes = [ctypes.c_int64, ctypes.c_int64, _i, _i]
_lib.dmuon_ns_variant_for.restype = _i
_lib.dmuon_pack.argtypes = [_i, _ShapeP, _VPP, _i, _VPP, _f, _vp, _i64p, _vp, _sz, _vp]
_lib.dmuon_pack.restype = _i
_lib.dmuon_ns_batched.argtypes = [_i, _ShapeP, _vp, _i64p, _i, _i, ctypes.POINTER(ctypes.c_float),
                                  _f, _i, _vp, _sz, _vp]
_lib.dmuon_ns_batched.restype = _i
_lib.dmuon_unpack_update.argtypes = [_i, _ShapeP, _VPP, _i, _f, _vp, _i64p, _vp, _sz, _vp]
_lib.dmuon_unpack_update.restype = _i
_lib.dmuon_muon_step.argtypes = [_i, _ShapeP, _VPP, _i, _VPP, _VPP, _i, _f, _f, _i, _i, _vp,
                                 _i64p, _vp, _sz, _vp]
_lib.dmuon_muon_step.restype = _i
_lib.dmuon_ns_batched_noalloc.argtypes = [_i, _ShapeP, _vp, _i64p, _i, _i,
                                          ctypes.POINTER(ctypes.c_float), _f, _vp]
_lib.dmuon_ns_batched_noalloc.restype = _i
_lib.dmuon_noalloc_status.argtypes = [_vp]
_lib.dmuon_noalloc_status.restype = _i
_lib.dmuon_adamw_workspace_bytes.argtypes = [_i]
_lib.dmuon_adamw_workspace_bytes.restype = _sz
_d = ctypes.c_double
_lib.dmuon_adamw.argtypes = [_i, _i64p, _VPP, _i, _VPP, _i, _VPP, _VPP, _d, _d, _d, _d, _d, _i,
                             _vp, _sz, _vp]
_lib.dmuon_adamw.restype = _i
_int64 = ctypes.c_int64
_FfnP, _XentP = ctypes.POINTER(FfnShape), ctypes.POINTER(XentShape)
_lib.dmuon_act8_save.argtypes = [_int64, _int64, _vp, _int64, _i, _vp, _vp, _vp]
_lib.dmuon_act8_save.restype = _i
_lib.dmuon_act8_load.argtypes = [_int64, _int64, _vp, _vp, _vp, _int64, _i, _vp]
_lib.dmuon_act8_load.restype = _i
_lib.dmuon_ffn_workspace_bytes.argtypes = [_FfnP, _i]
_lib.dmuon_ffn_workspace_bytes.restype = _sz
_lib.dmuon_ffn_forward.argtypes = [_FfnP, _vp, _int64, _vp, _vp, _vp, _vp, _int64, _VPP, _vp, _sz, _vp]
_lib.dmuon_ffn_forward.restype = _i
_lib.dmuon_ffn_backward.argtypes = [_FfnP, _vp, _int64, _vp, _int64, _vp, _vp, _vp, _VPP, _vp, _int64,
                                    _vp, _vp, _vp, _vp, _sz, _vp]
_lib.dmuon_ffn_backward.restype = _i
_lib.dmuon_xent_workspace_bytes.argtypes = [_XentP, _i]
_lib.dmuon_xent_workspace_bytes.restype = _sz
_lib.dmuon_xent.argtypes = [_XentP, _vp, _int64, _vp, _vp, _vp, _vp, _vp, _vp, _int64, _vp, _vp, _sz,
                            _vp]
_lib.dmuon_xent.restype = _i
_lib.dmuon_stream_status.argtypes = [_vp, _vp]
_lib.dmuon_stream_status.restype = _i
_lib.dmuon_debug_wait_timeout.argtypes = [_vp, _sz, _i, _vp]
_lib.dmuon_debug_wait_timeout.restype = _i
_lib.dmuon_status_string.argtypes = [_i]
_lib.dmuon_status_string.restype = ctypes.c_char_p
_lib.dmuon_version.argtypes = []
_lib.dmuon_version.restype = _i
_lib.dmuon_launch_count.argtypes = [_i]
_lib.dmuon_launch_count.restype = ctypes.c_longlong
_lib.dmuon_trace_begin.argtypes = [_vp, _sz]
_lib.dmuon_trace_begin.restype = _i
_lib.dmuon_trace_end.argtypes = []
_lib.dmuon_trace_end.restype = ctypes.c_longlong
TRACE_RECORD_BYTES = 72


class DMuonError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {status_string(status)} ({status})")
        self.status = status


def lib() -> ctypes.CDLL:
    return _lib


def library_path() -> str:
    return _LIB_PATH


def status_string(status: int) -> str:
    return _lib.dmuon_status_string(int(status)).decode()


def version() -> int:
    return int(_lib.dmuon_version())


def launch_count(reset: bool = False) -> int:
    """Kernels the library launched from this host thread since the last reset."""
    return int(_lib.dmuon_launch_count(1 if reset else 0))


def _check(status: int, where: str) -> None:
    if status != OK:
        raise DMuonError(status, where)


def _shapes(shapes: Sequence[Tuple[int, int]]):
    arr = (Shape * max(1, len(shapes)))()
    for i, (r, c) in enumerate(shapes):
        arr[i].rows, arr[i].cols = int(r), int(c)
    return arr


def _ptrs(ts) -> ctypes.Array:
    arr = (ctypes.c_void_p * max(1, len(ts)))()
    for i, t in enumerate(ts):
        arr[i] = t if isinstance(t, int) else t.data_ptr()
    return arr


def _i64(vals) -> ctypes.Array:
    arr = (ctypes.c_int64 * max(1, len(vals)))()
    for i, v in enumerate(vals):
        arr[i] = int(v)
    return arr


def _dtype(t) -> int:
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return F32
    raise TypeError(f"unsupported dtype {t.dtype}: expected bfloat16 or float32")


# handle of the current stream without building a Stream object (2.9 us a call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> int:
    if stream is None:
        if _raw_stream is not None and torch.cuda.is_initialized():
            return _raw_stream(torch._C._cuda_getDevice())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _addr(t) -> int:
    return t if isinstance(t, int) else t.data_ptr()


# ------------------------------------------------------------------ calls
def plan(shapes: Sequence[Tuple[int, int]], n_owners: int = 1) -> Tuple[List[int], List[int], List[int]]:
    """Owner map, packed offsets and owner buffer sizes (host only)."""
    n = len(shapes)
    own = (ctypes.c_int * max(1, n))()
    off = (ctypes.c_int64 * max(1, n))()
    oel = (ctypes.c_int64 * max(1, n_owners))()
    _check(_lib.dmuon_plan(n, _shapes(shapes), int(n_owners), own, off, oel), "dmuon_plan")
    return list(own[:n]), list(off[:n]), list(oel[:n_owners])


def workspace_bytes(shapes: Sequence[Tuple[int, int]], variant: int = NS_STANDARD) -> int:
    return int(_lib.dmuon_workspace_bytes(len(shapes), _shapes(shapes), int(variant)))


def ns_variant_for(shape: Tuple[int, int], ns_steps: int, variant: int = NS_GRAM) -> int:
    """The Newton-Schulz form (NS_STANDARD or NS_GRAM) a call with `variant`
    runs on one matrix of this shape at `ns_steps` steps (host only)."""
    st = int(_lib.dmuon_ns_variant_for(int(shape[0]), int(shape[1]), int(ns_steps), int(variant)))
    if st < 0:
        raise DMuonError(st, "dmuon_ns_variant_for")
    return st


def pack(shapes, grads, momenta, beta, packed, offsets, workspace, stream=None) -> None:
    n = len(shapes)
    gdt = _dtype(grads[0]) if n else BF16
    _check(_lib.dmuon_pack(n, _shapes(shapes), _ptrs(grads), gdt, _ptrs(momenta), float(beta),
                           _addr(packed), _i64(offsets), _addr(workspace), workspace.numel()
                           if hasattr(workspace, "numel") else 0, _stream(stream)), "dmuon_pack")


def ns_batched(shapes, packed, offsets, workspace, ns_steps: int = 5, variant: int = NS_STANDARD,
               abc: Optional[Sequence[float]] = None, eps: float = 1e-7,
               use_pack_norms: bool = False, stream=None, ws_bytes: Optional[int] = None) -> None:
    n = len(shapes)
    abc_arr = None if abc is None else (ctypes.c_float * 3)(*[float(v) for v in abc])
    wsb = ws_bytes if ws_bytes is not None else workspace.numel()
    _check(_lib.dmuon_ns_batched(n, _shapes(shapes), _addr(packed), _i64(offsets), int(ns_steps),
                                 int(variant), abc_arr, float(eps), int(bool(use_pack_norms)),
                                 _addr(workspace), wsb, _stream(stream)), "dmuon_ns_batched")


def ns_batched_noalloc(shapes, packed, offsets, ns_steps: int = 5, variant: int = NS_STANDARD,
                       abc: Optional[Sequence[float]] = None, eps: float = 1e-7,
                       stream=None) -> None:
    """dmuon_ns_batched on the library's built-in scratch array (no workspace,
    no device allocation); problems up to NOALLOC_SCRATCH_BYTES of workspace."""
    abc_arr = None if abc is None else (ctypes.c_float * 3)(*[float(v) for v in abc])
    _check(_lib.dmuon_ns_batched_noalloc(len(shapes), _shapes(shapes), _addr(packed),
                                         _i64(offsets), int(ns_steps), int(variant), abc_arr,
                                         float(eps), _stream(stream)),
           "dmuon_ns_batched_noalloc")


def noalloc_status(stream=None) -> int:
    """Synchronise the stream and report (and clear) the error word of the
    built-in scratch array used by :func:`ns_batched_noalloc`."""
    return int(_lib.dmuon_noalloc_status(_stream(stream)))


def unpack_update(shapes, weights, lr, packed, offsets, workspace, stream=None) -> None:
    n = len(shapes)
    wdt = _dtype(weights[0]) if n else BF16
    _check(_lib.dmuon_unpack_update(n, _shapes(shapes), _ptrs(weights), wdt, float(lr),
                                    _addr(packed), _i64(offsets), _addr(workspace),
                                    workspace.numel(), _stream(stream)), "dmuon_unpack_update")


def muon_step(shapes, grads, momenta, weights, packed, offsets, workspace, lr: float = 0.02,
              beta: float = 0.95, ns_steps: int = 5, variant: int = NS_STANDARD,
              stream=None) -> None:
    n = len(shapes)
    gdt = _dtype(grads[0]) if n else BF16
    wdt = _dtype(weights[0]) if n else BF16
    _check(_lib.dmuon_muon_step(n, _shapes(shapes), _ptrs(grads), gdt, _ptrs(momenta),
                                _ptrs(weights), wdt, float(lr), float(beta), int(ns_steps),
                                int(variant), _addr(packed), _i64(offsets), _addr(workspace),
                                workspace.numel(), _stream(stream)), "dmuon_muon_step")


def adamw_workspace_bytes(n: int) -> int:
    return int(_lib.dmuon_adamw_workspace_bytes(int(n)))


def adamw(params, grads, exp_avgs, exp_avg_sqs, step: int, workspace, lr: float = 1e-3,
          betas=(0.9, 0.999), eps: float = 1e-8, weight_decay: float = 0.01,
          stream=None) -> None:
    """One AdamW step over a list of tensors (one kernel launch)."""
    n = len(params)
    pdt = _dtype(params[0]) if n else F32
    gdt = _dtype(grads[0]) if n else F32
    numel = _i64([p.numel() for p in params])
    _check(_lib.dmuon_adamw(n, numel, _ptrs(params), pdt, _ptrs(grads), gdt, _ptrs(exp_avgs),
                            _ptrs(exp_avg_sqs), float(lr), float(betas[0]), float(betas[1]),
                            float(eps), float(weight_decay), int(step), _addr(workspace),
                            workspace.numel(), _stream(stream)), "dmuon_adamw")


def stream_status(workspace=None, stream=None) -> int:
    return int(_lib.dmuon_stream_status(_stream(stream),
                                        None if workspace is None else _addr(workspace)))


def debug_wait_timeout(workspace, budget_us: int, stream=None) -> None:
    """Make a bounded device wait run out; workspace None targets the built-in
    scratch array of :func:`ns_batched_noalloc`."""
    ws = None if workspace is None else _addr(workspace)
    nbytes = 0 if workspace is None else workspace.numel()
    _check(_lib.dmuon_debug_wait_timeout(ws, nbytes, int(budget_us), _stream(stream)),
           "dmuon_debug_wait_timeout")


def trace_begin(buffer) -> None:
    """Record one timestamp record per CTA of every product launch into
    `buffer` (a uint8 CUDA tensor) until :func:`trace_end`."""
    _check(_lib.dmuon_trace_begin(_addr(buffer), buffer.numel()), "dmuon_trace_begin")


def trace_end(buffer):
    """Stop tracing; return the records as a dict of int64 CPU tensors (read
    after the traced work has completed)."""
    n = int(_lib.dmuon_trace_end())
    raw = buffer[:n * TRACE_RECORD_BYTES].cpu()
    u32 = raw.view(torch.int32).view(n, 18).to(torch.int64) & 0xFFFFFFFF
    u64 = raw.view(torch.int64).view(n, 9)
    return {"launch": u32[:, 0], "cta": u32[:, 1], "kind": u32[:, 2], "tiles": u32[:, 3],
            "t_entry": u64[:, 2], "t_mma_first": u64[:, 3], "t_mma_last": u64[:, 4],
            "t_exit": u64[:, 5], "mma_span_cycles": u64[:, 6], "wait_operand_cycles": u64[:, 7],
            "wait_accum_cycles": u64[:, 8]}


class MuonOwner:
    """One owner's Muon state for a fixed list of matrix shapes.

    Holds the packed bf16 buffer and the workspace (both allocated through
    PyTorch), and runs :func:`muon_step` on caller tensors.  Home page ("What
    DMuon Can Do"): each owner runs Muon once per step for the matrices it owns;
    "Z2 vs Z3 Modes": those matrices share one contiguous packed buffer.
    """

    def __init__(self, shapes: Sequence[Tuple[int, int]], n_owners: int = 1,
                 variant: int = NS_STANDARD, device="cuda"):
        self.shapes = [(int(r), int(c)) for r, c in shapes]
        self.variant = int(variant)
        self.owner_of, self.offsets, self.owner_elems = plan(self.shapes, n_owners)
        total = max(sum(self.owner_elems), PACK_ALIGN_ELEMS)
        self.packed = torch.empty(total, dtype=torch.bfloat16, device=device)
        self.ws_bytes = workspace_bytes(self.shapes, self.variant)
        if self.ws_bytes == 0:
            raise DMuonError(ERR_INVALID_ARG, "dmuon_workspace_bytes")
        self.workspace = torch.zeros(self.ws_bytes, dtype=torch.uint8, device=device)

    def step(self, grads, momenta, weights, lr: float = 0.02, beta: float = 0.95,
             ns_steps: int = 5, stream=None) -> None:
        muon_step(self.shapes, grads, momenta, weights, self.packed, self.offsets, self.workspace,
                  lr=lr, beta=beta, ns_steps=ns_steps, variant=self.variant, stream=stream)

    def packed_view(self, i: int) -> torch.Tensor:
        r, c = self.shapes[i]
        o = self.offsets[i]
        return self.packed[o:o + r * c].view(r, c)

    def status(self, stream=None) -> int:
        return stream_status(self.workspace, stream)


# ------------------------------------------------------------------ training-side operators
# Tensors and workspace lie on the current device.
# current device without torch.cuda's check that CUDA is initialised (a tensor on one shows it)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _launch_device(t: torch.Tensor, what: str) -> int:
    """Index of the device that `t` lies on, which has to be the current one: that is where
    the library launches."""
    dev = t.get_device()            # -1: not on a GPU
    if dev < 0:
        raise ValueError(f"{what}: expected a CUDA tensor")
    now = _current_device()
    if dev != now:
        raise ValueError(f"{what} is on cuda:{dev}, the current device is cuda:{now}")
    return dev


def _launch_stream(stream, dev: int) -> int:
    """_stream(stream), where `dev` is known to be the current device."""
    return _raw_stream(dev) if stream is None and _raw_stream is not None else _stream(stream)


def _elsewhere(t: torch.Tensor, dev: Optional[int], what: str) -> ValueError:
    return ValueError(f"{what}: expected a CUDA tensor" +
                      (f" on cuda:{dev}, got one on {t.device}" if dev is not None else ""))


def _bf16_rows(t: torch.Tensor, rows: int, cols: int, what: str, dev: Optional[int] = None) -> int:
    """Check a (rows, cols) bf16 token matrix (on device `dev`); its row pitch in elements."""
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{what}: unsupported dtype {t.dtype}: expected bfloat16")
    if t.shape != (rows, cols):
        raise ValueError(f"{what}: expected shape ({rows}, {cols}), got {tuple(t.shape)}")
    at = t.get_device()
    if at < 0 or at != (at if dev is None else dev):
        raise _elsewhere(t, dev, what)
    ld, unit = t.stride()
    if rows <= 1 or cols == 0:
        ld = cols
    if (cols > 1 and unit != 1) or ld < cols:
        raise ValueError(f"{what}: the elements of a row must be contiguous, rows must not overlap")
    return ld


def _dense(t: torch.Tensor, dtype, shape, what: str, dev: Optional[int] = None) -> int:
    """Check a contiguous CUDA tensor (on device `dev`); its address."""
    if t.dtype != dtype:
        raise TypeError(f"{what}: unsupported dtype {t.dtype}: expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{what}: expected shape {shape}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{what}: expected a contiguous tensor")
    at = t.get_device()
    if at < 0 or at != (at if dev is None else dev):
        raise _elsewhere(t, dev, what)
    return t.data_ptr()


def _act8_blocks(cols: int) -> int:
    return (cols + ACT8_BLOCK - 1) // ACT8_BLOCK


def act8_empty(rows: int, cols: int, device="cuda") -> Tuple[torch.Tensor, torch.Tensor]:
    """Uninitialised (codes, scales) of an 8-bit activation of shape (rows, cols)."""
    return (torch.empty((rows, cols), dtype=torch.int8, device=device),
            torch.empty((rows, _act8_blocks(cols)), dtype=torch.bfloat16, device=device))


def _act8_args(t: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, where: str):
    if t.dim() != 2:
        raise ValueError(f"{where}: expected a 2-D tensor, got {tuple(t.shape)}")
    rows, cols = t.shape
    dt = _dtype(t)
    ld, unit = t.stride()
    if rows <= 1:
        ld = cols
    if (cols > 1 and unit != 1) or ld < cols:
        raise ValueError(f"{where}: expected a tensor whose rows are contiguous")
    dev = _launch_device(t, where)
    return (dev, rows, cols, dt, ld, _dense(codes, torch.int8, (rows, cols), "codes", dev),
            _dense(scales, torch.bfloat16, (rows, _act8_blocks(cols)), "scales", dev))


def act8_save(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, stream=None) -> None:
    """Keep a 2-D activation (bf16 or fp32) as 8-bit codes, 32 columns to a scale."""
    dev, rows, cols, dt, ld, c, s = _act8_args(x, codes, scales, "act8_save")
    _check(_lib.dmuon_act8_save(rows, cols, x.data_ptr(), ld, dt, c, s, _launch_stream(stream, dev)),
           "dmuon_act8_save")


def act8_load(codes: torch.Tensor, scales: torch.Tensor, out: torch.Tensor, stream=None) -> None:
    """Bring an 8-bit activation back into `out` (bf16 or fp32)."""
    dev, rows, cols, dt, ld, c, s = _act8_args(out, codes, scales, "act8_load")
    _check(_lib.dmuon_act8_load(rows, cols, c, s, out.data_ptr(), ld, dt, _launch_stream(stream, dev)),
           "dmuon_act8_load")


class GatedFFN:
    """Gated feed-forward block y = (act(x Wg^T) * (x Wu^T)) Wd^T and its backward
    pass, for up to `max_tokens` tokens.  Holds the workspace; tensors are the
    caller's, bf16, weights as PyTorch parameters (out, in).  The weight gradients
    are those the owner's step takes for the gate, up and down projections.

    `save` says what forward keeps for backward: SAVE_NONE, SAVE_BF16 or SAVE_ACT8
    (see :meth:`empty_saved`).  `backward=False` sizes the workspace for forward only.
    """

    def __init__(self, max_tokens: int, hidden: int, ffn: int, activation: int = ACT_SILU,
                 save: int = SAVE_BF16, backward: Optional[bool] = None, device="cuda"):
        self.max_tokens, self.hidden, self.ffn = int(max_tokens), int(hidden), int(ffn)
        self.activation, self.save = int(activation), int(save)
        self.with_backward = self.save != SAVE_NONE if backward is None else bool(backward)
        shape = self._shape(self.max_tokens)
        nbytes = int(_lib.dmuon_ffn_workspace_bytes(ctypes.byref(shape), int(self.with_backward)))
        if nbytes == 0:
            raise DMuonError(ERR_INVALID_ARG, "dmuon_ffn_workspace_bytes")
        self.workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
        self.workspace[:256].zero_()

    def _shape(self, tokens: int) -> FfnShape:
        return FfnShape(tokens, self.hidden, self.ffn, self.activation, self.save)

    def empty_saved(self, tokens: int) -> Tuple[torch.Tensor, ...]:
        """Uninitialised tensors for what forward keeps of `tokens` tokens: (),
        (gate, up), or (gate codes, gate scales, up codes, up scales)."""
        if self.save == SAVE_NONE:
            return ()
        dev = self.workspace.device
        if self.save == SAVE_BF16:
            return tuple(torch.empty((tokens, self.ffn), dtype=torch.bfloat16, device=dev)
                         for _ in range(2))
        return act8_empty(tokens, self.ffn, dev) + act8_empty(tokens, self.ffn, dev)

    def _tokens(self, x: torch.Tensor) -> int:
        t = x.shape[0] if x.dim() == 2 else -1
        if t < 0 or t > self.max_tokens:
            raise ValueError(f"x: expected (tokens <= {self.max_tokens}, {self.hidden}), "
                             f"got {tuple(x.shape)}")
        return t

    def _weights(self, dev: int, w_gate, w_up, w_down, what=""):
        bf, d, f = torch.bfloat16, self.hidden, self.ffn
        return (_dense(w_gate, bf, (f, d), what + "w_gate", dev),
                _dense(w_up, bf, (f, d), what + "w_up", dev),
                _dense(w_down, bf, (d, f), what + "w_down", dev))

    def _saved(self, saved, t: int, dev: int):
        saved = tuple(saved) if saved is not None else ()
        want = {SAVE_NONE: 0, SAVE_BF16: 2, SAVE_ACT8: 4}[self.save]
        if len(saved) != want:
            raise ValueError(f"saved: expected {want} tensors, got {len(saved)}")
        if self.save == SAVE_BF16:
            kinds = [(torch.bfloat16, (t, self.ffn))] * 2
        else:
            kinds = [(torch.int8, (t, self.ffn)), (torch.bfloat16, (t, _act8_blocks(self.ffn)))] * 2
        arr = (ctypes.c_void_p * 4)()
        for i, s in enumerate(saved):
            arr[i] = _dense(s, kinds[i][0], kinds[i][1], f"saved[{i}]", dev)
        return arr

    def forward(self, x, w_gate, w_up, w_down, y, saved=None, stream=None) -> None:
        """y <- block(x); x and y are (tokens, hidden), `saved` from :meth:`empty_saved`."""
        t = self._tokens(x)
        dev = _launch_device(self.workspace, "the workspace")
        x_ld, y_ld = (_bf16_rows(v, t, self.hidden, n, dev) for v, n in ((x, "x"), (y, "y")))
        wg, wu, wd = self._weights(dev, w_gate, w_up, w_down)
        shape = self._shape(t)
        _check(_lib.dmuon_ffn_forward(ctypes.byref(shape), x.data_ptr(), x_ld, wg, wu, wd,
                                      y.data_ptr(), y_ld, self._saved(saved, t, dev),
                                      self.workspace.data_ptr(), self.workspace.numel(),
                                      _launch_stream(stream, dev)), "dmuon_ffn_forward")

    def backward(self, dy, x, w_gate, w_up, w_down, saved, dx, dw_gate, dw_up, dw_down,
                 stream=None) -> None:
        """Gradients of x and the three weights from dy and what forward kept."""
        if not self.with_backward:
            raise ValueError("this GatedFFN was made without a backward pass")
        t = self._tokens(x)
        d, dev = self.hidden, _launch_device(self.workspace, "the workspace")
        dy_ld, x_ld = _bf16_rows(dy, t, d, "dy", dev), _bf16_rows(x, t, d, "x", dev)
        dx_ld = _bf16_rows(dx, t, d, "dx", dev)
        wg, wu, wd = self._weights(dev, w_gate, w_up, w_down)
        gg, gu, gd = self._weights(dev, dw_gate, dw_up, dw_down, "d")
        shape = self._shape(t)
        _check(_lib.dmuon_ffn_backward(ctypes.byref(shape), dy.data_ptr(), dy_ld, x.data_ptr(),
                                       x_ld, wg, wu, wd, self._saved(saved, t, dev), dx.data_ptr(),
                                       dx_ld, gg, gu, gd, self.workspace.data_ptr(),
                                       self.workspace.numel(), _launch_stream(stream, dev)),
               "dmuon_ffn_backward")

    def status(self, stream=None) -> int:
        return stream_status(self.workspace, stream)


class LinearXent:
    """Softmax cross entropy of hidden W^T against one target per token, for up to
    `max_tokens` tokens, without keeping the logits; with `grads` also the
    gradients of the hidden states and of the head W (vocab, hidden).  Holds the
    workspace; hidden, W and their gradients are bf16, losses fp32, targets int64.
    A target outside [0, vocab) masks its token.
    """

    def __init__(self, max_tokens: int, hidden: int, vocab: int, grads: bool = True,
                 device="cuda"):
        self.max_tokens, self.hidden, self.vocab = int(max_tokens), int(hidden), int(vocab)
        self.grads = bool(grads)
        shape = XentShape(self.max_tokens, self.hidden, self.vocab)
        nbytes = int(_lib.dmuon_xent_workspace_bytes(ctypes.byref(shape), int(self.grads)))
        if nbytes == 0:
            raise DMuonError(ERR_INVALID_ARG, "dmuon_xent_workspace_bytes")
        self.workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
        self.workspace[:256].zero_()

    def _run(self, hidden, weight, target, grad_loss, loss, lse, dhidden, dweight, stream):
        t, d = (hidden.shape[0] if hidden.dim() == 2 else -1), self.hidden
        if t < 0 or t > self.max_tokens:
            raise ValueError(f"hidden: expected (tokens <= {self.max_tokens}, {d}), "
                             f"got {tuple(hidden.shape)}")
        dev = _launch_device(self.workspace, "the workspace")
        h_ld = _bf16_rows(hidden, t, d, "hidden", dev)
        w = _dense(weight, torch.bfloat16, (self.vocab, d), "weight", dev)
        tg = _dense(target, torch.int64, (t,), "target", dev)
        lo = _dense(loss, torch.float32, (t,), "loss", dev)
        ls = _dense(lse, torch.float32, (t,), "lse", dev)
        gl = dh = dw = None
        dh_ld = 0
        if grad_loss is not None:
            gl = _dense(grad_loss, torch.float32, (t,), "grad_loss", dev)
            dh_ld, dh = _bf16_rows(dhidden, t, d, "dhidden", dev), dhidden.data_ptr()
            dw = _dense(dweight, torch.bfloat16, (self.vocab, d), "dweight", dev)
        shape = XentShape(t, d, self.vocab)
        _check(_lib.dmuon_xent(ctypes.byref(shape), hidden.data_ptr(), h_ld, w, tg, gl, lo, ls, dh,
                               dh_ld, dw, self.workspace.data_ptr(), self.workspace.numel(),
                               _launch_stream(stream, dev)), "dmuon_xent")

    def loss(self, hidden, weight, target, loss, lse, stream=None) -> None:
        """Per-token loss and log-sum-exp."""
        self._run(hidden, weight, target, None, loss, lse, None, None, stream)

    def loss_and_grads(self, hidden, weight, target, grad_loss, loss, lse, dhidden, dweight,
                       stream=None) -> None:
        """The same with the gradients of sum(grad_loss * loss)."""
        if not self.grads:
            raise ValueError("this LinearXent was made without gradients")
        for name, t in (("grad_loss", grad_loss), ("dhidden", dhidden), ("dweight", dweight)):
            if t is None:
                raise TypeError(f"{name}: expected a tensor, got None")
        self._run(hidden, weight, target, grad_loss, loss, lse, dhidden, dweight, stream)

    def status(self, stream=None) -> int:
        return stream_status(self.workspace, stream)
