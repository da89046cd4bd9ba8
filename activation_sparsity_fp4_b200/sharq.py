"""Thin Python binding of ``include/sharq.h`` (ctypes).

Every function named ``sharq_*`` here calls the C function of the same name in
``_lib/libsharq.so``; the classes only allocate the caller-owned device
buffers (PyTorch tensors, the library allocates nothing) and marshal pointers,
shapes and the current CUDA stream.  All arithmetic runs in the CUDA kernels.
There is no CPU fallback: without the built library every call raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os
from typing import NamedTuple

import torch

from . import build_ext

MXFP4, NVFP4 = 0, 1
NM_2_4, NM_4_8_PAIR, NM_8_16, NM_8_16_PAIR = 0, 1, 2, 3
F32, BF16 = 0, 1
DTYPES = {torch.float32: F32, torch.bfloat16: BF16}
FORMATS = {"mxfp4": MXFP4, "nvfp4": NVFP4}
SCORES = {"softmax": 0, "sigmoid": 1}
PATTERNS = {"2:4": NM_2_4, "4:8pair": NM_4_8_PAIR, "8:16": NM_8_16, "8:16pair": NM_8_16_PAIR}
STATUS = {0: "SHARQ_OK", 1: "SHARQ_ERR_INVALID", 2: "SHARQ_ERR_UNSUPPORTED", 3: "SHARQ_ERR_CUDA",
          4: "SHARQ_ERR_TIMEOUT", 5: "SHARQ_ERR_WORKSPACE"}
SYMBOLS = ["sharq_weight_sizes", "sharq_prepared_sizes", "sharq_quantize_weight", "sharq_prepare", "sharq_linear",
           "sharq_linear_paths", "sharq_linear_grouped", "sharq_sync_status", "sharq_selftest_wait_timeout",
           "sharq_last_error", "sharq_launch_count", "sharq_prepare_noalloc", "sharq_prepare_swiglu",
           "sharq_gather_prepared", "sharq_linear_ws", "sharq_linear_workspace_size",
           "sharq_linear_grouped_gather", "sharq_fp4_sizes", "sharq_quantize_fp4", "sharq_quantize_fp4_swiglu", "sharq_gather_fp4",
           "sharq_linear_fp4", "sharq_linear_fp4_grouped", "sharq_route", "sharq_route_rows_capacity",
           "sharq_route_rows", "sharq_combine"]
NOALLOC_MAX_ROWS = 65536  # SHARQ_NOALLOC_MAX_ROWS of the C header


class SharqError(RuntimeError):
    def __init__(self, status: int, where: str, msg: str):
        super().__init__(f"{where}: {STATUS.get(status, status)}: {msg}")
        self.status = status


class sharq_weight(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales_dense", ctypes.c_void_p), ("scales_sparse", ctypes.c_void_p),
                ("tensor", ctypes.c_void_p), ("n", ctypes.c_int64), ("k", ctypes.c_int64),
                ("experts", ctypes.c_int32), ("fmt", ctypes.c_int)]


class sharq_prepared(ctypes.Structure):
    _fields_ = [("meta", ctypes.c_void_p), ("bb_codes", ctypes.c_void_p), ("bb_scales", ctypes.c_void_p),
                ("res_codes", ctypes.c_void_p), ("res_scales", ctypes.c_void_p), ("tensor", ctypes.c_void_p),
                ("t", ctypes.c_int64), ("k", ctypes.c_int64), ("fmt", ctypes.c_int), ("pat", ctypes.c_int)]


class sharq_fp4(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("row_scale", ctypes.c_void_p),
                ("rows", ctypes.c_int64), ("k", ctypes.c_int64), ("experts", ctypes.c_int32), ("fmt", ctypes.c_int)]


_lib = None


def library_path() -> str:
    return build_ext.LIB_PATH


def lib() -> ctypes.CDLL:
    """The loaded CUDA library; raises if it has not been built."""
    global _lib
    if _lib is None:
        path = build_ext.LIB_PATH
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it with `python -m activation_sparsity_fp4_b200.build_ext` "
                               "(there is no CPU fallback)")
        L = ctypes.CDLL(path)
        P, I64, I32, I, F, SZ = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_int, ctypes.c_float,
                                 ctypes.POINTER(ctypes.c_size_t))
        sig = {
            "sharq_weight_sizes": [I64, I64, I, SZ, SZ, SZ],
            "sharq_prepared_sizes": [I64, I64, I, I, SZ, SZ, SZ, SZ, SZ, SZ],
            "sharq_quantize_weight": [P, I, ctypes.POINTER(sharq_weight), P],
            "sharq_prepare": [P, I, P, F, F, ctypes.POINTER(sharq_prepared), P, ctypes.c_size_t, P],
            "sharq_prepare_noalloc": [P, I, P, F, F, ctypes.POINTER(sharq_prepared), P],
            "sharq_prepare_swiglu": [P, P, I, F, ctypes.POINTER(sharq_prepared), P],
            "sharq_gather_prepared": [ctypes.POINTER(sharq_prepared), P, ctypes.POINTER(sharq_prepared), P],
            "sharq_linear_ws": [ctypes.POINTER(sharq_prepared), ctypes.POINTER(sharq_weight), P, I, P,
                                ctypes.c_size_t, P],
            "sharq_linear_workspace_size": [ctypes.POINTER(ctypes.c_size_t)],
            "sharq_linear": [ctypes.POINTER(sharq_prepared), ctypes.POINTER(sharq_weight), P, I, P],
            "sharq_linear_paths": [ctypes.POINTER(sharq_prepared), ctypes.POINTER(sharq_weight), P, I, I32, P],
            "sharq_linear_grouped": [ctypes.POINTER(sharq_prepared), ctypes.POINTER(sharq_weight), P, P, I, P],
            "sharq_linear_grouped_gather": [ctypes.POINTER(sharq_prepared), P, I64, ctypes.POINTER(sharq_weight), P,
                                            P, I, P],
            "sharq_fp4_sizes": [I64, I64, I32, I, SZ, SZ, SZ],
            "sharq_quantize_fp4": [P, I, I64, I64, P, P, P, F, F, ctypes.POINTER(sharq_fp4), P],
            "sharq_quantize_fp4_swiglu": [P, P, I, I64, P, F, ctypes.POINTER(sharq_fp4), P],
            "sharq_gather_fp4": [ctypes.POINTER(sharq_fp4), P, P, ctypes.POINTER(sharq_fp4), P],
            "sharq_linear_fp4": [ctypes.POINTER(sharq_fp4), ctypes.POINTER(sharq_fp4), P, I, P],
            "sharq_linear_fp4_grouped": [ctypes.POINTER(sharq_fp4), ctypes.POINTER(sharq_fp4), P, P, I, P],
            "sharq_route": [P, I, I64, I32, I64, P, I, I32, I32, I32, I32, I32, F, P, P, P],
            "sharq_route_rows_capacity": [I64, I32, I32, ctypes.POINTER(I64)],
            "sharq_route_rows": [P, I64, I32, I32, P, I64, P, P, P],
            "sharq_combine": [P, I, I64, I64, P, P, I64, I32, P, P, I, P],
            "sharq_sync_status": [P],
            "sharq_selftest_wait_timeout": [ctypes.c_uint64, P],
        }
        for name, args in sig.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = ctypes.c_int
        L.sharq_last_error.restype = ctypes.c_char_p
        L.sharq_last_error.argtypes = []
        L.sharq_launch_count.restype = ctypes.c_uint64
        L.sharq_launch_count.argtypes = [ctypes.c_int]
        _lib = L
    return _lib


def _check(status: int, where: str):
    if status != 0:
        raise SharqError(status, where, lib().sharq_last_error().decode())


def _stream(stream=None):
    if stream is None:
        # the handle of torch.cuda.current_stream() without the Stream object around it (0.1 instead of 3 us a call)
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _fmt(f) -> int:
    return FORMATS[f] if isinstance(f, str) else int(f)


def _score(v) -> int:
    return SCORES[v] if isinstance(v, str) else int(v)


def _pat(p) -> int:
    return PATTERNS[p] if isinstance(p, str) else int(p)


def _dt(d) -> int:
    v = DTYPES.get(d)
    if v is not None:
        return v
    if isinstance(d, torch.dtype):
        raise ValueError(f"unsupported dtype {d}")
    return int(d)


# ------------------------------------------------------- same-name wrappers
def sharq_weight_sizes(n: int, k: int, fmt) -> tuple[int, int, int]:
    out = [ctypes.c_size_t() for _ in range(3)]
    _check(lib().sharq_weight_sizes(n, k, _fmt(fmt), *[ctypes.byref(o) for o in out]), "sharq_weight_sizes")
    return tuple(o.value for o in out)


def sharq_prepared_sizes(t: int, k: int, fmt, pat) -> tuple[int, int, int, int, int, int]:
    out = [ctypes.c_size_t() for _ in range(6)]
    _check(lib().sharq_prepared_sizes(t, k, _fmt(fmt), _pat(pat), *[ctypes.byref(o) for o in out]),
           "sharq_prepared_sizes")
    return tuple(o.value for o in out)


def sharq_quantize_weight(w_ptr: int, w_dt, out: sharq_weight, stream=None):
    _check(lib().sharq_quantize_weight(ctypes.c_void_p(w_ptr), _dt(w_dt), ctypes.byref(out), _stream(stream)),
           "sharq_quantize_weight")


def sharq_prepare(x_ptr: int, x_dt, gamma_ptr, eps: float, act_amax: float, out: sharq_prepared, workspace_ptr=None,
                  workspace_bytes: int = 0, stream=None):
    _check(lib().sharq_prepare(ctypes.c_void_p(x_ptr), _dt(x_dt), ctypes.c_void_p(gamma_ptr) if gamma_ptr else None,
                               float(eps), float(act_amax), ctypes.byref(out),
                               ctypes.c_void_p(workspace_ptr) if workspace_ptr else None, workspace_bytes,
                               _stream(stream)), "sharq_prepare")


def sharq_prepare_noalloc(x_ptr: int, x_dt, gamma_ptr, eps: float, act_amax: float, out: sharq_prepared,
                          stream=None):
    """sharq_prepare with the library's static per-row scratch: nothing is
    allocated, t <= NOALLOC_MAX_ROWS, first call per device before any stream
    capture, overlapping calls on one device race."""
    _check(lib().sharq_prepare_noalloc(ctypes.c_void_p(x_ptr), _dt(x_dt),
                                       ctypes.c_void_p(gamma_ptr) if gamma_ptr else None, float(eps), float(act_amax),
                                       ctypes.byref(out), _stream(stream)), "sharq_prepare_noalloc")


def sharq_prepare_swiglu(gate_ptr: int, up_ptr: int, dt, act_amax: float, out: sharq_prepared, stream=None):
    _check(lib().sharq_prepare_swiglu(ctypes.c_void_p(gate_ptr), ctypes.c_void_p(up_ptr), _dt(dt), float(act_amax),
                                      ctypes.byref(out), _stream(stream)), "sharq_prepare_swiglu")


def sharq_gather_prepared(src: sharq_prepared, rows_ptr: int, dst: sharq_prepared, stream=None):
    _check(lib().sharq_gather_prepared(ctypes.byref(src), ctypes.c_void_p(rows_ptr), ctypes.byref(dst),
                                       _stream(stream)), "sharq_gather_prepared")


def sharq_linear(a: sharq_prepared, w: sharq_weight, y_ptr: int, y_dt, stream=None):
    _check(lib().sharq_linear(ctypes.byref(a), ctypes.byref(w), ctypes.c_void_p(y_ptr), _dt(y_dt), _stream(stream)),
           "sharq_linear")


def sharq_linear_ws(a: sharq_prepared, w: sharq_weight, y_ptr: int, y_dt, ws_ptr: int, ws_bytes: int, stream=None):
    _check(lib().sharq_linear_ws(ctypes.byref(a), ctypes.byref(w), ctypes.c_void_p(y_ptr), _dt(y_dt),
                                 ctypes.c_void_p(ws_ptr), ctypes.c_size_t(ws_bytes), _stream(stream)),
           "sharq_linear_ws")


def sharq_linear_workspace_size() -> int:
    out = ctypes.c_size_t(0)
    _check(lib().sharq_linear_workspace_size(ctypes.byref(out)), "sharq_linear_workspace_size")
    return int(out.value)


def sharq_linear_paths(a: sharq_prepared, w: sharq_weight, y_ptr: int, y_dt, paths: int, stream=None):
    _check(lib().sharq_linear_paths(ctypes.byref(a), ctypes.byref(w), ctypes.c_void_p(y_ptr), _dt(y_dt), paths,
                                    _stream(stream)), "sharq_linear_paths")


def sharq_linear_grouped(a: sharq_prepared, w: sharq_weight, offsets_ptr: int, y_ptr: int, y_dt, stream=None):
    _check(lib().sharq_linear_grouped(ctypes.byref(a), ctypes.byref(w), ctypes.c_void_p(offsets_ptr),
                                      ctypes.c_void_p(y_ptr), _dt(y_dt), _stream(stream)), "sharq_linear_grouped")


def sharq_linear_grouped_gather(tokens: sharq_prepared, rows_ptr: int, routed_rows: int, w: sharq_weight,
                                offsets_ptr: int, y_ptr: int, y_dt, stream=None):
    _check(lib().sharq_linear_grouped_gather(ctypes.byref(tokens), ctypes.c_void_p(rows_ptr), int(routed_rows),
                                             ctypes.byref(w), ctypes.c_void_p(offsets_ptr), ctypes.c_void_p(y_ptr),
                                             _dt(y_dt), _stream(stream)), "sharq_linear_grouped_gather")


def sharq_fp4_sizes(rows: int, k: int, experts: int, fmt) -> tuple[int, int, int]:
    out = [ctypes.c_size_t() for _ in range(3)]
    _check(lib().sharq_fp4_sizes(rows, k, experts, _fmt(fmt), *[ctypes.byref(o) for o in out]), "sharq_fp4_sizes")
    return tuple(o.value for o in out)


def sharq_quantize_fp4(x_ptr: int, x_dt, x_rows: int, x_stride: int, rows_ptr, count_ptr, gamma_ptr, eps: float,
                       amax: float, out: sharq_fp4, stream=None):
    _check(lib().sharq_quantize_fp4(x_ptr, _dt(x_dt), x_rows, x_stride, rows_ptr, count_ptr, gamma_ptr, eps, amax,
                                    ctypes.byref(out), _stream(stream)), "sharq_quantize_fp4")


def sharq_quantize_fp4_swiglu(gate_ptr: int, up_ptr: int, dt, stride: int, count_ptr, amax: float, out: sharq_fp4,
                              stream=None):
    _check(lib().sharq_quantize_fp4_swiglu(gate_ptr, up_ptr, _dt(dt), stride, count_ptr, amax, ctypes.byref(out),
                                           _stream(stream)), "sharq_quantize_fp4_swiglu")


def sharq_gather_fp4(src: sharq_fp4, rows_ptr: int, count_ptr, dst: sharq_fp4, stream=None):
    _check(lib().sharq_gather_fp4(ctypes.byref(src), rows_ptr, count_ptr, ctypes.byref(dst), _stream(stream)),
           "sharq_gather_fp4")


def sharq_linear_fp4(x: sharq_fp4, w: sharq_fp4, y_ptr: int, y_dt, stream=None):
    _check(lib().sharq_linear_fp4(ctypes.byref(x), ctypes.byref(w), y_ptr, _dt(y_dt), _stream(stream)),
           "sharq_linear_fp4")


def sharq_linear_fp4_grouped(x: sharq_fp4, w: sharq_fp4, offsets_ptr: int, y_ptr: int, y_dt, stream=None):
    _check(lib().sharq_linear_fp4_grouped(ctypes.byref(x), ctypes.byref(w), offsets_ptr, y_ptr, _dt(y_dt),
                                          _stream(stream)), "sharq_linear_fp4_grouped")


def sharq_route(logits_ptr: int, dt, t: int, experts: int, stride: int, bias_ptr, score, groups: int, top_groups: int,
                group_top: int, top_k: int, renormalize: bool, scale: float, ids_ptr: int, weights_ptr: int,
                stream=None):
    _check(lib().sharq_route(logits_ptr, _dt(dt), t, experts, stride, bias_ptr, _score(score), groups, top_groups,
                             group_top, top_k, 1 if renormalize else 0, scale, ids_ptr, weights_ptr, _stream(stream)),
           "sharq_route")


@functools.lru_cache(maxsize=1024)
def sharq_route_rows_capacity(t: int, top_k: int, experts: int) -> int:
    out = ctypes.c_int64(0)
    _check(lib().sharq_route_rows_capacity(t, top_k, experts, ctypes.byref(out)), "sharq_route_rows_capacity")
    return int(out.value)


def sharq_route_rows(ids_ptr: int, t: int, top_k: int, experts: int, rows_ptr: int, capacity: int, offsets_ptr: int,
                     slots_ptr: int, stream=None):
    _check(lib().sharq_route_rows(ids_ptr, t, top_k, experts, rows_ptr, capacity, offsets_ptr, slots_ptr,
                                  _stream(stream)), "sharq_route_rows")


def sharq_combine(y_ptr: int, y_dt, y_rows: int, n: int, slots_ptr: int, weights_ptr: int, t: int, top_k: int, add_ptr,
                  out_ptr: int, out_dt, stream=None):
    _check(lib().sharq_combine(y_ptr, _dt(y_dt), y_rows, n, slots_ptr, weights_ptr, t, top_k, add_ptr, out_ptr,
                               _dt(out_dt), _stream(stream)), "sharq_combine")


def sharq_sync_status(stream=None):
    _check(lib().sharq_sync_status(_stream(stream)), "sharq_sync_status")


def sharq_selftest_wait_timeout(timeout_ns: int, stream=None):
    _check(lib().sharq_selftest_wait_timeout(int(timeout_ns), _stream(stream)), "sharq_selftest_wait_timeout")


def sharq_last_error() -> str:
    return lib().sharq_last_error().decode()


def sharq_launch_count(reset: bool = False) -> int:
    return int(lib().sharq_launch_count(1 if reset else 0))


# ------------------------------------------------------------ buffer owners
def _alloc(nbytes: int, device) -> torch.Tensor:
    # 256-byte aligned (PyTorch's caching allocator aligns blocks to 512 bytes)
    return torch.empty(max(int(nbytes), 16), dtype=torch.uint8, device=device)


class FP4Weight:
    """Device buffers of a shared FP4 weight (one or ``experts`` stacked)."""

    def __init__(self, n: int, k: int, fmt, experts: int = 1, device="cuda"):
        self.n, self.k, self.fmt, self.experts = n, k, _fmt(fmt), experts
        c, d, s = sharq_weight_sizes(n, k, self.fmt)
        self.codes = _alloc(c * experts, device)
        self.scales_dense = _alloc(d * experts, device)
        self.scales_sparse = _alloc(s * experts, device)
        self.tensor = torch.zeros(3 * experts, dtype=torch.float32, device=device)
        self.struct = sharq_weight(self.codes.data_ptr(), self.scales_dense.data_ptr(),
                                   self.scales_sparse.data_ptr(), self.tensor.data_ptr(), n, k, experts, self.fmt)

    @classmethod
    def quantize(cls, w: torch.Tensor, fmt, stream=None) -> "FP4Weight":
        """w: (n, k) or (experts, n, k), bf16 or fp32, on the GPU."""
        w = w.contiguous()
        experts = w.shape[0] if w.dim() == 3 else 1
        n, k = w.shape[-2], w.shape[-1]
        obj = cls(n, k, fmt, experts, w.device)
        sharq_quantize_weight(w.data_ptr(), w.dtype, obj.struct, stream)
        obj._src = w  # keep the source alive until the stream has consumed it
        return obj


class Prepared:
    """Device buffers of prepared activations for t rows."""

    def __init__(self, t: int, k: int, fmt, pat, device="cuda"):
        self.t, self.k, self.fmt, self.pat = t, k, _fmt(fmt), _pat(pat)
        m, bc, bs, rc, rs, ws = sharq_prepared_sizes(t, k, self.fmt, self.pat)
        self.meta = _alloc(m, device)
        self.bb_codes = _alloc(bc, device)
        self.bb_scales = _alloc(bs, device)
        self.res_codes = _alloc(rc, device)
        self.res_scales = _alloc(rs, device)
        self.tensor = torch.zeros(3, dtype=torch.float32, device=device)
        self.workspace = _alloc(ws, device) if ws else None
        self.struct = sharq_prepared(self.meta.data_ptr(), self.bb_codes.data_ptr(), self.bb_scales.data_ptr(),
                                     self.res_codes.data_ptr(), self.res_scales.data_ptr(), self.tensor.data_ptr(),
                                     t, k, self.fmt, self.pat)


def prepare(x: torch.Tensor, fmt, pat, gamma: torch.Tensor | None = None, eps: float = 1e-6, act_amax: float = 0.0,
            out: Prepared | None = None, stream=None, use_workspace: bool = True) -> Prepared:
    """Fused preprocessing of x (t, k) on the GPU; returns (or fills) a Prepared.
    use_workspace=False runs without the per-row scratch (same results)."""
    x = x.contiguous()
    t, k = x.shape
    if out is None:
        out = Prepared(t, k, fmt, pat, x.device)
    if gamma is not None:
        gamma = gamma.to(x.dtype).contiguous()
    ws = out.workspace if use_workspace else None
    sharq_prepare(x.data_ptr(), x.dtype, gamma.data_ptr() if gamma is not None else None, eps, act_amax, out.struct,
                  ws.data_ptr() if ws is not None else None, ws.numel() if ws is not None else 0, stream)
    return out


def prepare_swiglu(gate: torch.Tensor, up: torch.Tensor, fmt, pat, act_amax: float = 0.0,
                   out: Prepared | None = None, stream=None) -> Prepared:
    """Preprocessing of h = SiLU(gate) * up (t, k), formed inside the kernel."""
    gate, up = gate.contiguous(), up.to(gate.dtype).contiguous()
    assert gate.shape == up.shape
    t, k = gate.shape
    if out is None:
        out = Prepared(t, k, fmt, pat, gate.device)
    sharq_prepare_swiglu(gate.data_ptr(), up.data_ptr(), gate.dtype, act_amax, out.struct, stream)
    return out


def gather_prepared(src: Prepared, rows: torch.Tensor, out: Prepared | None = None, stream=None) -> Prepared:
    """Prepared rows laid out again: row i of the result is src row rows[i] (a zero row for
    rows[i] < 0)."""
    rows = rows.to(torch.int32).contiguous()
    if out is None:
        out = Prepared(rows.numel(), src.k, src.fmt, src.pat, src.meta.device)
    sharq_gather_prepared(src.struct, rows.data_ptr(), out.struct, stream)
    return out


def linear_workspace(device="cuda") -> torch.Tensor:
    """A zero-filled stream-K workspace for `linear(..., workspace=...)` on this device."""
    with torch.cuda.device(torch.device(device)):
        return torch.zeros(sharq_linear_workspace_size(), dtype=torch.uint8, device=device)


def linear(a: Prepared, w: FP4Weight, out_dtype=torch.bfloat16, out: torch.Tensor | None = None, paths: int = 3,
           stream=None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """y = the sparse backbone GEMM plus the dense residual GEMM, (t, n).  With a
    workspace (see `linear_workspace`) the CTA-pair GEMM may split its K loops
    over every SM pair (stream-K)."""
    if out is None:
        out = torch.empty((a.t, w.n), dtype=out_dtype, device=a.meta.device)
    if workspace is not None:
        assert paths == 3, "the stream-K form runs both paths"
        sharq_linear_ws(a.struct, w.struct, out.data_ptr(), out.dtype, workspace.data_ptr(),
                        workspace.numel() * workspace.element_size(), stream)
    elif paths == 3:
        sharq_linear(a.struct, w.struct, out.data_ptr(), out.dtype, stream)
    else:
        sharq_linear_paths(a.struct, w.struct, out.data_ptr(), out.dtype, paths, stream)
    return out


def linear_grouped(a: Prepared, w: FP4Weight, offsets: torch.Tensor, out_dtype=torch.bfloat16,
                   out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    if out is None:
        out = torch.zeros((a.t, w.n), dtype=out_dtype, device=a.meta.device)
    offsets = offsets.to(torch.int32).contiguous()
    sharq_linear_grouped(a.struct, w.struct, offsets.data_ptr(), out.data_ptr(), out.dtype, stream)
    return out


def linear_grouped_gather(tokens: Prepared, rows: torch.Tensor, w: FP4Weight, offsets: torch.Tensor,
                          out_dtype=torch.bfloat16, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Grouped linear over routed rows read by index from the token-prepared buffers
    (rows[r] = token of routed row r, < 0 for a padding row)."""
    rows = rows.to(torch.int32).contiguous()
    if out is None:
        out = torch.zeros((rows.numel(), w.n), dtype=out_dtype, device=tokens.meta.device)
    offsets = offsets.to(torch.int32).contiguous()
    sharq_linear_grouped_gather(tokens.struct, rows.data_ptr(), rows.numel(), w.struct, offsets.data_ptr(),
                                out.data_ptr(), out.dtype, stream)
    return out


# ------------------------------------- plain FP4 layers and expert routing
@contextlib.contextmanager
def _on(x: torch.Tensor, stream, used):
    """Allocate and launch where x lives: its device, and the given stream (default: that device's current one).  The
    memory of the tensors used is not given to other work before that stream is through with them."""
    if not x.is_cuda:
        raise ValueError("a CUDA tensor is needed")
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=x.device)
    if stream is not None and stream.device != x.device:
        raise ValueError(f"a stream of {stream.device} for tensors on {x.device}")
    with torch.cuda.device(x.device), torch.cuda.stream(stream):
        try:
            yield
        finally:
            if stream is not None:
                for t in (x, *used):
                    if t is not None:
                        (t.buffer if isinstance(t, FP4Matrix) else t).record_stream(stream)


class _Here:
    def __enter__(self):
        return None

    def __exit__(self, *exc):
        return None


_HERE = _Here()


def _place(x: torch.Tensor, stream, *used):
    # the usual call, on the current device's current stream, needs no context at all
    if stream is None and x.is_cuda and x.get_device() == torch._C._cuda_getDevice():
        return _HERE
    return _on(x, stream, used)


def _same_device(x: torch.Tensor, *others):
    d = x.get_device()
    for o in others:
        if o is not None and o.get_device() != d:
            raise ValueError(f"tensors on {x.device} and {o.device} in one call")


def _empty(rows: int, n: int, dtype, x: torch.Tensor) -> torch.Tensor:
    return torch.empty_strided((rows, n), (n, 1), dtype=dtype, device=x.device)  # (the cheapest of torch's forms)


def _rows_of(x: torch.Tensor, what: str) -> torch.Tensor:
    """x as rows of adjacent values whose starts are 16-byte aligned (a copy only where it is not so already)."""
    if x.dim() != 2:
        raise ValueError(f"{what} must have two dimensions, has {x.dim()}")
    size = x.element_size()
    if x.stride(1) != 1 or x.stride(0) < x.shape[1] or (x.stride(0) * size) % 16 or x.data_ptr() % 16:
        x = x.clone(memory_format=torch.contiguous_format)
    return x


def _i32(x: torch.Tensor, what: str, shape=None) -> torch.Tensor:
    if x.dtype != torch.int32:
        raise ValueError(f"{what} must be int32, is {x.dtype}")
    if shape is not None and tuple(x.shape) != tuple(shape):
        raise ValueError(f"{what} must have shape {tuple(shape)}, has {tuple(x.shape)}")
    return x.contiguous()


def _ptr(x: torch.Tensor | None):
    return None if x is None else x.data_ptr()


@functools.lru_cache(maxsize=1024)
def _fp4_layout(rows: int, k: int, experts: int, fmt: int) -> tuple[int, int, int]:
    """Offsets of the scales and row scales, and the size, of one buffer for an FP4 matrix (256-byte aligned parts)."""
    c, s, r = sharq_fp4_sizes(rows, k, experts, fmt)
    at = (c + 255) // 256 * 256
    end = at + (s + 255) // 256 * 256
    return at, end, end + r


class FP4Matrix:
    """Device buffer of a microscaled FP4 matrix: activations, or a weight of one or ``experts`` stacked blocks."""

    __slots__ = ("rows", "k", "fmt", "experts", "buffer", "struct", "_at", "_end", "__weakref__")

    def __init__(self, rows: int, k: int, fmt, experts: int = 1, device="cuda"):
        self.rows, self.k, self.fmt, self.experts = rows, k, _fmt(fmt), experts
        self._at, self._end, size = _fp4_layout(rows, k, experts, self.fmt)
        self.buffer = torch.empty_strided((size,), (1,), dtype=torch.uint8, device=device)
        p = self.buffer.data_ptr()
        self.struct = sharq_fp4(p, p + self._at, p + self._end, rows, k, experts, self.fmt)

    @property
    def device(self):
        return self.buffer.device

    @property
    def codes(self) -> torch.Tensor:
        return self.buffer[: self.experts * self.rows * self.k // 2]

    @property
    def scales(self) -> torch.Tensor:
        return self.buffer[self._at : self._at + sharq_fp4_sizes(self.rows, self.k, self.experts, self.fmt)[1]]

    @property
    def row_scale(self) -> torch.Tensor:
        return self.buffer[self._end :].view(torch.float32)


def _fp4_out(out: FP4Matrix | None, rows: int, k: int, fmt, experts: int, x: torch.Tensor) -> FP4Matrix:
    if out is None:
        return FP4Matrix(rows, k, fmt, experts, x.device)
    if (out.rows, out.k, out.fmt, out.experts, out.device) != (rows, k, _fmt(fmt), experts, x.device):
        raise ValueError("out does not fit: another shape, format or device")
    return out


def quantize_fp4(x: torch.Tensor, fmt, rows: torch.Tensor | None = None, gamma: torch.Tensor | None = None,
                 eps: float = 1e-6, amax: float = 0.0, count: torch.Tensor | None = None,
                 out: FP4Matrix | None = None, stream=None) -> FP4Matrix:
    """Rows of x as an FP4 matrix: x (t, k), or (experts, n, k) for a stacked weight.
    rows: int32 indexes of the rows to take (out of range: a zero row).  gamma: RMSNorm
    in front.  count: one int32 on the GPU; rows from it on are left as they were.
    With more rows taken than x has, x is quantized once and its FP4 rows are gathered
    (`gather_fp4`; the same bits)."""
    if x.dim() not in (2, 3):
        raise ValueError(f"x must be (t, k) or (experts, n, k), has {x.dim()} dimensions")
    _same_device(x, rows, gamma, count)
    with _place(x, stream, rows, gamma, count, out):
        experts = x.shape[0] if x.dim() == 3 else 1
        if experts > 1 and (rows is not None or count is not None):
            raise ValueError("rows and count go with one matrix, not with a stack")
        x2 = _rows_of(x if x.dim() == 2 else x.flatten(0, 1), "x")
        if gamma is not None:
            if tuple(gamma.shape) != (x2.shape[1],):
                raise ValueError(f"gamma must have shape ({x2.shape[1]},)")
            gamma = _aligned(gamma.to(x.dtype))
        if rows is not None:
            rows = _i32(rows, "rows", (rows.numel(),))
        if count is not None:
            count = _i32(count, "count", (1,))
        n_rows = x.shape[-2] if rows is None else rows.numel()
        out = _fp4_out(out, n_rows, x2.shape[1], fmt, experts, x)
        if rows is not None and n_rows > x2.shape[0]:
            tokens = FP4Matrix(x2.shape[0], x2.shape[1], fmt, 1, x.device)
            sharq_quantize_fp4(x2.data_ptr(), x.dtype, x2.shape[0], max(x2.stride(0), x2.shape[1]), None, None,
                               _ptr(gamma), eps, amax, tokens.struct)
            sharq_gather_fp4(tokens.struct, rows.data_ptr(), _ptr(count), out.struct)
            return out
        sharq_quantize_fp4(x2.data_ptr(), x.dtype, x2.shape[0], max(x2.stride(0), x2.shape[1]), _ptr(rows), _ptr(count),
                           _ptr(gamma), eps, amax, out.struct)
    return out


def gather_fp4(src: FP4Matrix, rows: torch.Tensor, count: torch.Tensor | None = None, out: FP4Matrix | None = None,
               stream=None) -> FP4Matrix:
    """FP4 rows laid out again: row i of the result is src row rows[i] (int32; out of range: a zero row)."""
    _same_device(src.buffer, rows, count)
    with _place(src.buffer, stream, rows, count, out):
        rows = _i32(rows, "rows", (rows.numel(),))
        if count is not None:
            count = _i32(count, "count", (1,))
        out = _fp4_out(out, rows.numel(), src.k, src.fmt, 1, src.buffer)
        if out is src:
            raise ValueError("rows cannot be gathered in place")
        sharq_gather_fp4(src.struct, rows.data_ptr(), _ptr(count), out.struct)
    return out


def quantize_fp4_swiglu(gate: torch.Tensor, up: torch.Tensor, fmt, amax: float = 0.0,
                        count: torch.Tensor | None = None, out: FP4Matrix | None = None, stream=None) -> FP4Matrix:
    """SiLU(gate) * up (t, k) as an FP4 matrix; the halves of one (t, 2k) product need no copy."""
    if gate.shape != up.shape or gate.dtype != up.dtype:
        raise ValueError("gate and up must have one shape and dtype")
    _same_device(gate, up, count)
    with _place(gate, stream, up, count, out):
        gate, up = _rows_of(gate, "gate"), _rows_of(up, "up")
        if gate.stride(0) != up.stride(0):
            gate, up = gate.contiguous(), up.contiguous()
        if count is not None:
            count = _i32(count, "count", (1,))
        t, k = gate.shape
        out = _fp4_out(out, t, k, fmt, 1, gate)
        sharq_quantize_fp4_swiglu(gate.data_ptr(), up.data_ptr(), gate.dtype, max(gate.stride(0), k), _ptr(count), amax,
                                  out.struct)
    return out


def _aligned(x: torch.Tensor) -> torch.Tensor:
    x = x.contiguous()
    return x if x.data_ptr() % 16 == 0 else x.clone()


def _product_out(out, rows: int, n: int, dtype, a: FP4Matrix) -> torch.Tensor:
    if out is None:
        return _empty(rows, n, dtype, a.buffer)
    if tuple(out.shape) != (rows, n) or not out.is_contiguous() or out.device != a.device:
        raise ValueError(f"out must be a contiguous ({rows}, {n}) tensor on {a.device}")
    return out


def linear_fp4(a: FP4Matrix, w: FP4Matrix, out_dtype=torch.bfloat16, out: torch.Tensor | None = None,
               stream=None) -> torch.Tensor:
    """y = a w^T, (rows of a, rows of w)."""
    _same_device(a.buffer, w.buffer)
    with _place(a.buffer, stream, w, out):
        out = _product_out(out, a.rows, w.rows, out_dtype, a)
        sharq_linear_fp4(a.struct, w.struct, out.data_ptr(), out.dtype)
    return out


def linear_fp4_grouped(a: FP4Matrix, w: FP4Matrix, offsets: torch.Tensor, out_dtype=torch.bfloat16,
                       out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Rows [offsets[e], offsets[e + 1]) of a times expert e's weight.  Rows outside every
    group are left as they were (undefined in an ``out`` allocated here)."""
    _same_device(a.buffer, w.buffer, offsets)
    with _place(a.buffer, stream, w, offsets, out):
        offsets = _i32(offsets, "offsets", (w.experts + 1,))
        out = _product_out(out, a.rows, w.rows, out_dtype, a)
        sharq_linear_fp4_grouped(a.struct, w.struct, offsets.data_ptr(), out.data_ptr(), out.dtype)
    return out


def route(logits: torch.Tensor, top_k: int, score="softmax", bias: torch.Tensor | None = None, groups: int = 1,
          top_groups: int = 1, group_top: int = 1, renormalize: bool = True, scale: float = 1.0,
          stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """Expert ids (t, top_k) int32 and weights (t, top_k) fp32 of the tokens' logits (t, experts)."""
    if logits.dim() != 2:
        raise ValueError(f"logits must be (t, experts), has {logits.dim()} dimensions")
    _same_device(logits, bias)
    with _place(logits, stream, bias):
        t, experts = logits.shape
        if logits.stride(1) != 1 or logits.stride(0) < experts:
            logits = logits.contiguous()
        if bias is not None:
            if tuple(bias.shape) != (experts,):
                raise ValueError(f"bias must have shape ({experts},)")
            bias = bias.float().contiguous()
        ids, weights = _empty(t, top_k, torch.int32, logits), _empty(t, top_k, torch.float32, logits)
        sharq_route(logits.data_ptr(), logits.dtype, t, experts, max(logits.stride(0), experts), _ptr(bias), score,
                    groups, top_groups, group_top, top_k, renormalize, scale, ids.data_ptr(), weights.data_ptr())
    return ids, weights


class RoutedRows(NamedTuple):
    """Routed-row layout of an assignment: token of each row (-1: padding), (experts + 1) offsets, row of each place."""

    rows: torch.Tensor
    offsets: torch.Tensor
    slots: torch.Tensor


def route_rows(ids: torch.Tensor, experts: int, stream=None) -> RoutedRows:
    """Rows of an assignment ids (t, top_k), grouped by expert, each group padded to 128 rows.  Nothing is read
    back: ``rows`` has the size that any assignment of this shape fits in; offsets[-1] rows of it are in use."""
    if ids.dim() != 2:
        raise ValueError(f"ids must be (t, top_k), has {ids.dim()} dimensions")
    with _place(ids, stream):
        ids = _i32(ids, "ids")
        t, top_k = ids.shape
        capacity = sharq_route_rows_capacity(t, top_k, experts)
        rows, offsets, slots = ids.new_empty((capacity,)), ids.new_empty((experts + 1,)), torch.empty_like(ids)
        sharq_route_rows(ids.data_ptr(), t, top_k, experts, rows.data_ptr(), capacity, offsets.data_ptr(),
                         slots.data_ptr())
    return RoutedRows(rows, offsets, slots)


def combine(y: torch.Tensor, slots: torch.Tensor, weights: torch.Tensor, add: torch.Tensor | None = None,
            out_dtype=None, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """out[t] = add[t] + sum_j weights[t, j] * y[slots[t, j]] (places with a slot below 0 are left out)."""
    if y.dim() != 2 or slots.dim() != 2:
        raise ValueError("y must be (rows, n), slots (t, top_k)")
    _same_device(y, slots, weights, add, out)
    with _place(y, stream, slots, weights, add, out):
        t, top_k = slots.shape
        n = y.shape[1]
        slots = _i32(slots, "slots")
        if weights.dtype != torch.float32 or tuple(weights.shape) != (t, top_k):
            raise ValueError(f"weights must be fp32 ({t}, {top_k})")
        if add is not None:
            if tuple(add.shape) != (t, n) or add.dtype != y.dtype:
                raise ValueError(f"add must be ({t}, {n}) of y's dtype")
            add = _aligned(add)
        if out is None:
            out = _empty(t, n, out_dtype or y.dtype, y)
        elif tuple(out.shape) != (t, n) or not out.is_contiguous():
            raise ValueError(f"out must be a contiguous ({t}, {n}) tensor")
        y, weights = _aligned(y), weights.contiguous()
        sharq_combine(y.data_ptr(), y.dtype, y.shape[0], n, slots.data_ptr(), weights.data_ptr(), t, top_k, _ptr(add),
                      out.data_ptr(), out.dtype)
    return out
