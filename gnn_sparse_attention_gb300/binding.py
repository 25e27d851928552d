"""Thin Python binding of the C ABI in ``include/gattn.h`` (ctypes).

Argument marshalling only: every step of the attention path runs in the CUDA
library ``_build/libgattn.so``.  There is no fallback -- if the library is not
built or cannot be loaded, every call raises.  PyTorch supplies device memory
and the current stream.
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading

import numpy as np
import torch

from . import build as _build

GATTN_OK = 0
STATUS = {0: "GATTN_OK", 1: "GATTN_ERR_INVALID_ARG", 2: "GATTN_ERR_BAD_GRAPH",
          3: "GATTN_ERR_UNSUPPORTED", 4: "GATTN_ERR_OOM", 5: "GATTN_ERR_CUDA",
          6: "GATTN_ERR_TIMEOUT"}
GATTN_F32, GATTN_BF16 = 0, 1
GATTN_SCORE_DOT, GATTN_SCORE_GATV2 = 0, 1
EXPORTED = ("gattn_plan_create", "gattn_plan_destroy", "gattn_plan_get_info",
            "gattn_plan_export", "gattn_workspace_size", "gattn_fwd", "gattn_bwd",
            "gattn_bwd_dq", "gattn_bwd_dkdv", "gattn_plan_check_errors", "gattn_fwd_noalloc",
            "gattn_plan_export_tiles", "gattn_plan_export_tile_bwd", "gattn_reorder", "gattn_permute_csr",
            "gattn_permute_rows", "gattn_pool_workspace_size", "gattn_pool_fwd",
            "gattn_pool_bwd", "gattn_spmm_workspace_size", "gattn_spmm",
            "gattn_plan_set_wait_test", "gattn_block_sums", "gattn_block_select_workspace_size",
            "gattn_block_select", "gattn_block_fwd_workspace_size", "gattn_block_fwd",
            "gattn_block_bwd_workspace_size", "gattn_block_bwd", "gattn_block_check_errors",
            "gattn_block_set_wait_test",
            "gattn_norm_workspace_size", "gattn_norm_fwd", "gattn_norm_bwd", "gattn_rotary",
            "gattn_rotary_freqs", "gattn_cache_write", "gattn_cache_read", "gattn_cache_sums",
            "gattn_cache_fwd_workspace_size", "gattn_cache_fwd", "gattn_last_error",
            "gattn_version")


class GattnError(RuntimeError):
    def __init__(self, status: int, where: str, msg: str):
        super().__init__(f"{where}: {STATUS.get(status, status)}: {msg}")
        self.status = status


class _Score(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("scale", ctypes.c_float), ("a", ctypes.c_void_p),
                ("neg_slope", ctypes.c_float)]


class _PlanOpts(ctypes.Structure):
    _fields_ = [("heavy_threshold", ctypes.c_int32), ("chunk", ctypes.c_int32),
                ("tile_enable", ctypes.c_int32), ("tile_density", ctypes.c_float)]


class _PlanInfo(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int32), ("M", ctypes.c_int64),
                ("heavy_threshold", ctypes.c_int32), ("chunk", ctypes.c_int32),
                ("n_light", ctypes.c_int64), ("n_heavy", ctypes.c_int64),
                ("n_chunks", ctypes.c_int64), ("n_light_src", ctypes.c_int64),
                ("n_heavy_src", ctypes.c_int64), ("n_src_chunks", ctypes.c_int64),
                ("max_deg", ctypes.c_int32), ("max_outdeg", ctypes.c_int32),
                ("device_bytes", ctypes.c_size_t), ("n_tiles", ctypes.c_int64),
                ("n_tile_rows", ctypes.c_int64), ("tile_edges", ctypes.c_int64),
                ("tile_min_edges", ctypes.c_int32)]


class _BlockDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("S", "Nq", "Nk", "H", "Hkv", "D", "dtype", "block",
                                              "q_block", "topk", "causal")]
    _fields_ += [("scale", ctypes.c_float), ("max_len_k", ctypes.c_int32),
                 ("seq_q", ctypes.c_void_p), ("seq_k", ctypes.c_void_p),
                 ("len_k", ctypes.c_void_p), ("idx_stride", ctypes.c_int64 * 2)]


class _NormDesc(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int64), ("F", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("kind", ctypes.c_int32), ("gate", ctypes.c_int32), ("alpha", ctypes.c_float),
                ("eps", ctypes.c_float), ("w_post", ctypes.c_void_p), ("b_post", ctypes.c_void_p),
                ("w_pre", ctypes.c_void_p), ("b_pre", ctypes.c_void_p)]


class _RotaryDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("N", "H", "Hkv", "D", "dtype", "width", "layout",
                                              "inverse", "S")]
    _fields_ += [("amp", ctypes.c_float)]
    _fields_ += [(n, ctypes.c_void_p) for n in ("freqs", "pos", "seq_q", "seq_k", "len_k")]
    _fields_ += [(n, ctypes.c_int64) for n in ("q_stride", "k_stride", "q_out_stride",
                                              "k_out_stride")]


class _CacheDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("S", "N", "Nk", "H", "Hkv", "D", "dtype", "bits",
                                              "block", "topk", "causal")]
    _fields_ += [("scale", ctypes.c_float), ("max_len_k", ctypes.c_int32),
                 ("seq_q", ctypes.c_void_p), ("seq_k", ctypes.c_void_p),
                 ("len_k", ctypes.c_void_p), ("idx_stride", ctypes.c_int64 * 2),
                 ("row_stride", ctypes.c_int64 * 2), ("k", ctypes.c_void_p),
                 ("v", ctypes.c_void_p), ("par", ctypes.c_void_p)]


_lock = threading.Lock()
_lib = None


def library_path() -> str:
    return _build.LIB


def load_library(path: str | None = None):
    """Load the CUDA library (no compute call is made).

    Without ``path`` the in-tree build is loaded once and cached for every
    call of this module.  With ``path`` that library is loaded and returned
    but not cached: the module's own calls keep using the default library
    unless the caller assigns the result to ``binding._lib``.
    """
    global _lib
    with _lock:
        if _lib is not None and path is None:
            return _lib
        p = path or _build.LIB
        if not os.path.exists(p):
            raise RuntimeError(f"gattn CUDA library not found at {p}; build it first "
                               "(python -c 'import __graft_entry__ as g; g.build()')")
        lib = ctypes.CDLL(p)
        P, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        st = ctypes.c_int
        lib.gattn_plan_create.argtypes = [P, P, i32, i64, ctypes.POINTER(_PlanOpts), P,
                                          ctypes.POINTER(P)]
        lib.gattn_plan_destroy.argtypes = [P]
        lib.gattn_plan_get_info.argtypes = [P, ctypes.POINTER(_PlanInfo)]
        lib.gattn_plan_export.argtypes = [P] + [P] * 11
        lib.gattn_workspace_size.argtypes = [P, i32, i32, ctypes.c_int, ctypes.POINTER(sz)]
        lib.gattn_fwd.argtypes = [P, i32, i32, ctypes.c_int, P, P, P, ctypes.POINTER(_Score), P,
                                  P, P, sz, P]
        lib.gattn_bwd.argtypes = [P, i32, i32, ctypes.c_int, P, P, P, ctypes.POINTER(_Score), P,
                                  P, P, P, P, P, P, P, sz, P]
        lib.gattn_bwd_dq.argtypes = [P, i32, i32, ctypes.c_int, P, P, P, ctypes.POINTER(_Score),
                                     P, P, P, P, P, P, sz, P]
        lib.gattn_bwd_dkdv.argtypes = [P, i32, i32, ctypes.c_int, P, P, P,
                                       ctypes.POINTER(_Score), P, P, P, P, P, sz, P]
        lib.gattn_plan_check_errors.argtypes = [P]
        lib.gattn_fwd_noalloc.argtypes = [P, i32, i32, ctypes.c_int, P, P, P,
                                          ctypes.POINTER(_Score), P, P, P]
        lib.gattn_plan_export_tiles.argtypes = [P] * 6
        lib.gattn_plan_export_tile_bwd.argtypes = [P, ctypes.POINTER(i64)] + [P] * 6
        lib.gattn_reorder.argtypes = [P, P, i32, i64, i32, P]
        lib.gattn_permute_csr.argtypes = [P, P, i32, i64, P, P, P]
        lib.gattn_permute_rows.argtypes = [P, P, P, i32, i64, i32, P]
        lib.gattn_pool_workspace_size.argtypes = [P, i32, ctypes.c_int, ctypes.POINTER(sz)]
        lib.gattn_pool_fwd.argtypes = [P, i32, ctypes.c_int, i32, P, P, P, P, sz, P]
        lib.gattn_pool_bwd.argtypes = [P, i32, ctypes.c_int, P, P, P, P, sz, P]
        lib.gattn_spmm_workspace_size.argtypes = [P, i32, ctypes.c_int, ctypes.POINTER(sz)]
        lib.gattn_spmm.argtypes = [P, i32, ctypes.c_int, P, P, P, i32, P, sz, P]
        lib.gattn_plan_set_wait_test.argtypes = [P, i32]
        bd, nd, psz = P, P, ctypes.POINTER(sz)  # descriptors: packed bytes or byref
        lib.gattn_block_sums.argtypes = [bd, P, P, P, P]
        lib.gattn_block_select_workspace_size.argtypes = [bd, psz]
        lib.gattn_block_select.argtypes = [bd, P, P, P, P, sz, P]
        lib.gattn_block_fwd_workspace_size.argtypes = [bd, psz]
        lib.gattn_block_fwd.argtypes = [bd] + [P] * 7 + [sz, P]
        lib.gattn_block_bwd_workspace_size.argtypes = [bd, psz]
        lib.gattn_block_bwd.argtypes = [bd] + [P] * 11 + [sz, P]
        lib.gattn_block_check_errors.argtypes = []
        lib.gattn_block_set_wait_test.argtypes = [i32]
        lib.gattn_norm_workspace_size.argtypes = [nd, psz]
        lib.gattn_norm_fwd.argtypes = [nd] + [P] * 7
        lib.gattn_norm_bwd.argtypes = [nd] + [P] * 14 + [sz, P]
        f64 = ctypes.c_double
        lib.gattn_rotary.argtypes = [P] * 6
        lib.gattn_rotary_freqs.argtypes = [i32, f64, i32, f64, f64, f64, f64, P]
        lib.gattn_cache_write.argtypes = [P] * 4
        lib.gattn_cache_read.argtypes = [P] * 5
        lib.gattn_cache_sums.argtypes = [P] * 4
        lib.gattn_cache_fwd_workspace_size.argtypes = [P, psz]
        lib.gattn_cache_fwd.argtypes = [P] * 6 + [sz, P]
        for name in EXPORTED:
            if name not in ("gattn_last_error", "gattn_version"):
                getattr(lib, name).restype = st
        lib.gattn_last_error.restype = ctypes.c_char_p
        lib.gattn_last_error.argtypes = []
        lib.gattn_version.restype = ctypes.c_char_p
        lib.gattn_version.argtypes = []
        if path is None:
            _lib = lib
        return lib


def _check(status: int, where: str):
    if status != GATTN_OK:
        raise GattnError(status, where, load_library().gattn_last_error().decode())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _dtype_code(dt):
    if dt == torch.float32:
        return GATTN_F32
    if dt == torch.bfloat16:
        return GATTN_BF16
    raise GattnError(1, "dtype", f"unsupported dtype {dt}")


class Score:
    """Score function: ``Score("dot", scale=0.0)`` or ``Score("gatv2", a=a, neg_slope=0.2)``.

    ``a`` is a CUDA fp32 tensor [H, D]; scale 0 means 1/sqrt(D).
    """

    def __init__(self, kind: str = "dot", scale: float = 0.0, a: torch.Tensor | None = None,
                 neg_slope: float = 0.2):
        if kind not in ("dot", "gatv2"):
            raise ValueError(kind)
        self.kind, self.scale, self.a, self.neg_slope = kind, scale, a, neg_slope

    def _struct(self):
        a = None
        if self.kind == "gatv2":
            if self.a is None or self.a.dtype != torch.float32 or not self.a.is_contiguous():
                raise ValueError("GATv2 needs a contiguous fp32 CUDA tensor a[H, D]")
            a = self.a.data_ptr()
        return _Score(GATTN_SCORE_DOT if self.kind == "dot" else GATTN_SCORE_GATV2,
                      float(self.scale), a, float(self.neg_slope))


class Plan:
    """Per-graph plan (``gattn_plan_create``); frees its device memory on close()."""

    def __init__(self, handle, indptr_len: int):
        self._h = handle
        self._ws = {}

    @property
    def handle(self):
        if self._h is None:
            raise RuntimeError("plan already destroyed")
        return self._h

    def info(self) -> dict:
        return gattn_plan_get_info(self)

    def workspace(self, H: int, D: int, dtype, device=None) -> torch.Tensor:
        key = (H, D, dtype)
        if key not in self._ws:
            n = gattn_workspace_size(self, H, D, dtype)
            self._ws[key] = torch.empty(max(n, 16), dtype=torch.uint8,
                                        device=device or torch.device("cuda"))
        return self._ws[key]

    def close(self):
        if self._h is not None:
            self._ws.clear()
            _check(load_library().gattn_plan_destroy(self._h), "gattn_plan_destroy")
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ----------------------------------------------------------------------------
# the C ABI, one Python function per entry point
# ----------------------------------------------------------------------------
def gattn_version() -> str:
    return load_library().gattn_version().decode()


def gattn_plan_create(indptr: torch.Tensor, indices: torch.Tensor, heavy_threshold: int = 0,
                      chunk: int = 0, stream=None, tile_enable: bool = False,
                      tile_density: float = 0.0) -> Plan:
    lib = load_library()
    for t, name in ((indptr, "indptr"), (indices, "indices")):
        if not t.is_cuda or t.dtype != torch.int32 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous int32 CUDA tensor")
    opts = _PlanOpts(int(heavy_threshold), int(chunk), int(bool(tile_enable)),
                     float(tile_density))
    h = ctypes.c_void_p()
    N = indptr.numel() - 1
    _check(lib.gattn_plan_create(_ptr(indptr), _ptr(indices) if indices.numel() else None,
                                 N, indices.numel(), ctypes.byref(opts), _stream(stream),
                                 ctypes.byref(h)), "gattn_plan_create")
    return Plan(h, indptr.numel())


def gattn_plan_get_info(plan: Plan) -> dict:
    info = _PlanInfo()
    _check(load_library().gattn_plan_get_info(plan.handle, ctypes.byref(info)),
           "gattn_plan_get_info")
    return {name: getattr(info, name) for name, _ in _PlanInfo._fields_}


def gattn_plan_export(plan: Plan) -> dict:
    info = gattn_plan_get_info(plan)
    N, M = info["N"], info["M"]
    arr = {
        "deg": np.zeros(N, np.int32), "hist": np.zeros(33, np.int32),
        "light": np.zeros(info["n_light"], np.int32),
        "chunks": np.zeros((info["n_chunks"], 3), np.int32),
        "indptrT": np.zeros(N + 1, np.int32), "csc_dst": np.zeros(M, np.int32),
        "csc_eid": np.zeros(M, np.int32), "outdeg": np.zeros(N, np.int32),
        "hist_out": np.zeros(33, np.int32), "light_src": np.zeros(info["n_light_src"], np.int32),
        "src_chunks": np.zeros((info["n_src_chunks"], 3), np.int32),
    }
    order = ("deg", "hist", "light", "chunks", "indptrT", "csc_dst", "csc_eid", "outdeg",
             "hist_out", "light_src", "src_chunks")
    ptrs = [arr[k].ctypes.data_as(ctypes.c_void_p) if arr[k].size else None for k in order]
    _check(load_library().gattn_plan_export(plan.handle, *ptrs), "gattn_plan_export")
    return arr


def gattn_plan_export_tiles(plan: Plan) -> dict:
    """Dense-tile split of a plan built with tile_enable: tiles, masks, residual CSR."""
    info = gattn_plan_get_info(plan)
    nt, N = info["n_tiles"], info["N"]
    arr = {
        "tile_rb": np.zeros(nt, np.int32), "tile_cb": np.zeros(nt, np.int32),
        "masks": np.zeros((nt, 128, 4), np.uint32), "indptr_r": np.zeros(N + 1, np.int32),
        "indices_r": np.zeros(info["M"] - info["tile_edges"], np.int32),
    }
    order = ("tile_rb", "tile_cb", "masks", "indptr_r", "indices_r")
    ptrs = [arr[k].ctypes.data_as(ctypes.c_void_p) if arr[k].size else None for k in order]
    _check(load_library().gattn_plan_export_tiles(plan.handle, *ptrs), "gattn_plan_export_tiles")
    return arr


def gattn_plan_export_tile_bwd(plan: Plan) -> dict:
    """Structures of the tile backward: tiles by column block, transposed
    masks, and the residual CSC."""
    info = gattn_plan_get_info(plan)
    nt, N = info["n_tiles"], info["N"]
    lib = load_library()
    n = ctypes.c_int64(0)
    _check(lib.gattn_plan_export_tile_bwd(plan.handle, ctypes.byref(n), *([None] * 6)),
           "gattn_plan_export_tile_bwd")
    nc = int(n.value)
    arr = {
        "tcol_cb": np.zeros(nc, np.int32), "tcol_ptr": np.zeros(nc + 1, np.int32),
        "tcol_tile": np.zeros(nt, np.int32), "masks_t": np.zeros((nt, 128, 4), np.uint32),
        "indptrT_r": np.zeros(N + 1, np.int32),
        "csc_dst_r": np.zeros(info["M"] - info["tile_edges"], np.int32),
    }
    order = ("tcol_cb", "tcol_ptr", "tcol_tile", "masks_t", "indptrT_r", "csc_dst_r")
    ptrs = [arr[k].ctypes.data_as(ctypes.c_void_p) if arr[k].size else None for k in order]
    _check(lib.gattn_plan_export_tile_bwd(plan.handle, None, *ptrs), "gattn_plan_export_tile_bwd")
    return arr


REORDER = {"degree": 0, "rcm": 1}


def gattn_reorder(indptr: np.ndarray, indices: np.ndarray, kind: str = "rcm") -> np.ndarray:
    """Relabelling of a host CSR graph: perm[new] = old (host call)."""
    indptr = np.ascontiguousarray(indptr, dtype=np.int32)
    indices = np.ascontiguousarray(indices, dtype=np.int32)
    N = len(indptr) - 1
    perm = np.zeros(max(N, 1), np.int32)
    _check(load_library().gattn_reorder(indptr.ctypes.data, indices.ctypes.data if indices.size
                                        else None, N, int(indptr[-1]), REORDER[kind],
                                        perm.ctypes.data), "gattn_reorder")
    return perm[:N]


def gattn_permute_csr(indptr: np.ndarray, indices: np.ndarray, perm: np.ndarray):
    """The host CSR graph under a relabelling: (indptr, indices) with sorted rows."""
    indptr = np.ascontiguousarray(indptr, dtype=np.int32)
    indices = np.ascontiguousarray(indices, dtype=np.int32)
    perm = np.ascontiguousarray(perm, dtype=np.int32)
    N, M = len(indptr) - 1, int(indptr[-1])
    ptr = np.zeros(N + 1, np.int32)
    idx = np.zeros(max(M, 1), np.int32)
    _check(load_library().gattn_permute_csr(indptr.ctypes.data, indices.ctypes.data if M else None,
                                            N, M, perm.ctypes.data if N else None, ptr.ctypes.data,
                                            idx.ctypes.data), "gattn_permute_csr")
    return ptr, idx[:M]


def gattn_permute_rows(x: torch.Tensor, perm: torch.Tensor, inverse: bool = False, out=None,
                       stream=None) -> torch.Tensor:
    """Rows of a CUDA tensor under perm: out[i] = x[perm[i]] (or out[perm[i]] = x[i])."""
    if not x.is_cuda or not x.is_contiguous() or perm.dtype != torch.int32 or not perm.is_cuda:
        raise ValueError("x must be a contiguous CUDA tensor and perm a CUDA int32 tensor")
    out = torch.empty_like(x) if out is None else out
    N = x.shape[0]
    row_bytes = x[0].numel() * x.element_size() if N else 16
    _check(load_library().gattn_permute_rows(_ptr(x), _ptr(out), _ptr(perm), N, row_bytes,
                                             int(bool(inverse)), _stream(stream)),
           "gattn_permute_rows")
    return out


POOL = {"max": 0, "min": 1}


def gattn_pool_workspace_size(plan: Plan, F: int, dtype) -> int:
    n = ctypes.c_size_t()
    _check(load_library().gattn_pool_workspace_size(plan.handle, F, _dtype_code(dtype),
                                                     ctypes.byref(n)), "gattn_pool_workspace_size")
    return n.value


def _pool_ws(plan: Plan, F: int, dtype, device, workspace):
    if workspace is not None:
        return workspace
    return torch.empty(gattn_pool_workspace_size(plan, F, dtype), dtype=torch.uint8,
                       device=device)


def gattn_pool_fwd(plan: Plan, x: torch.Tensor, op: str = "max", out=None, arg=None,
                   workspace=None, stream=None):
    """Max / min pooling of source rows: returns (out [N, F] in x's dtype, arg int32 [N, F])."""
    if not x.is_cuda or not x.is_contiguous():
        raise ValueError("x must be a contiguous CUDA tensor [N, F]")
    x2 = x.reshape(x.shape[0], -1)
    F = x2.shape[1]
    out = torch.empty_like(x2) if out is None else out
    arg = torch.empty(x2.shape, dtype=torch.int32, device=x.device) if arg is None else arg
    ws = _pool_ws(plan, F, x.dtype, x.device, workspace)
    _check(load_library().gattn_pool_fwd(plan.handle, F, _dtype_code(x.dtype), POOL[op], _ptr(x2),
                                         _ptr(out), _ptr(arg), _ptr(ws), ws.numel(),
                                         _stream(stream)), "gattn_pool_fwd")
    return out.view(x.shape), arg.view(x.shape)


def gattn_pool_bwd(plan: Plan, arg: torch.Tensor, dout: torch.Tensor, dx=None, workspace=None,
                   stream=None):
    """Gradient of pooling: dx[j] collects dout[i] wherever arg[i] == j."""
    d2 = dout.contiguous().reshape(dout.shape[0], -1)
    F = d2.shape[1]
    dx = torch.empty_like(d2) if dx is None else dx
    ws = _pool_ws(plan, F, dout.dtype, dout.device, workspace)
    _check(load_library().gattn_pool_bwd(plan.handle, F, _dtype_code(dout.dtype),
                                         _ptr(arg.contiguous()), _ptr(d2), _ptr(dx), _ptr(ws),
                                         ws.numel(), _stream(stream)), "gattn_pool_bwd")
    return dx.view(dout.shape)


def gattn_spmm_workspace_size(plan: Plan, F: int, dtype) -> int:
    n = ctypes.c_size_t()
    _check(load_library().gattn_spmm_workspace_size(plan.handle, F, _dtype_code(dtype),
                                                     ctypes.byref(n)), "gattn_spmm_workspace_size")
    return n.value


def gattn_spmm(plan: Plan, w: torch.Tensor, x: torch.Tensor, transpose: bool = False, y=None,
               workspace=None, stream=None) -> torch.Tensor:
    """y = A x (or A^T x) with edge weights w (fp32 [M], the plan's CSR order)."""
    if not x.is_cuda or not x.is_contiguous() or w.dtype != torch.float32 or not w.is_cuda:
        raise ValueError("x must be a contiguous CUDA tensor and w a CUDA fp32 tensor")
    x2 = x.reshape(x.shape[0], -1)
    F = x2.shape[1]
    y = torch.empty_like(x2) if y is None else y
    ws = workspace
    if ws is None:
        ws = torch.empty(gattn_spmm_workspace_size(plan, F, x.dtype), dtype=torch.uint8,
                         device=x.device)
    _check(load_library().gattn_spmm(plan.handle, F, _dtype_code(x.dtype), _ptr(w.contiguous()),
                                     _ptr(x2), _ptr(y), int(bool(transpose)), _ptr(ws), ws.numel(),
                                     _stream(stream)), "gattn_spmm")
    return y.view(x.shape)


def gattn_workspace_size(plan: Plan, H: int, D: int, dtype) -> int:
    n = ctypes.c_size_t()
    _check(load_library().gattn_workspace_size(plan.handle, H, D, _dtype_code(dtype),
                                                ctypes.byref(n)), "gattn_workspace_size")
    return n.value


def _shape(Q):
    if Q.dim() != 3 or not Q.is_cuda or not Q.is_contiguous():
        raise ValueError("tensors must be contiguous CUDA tensors of shape [N, H, D]")
    return Q.shape[1], Q.shape[2]


def gattn_fwd(plan: Plan, Q, K, V, score: Score, out=None, lse=None, workspace=None,
              stream=None):
    """Forward: returns (out [N,H,D] in Q's dtype, lse fp32 [N,H])."""
    H, D = _shape(Q)
    for t in (K, V):
        if t.shape != Q.shape or t.dtype != Q.dtype or not t.is_contiguous():
            raise ValueError("Q, K, V must share shape, dtype and be contiguous")
    out = torch.empty_like(Q) if out is None else out
    lse = torch.empty(Q.shape[:2], dtype=torch.float32, device=Q.device) if lse is None else lse
    ws = plan.workspace(H, D, Q.dtype, Q.device) if workspace is None else workspace
    sc = score._struct()
    _check(load_library().gattn_fwd(plan.handle, H, D, _dtype_code(Q.dtype), _ptr(Q), _ptr(K),
                                    _ptr(V), ctypes.byref(sc), _ptr(out), _ptr(lse), _ptr(ws),
                                    ws.numel(), _stream(stream)), "gattn_fwd")
    return out, lse


def gattn_bwd(plan: Plan, Q, K, V, out, dout, lse, score: Score, dQ=None, dK=None, dV=None,
              da=None, workspace=None, stream=None):
    """Backward: returns (dQ, dK, dV, da) -- da is None for the dot score."""
    H, D = _shape(Q)
    dQ = torch.empty_like(Q) if dQ is None else dQ
    dK = torch.empty_like(Q) if dK is None else dK
    dV = torch.empty_like(Q) if dV is None else dV
    if score.kind == "gatv2" and da is None:
        da = torch.empty((H, D), dtype=torch.float32, device=Q.device)
    ws = plan.workspace(H, D, Q.dtype, Q.device) if workspace is None else workspace
    sc = score._struct()
    _check(load_library().gattn_bwd(plan.handle, H, D, _dtype_code(Q.dtype), _ptr(Q), _ptr(K),
                                    _ptr(V), ctypes.byref(sc), _ptr(out), _ptr(dout), _ptr(lse),
                                    _ptr(dQ), _ptr(dK), _ptr(dV),
                                    _ptr(da) if score.kind == "gatv2" else None, _ptr(ws),
                                    ws.numel(), _stream(stream)), "gattn_bwd")
    return dQ, dK, dV, (da if score.kind == "gatv2" else None)


def gattn_bwd_dq(plan: Plan, Q, K, V, out, dout, lse, score: Score, dQ=None, da=None,
                 workspace=None, stream=None):
    """CSR pass of the backward: returns (dQ, da); leaves Delta in the workspace."""
    H, D = _shape(Q)
    dQ = torch.empty_like(Q) if dQ is None else dQ
    if score.kind == "gatv2" and da is None:
        da = torch.empty((H, D), dtype=torch.float32, device=Q.device)
    ws = plan.workspace(H, D, Q.dtype, Q.device) if workspace is None else workspace
    sc = score._struct()
    _check(load_library().gattn_bwd_dq(plan.handle, H, D, _dtype_code(Q.dtype), _ptr(Q), _ptr(K),
                                       _ptr(V), ctypes.byref(sc), _ptr(out), _ptr(dout),
                                       _ptr(lse), _ptr(dQ),
                                       _ptr(da) if score.kind == "gatv2" else None, _ptr(ws),
                                       ws.numel(), _stream(stream)), "gattn_bwd_dq")
    return dQ, (da if score.kind == "gatv2" else None)


def gattn_bwd_dkdv(plan: Plan, Q, K, V, dout, lse, score: Score, dK=None, dV=None,
                   workspace=None, stream=None):
    """CSC pass of the backward (after gattn_bwd_dq on the same workspace): (dK, dV)."""
    H, D = _shape(Q)
    dK = torch.empty_like(Q) if dK is None else dK
    dV = torch.empty_like(Q) if dV is None else dV
    ws = plan.workspace(H, D, Q.dtype, Q.device) if workspace is None else workspace
    sc = score._struct()
    _check(load_library().gattn_bwd_dkdv(plan.handle, H, D, _dtype_code(Q.dtype), _ptr(Q),
                                         _ptr(K), _ptr(V), ctypes.byref(sc), _ptr(dout),
                                         _ptr(lse), _ptr(dK), _ptr(dV), _ptr(ws), ws.numel(),
                                         _stream(stream)), "gattn_bwd_dkdv")
    return dK, dV


def gattn_plan_check_errors(plan: Plan) -> None:
    """Raise GattnError(GATTN_ERR_TIMEOUT) if a kernel gave up a bounded wait."""
    _check(load_library().gattn_plan_check_errors(plan.handle), "gattn_plan_check_errors")


def gattn_plan_set_wait_test(plan: Plan, fail_first_wait: bool) -> None:
    """Test hook of the bounded-wait failure path: while set, every warp of the
    attention passes run with ``plan`` gives up its first wait at once (and
    still waits for the copies it issued), so the next
    gattn_plan_check_errors raises GATTN_ERR_TIMEOUT."""
    _check(load_library().gattn_plan_set_wait_test(plan.handle, int(bool(fail_first_wait))),
           "gattn_plan_set_wait_test")


def gattn_fwd_noalloc(plan: Plan, Q, K, V, score: Score, out, lse, stream=None):
    """Forward pass that allocates nothing: ``out`` and ``lse`` must be given,
    and the heavy-chunk scratch comes from the library's fixed 32 MiB array
    (for callers that cannot allocate device memory where they run the layer,
    e.g. under an allocator or memory pool they do not own)."""
    H, D = _shape(Q)
    sc = score._struct()
    _check(load_library().gattn_fwd_noalloc(plan.handle, H, D, _dtype_code(Q.dtype), _ptr(Q),
                                            _ptr(K), _ptr(V), ctypes.byref(sc), _ptr(out),
                                            _ptr(lse), _stream(stream)), "gattn_fwd_noalloc")
    return out, lse


# ----------------------------------------------------------------------------
# attention over selected blocks, and the gated residual norm
# ----------------------------------------------------------------------------
# These calls may take a few microseconds on the GPU (one new token), so their
# marshalling is lean: descriptors are packed bytes, pointers plain integers,
# and workspace sizes are kept by shape.
#
# `stream` (the current one by default) is where a call runs.  What the call
# allocates, workspaces too, comes from that stream's memory; as everywhere in
# torch, the caller has its tensors ready there, keeps them until the call is
# done, and waits for it before another stream reads the results.
_BLOCK_PACK = struct.Struct("@11ifi4xPPPqq")   # _BlockDesc
_NORM_PACK = struct.Struct("@qiiiiffPPPP")     # _NormDesc
assert _BLOCK_PACK.size == ctypes.sizeof(_BlockDesc)
assert _NORM_PACK.size == ctypes.sizeof(_NormDesc)
_sizes = {}


def _want(name, t, shape, dtype, dev):
    """Raise unless t is a contiguous tensor of this shape and dtype on device number dev."""
    if t.get_device() != dev or t.dtype != dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor, {dtype}, of shape "
                         f"{tuple(shape)}, on device {dev}")


def _cuda_index(name, t, dims):
    """Device number of the tensor that a call's other tensors have to match."""
    if not t.is_cuda or not t.is_contiguous() or t.dim() != dims:
        raise ValueError(f"{name} must be a contiguous CUDA tensor with {dims} dimensions, "
                         f"has the shape {tuple(t.shape)}")
    return t.get_device()


def _at(t):
    return None if t is None else t.data_ptr()


def _stream_of(dev, stream):
    """(handle, the stream where it is not the current one) of a call on device number dev."""
    handle = torch._C._cuda_getCurrentRawStream(dev)
    if stream is None:
        return handle, None
    if stream.device.index != dev:
        raise ValueError(f"stream of {stream.device} for tensors on device {dev}")
    return stream.cuda_stream, (stream if stream.cuda_stream != handle else None)


def _new(dev, other, shape, dtype):
    """A tensor that the call allocates and returns.

    With another stream it comes from that stream's memory: memory of the current one may still
    be in use there by work that was queued before.  The current stream, where the caller goes
    on with it, is recorded for its release.
    """
    if other is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(other):
        t = torch.empty(shape, dtype=dtype, device=dev)
    t.record_stream(torch.cuda.current_stream(dev))
    return t


def _like(t, other):
    return torch.empty_like(t) if other is None else _new(t.device, other, t.shape, t.dtype)


def _workspace(given, dev, other, fn, desc, key):
    """The caller's workspace, or a new one of the size that `fn` names (None for 0)."""
    if given is not None:
        if given.get_device() != dev or not given.is_contiguous():
            raise ValueError(f"workspace must be a contiguous tensor on device {dev}")
        return given
    n = _sizes.get((fn, dev, key))
    if n is None:
        size = ctypes.c_size_t()
        _check(getattr(load_library(), fn)(desc, ctypes.byref(size)), fn)
        n = size.value
        if len(_sizes) > 4096:
            _sizes.clear()
        _sizes[(fn, dev, key)] = n
    if not n:
        return None
    if other is None:
        return torch.empty(n, dtype=torch.uint8, device=dev)
    with torch.cuda.stream(other):  # used there alone
        return torch.empty(n, dtype=torch.uint8, device=dev)


def _bytes(t):
    return 0 if t is None else t.numel() * t.element_size()


def _sequences(seq_q, seq_k, len_k, dev):
    S = seq_k.numel() - 1
    if S < 0:
        raise ValueError("seq_q and seq_k need S + 1 entries and len_k S")
    for name, t, n in (("seq_q", seq_q, S + 1), ("seq_k", seq_k, S + 1), ("len_k", len_k, S)):
        if t is not None:
            _want(name, t, (n,), torch.int32, dev)
    return S


def gattn_block_units(Nq: int, S: int, q_block: int) -> int:
    """Rows of idx: table rows of the query units of S sequences with Nq rows together."""
    if q_block <= 0:
        raise ValueError("q_block must be positive")
    return (Nq // q_block + (S if q_block > 1 else 0)) if S else 0


def gattn_block_count(Nk: int, S: int, block: int) -> int:
    """Rows of sums: table rows of the key blocks of S sequences with Nk rows together."""
    if block <= 0:
        raise ValueError("block must be positive")
    return (Nk // block + S) if S else 0


def gattn_block_sums(K: torch.Tensor, seq_k: torch.Tensor, block: int, lens=None, since=None,
                     sums=None, stream=None) -> torch.Tensor:
    """fp64 sums [blocks, Hkv, D] of the keys of each block (include/gattn.h).

    ``since`` (int32 [S]) renews only the blocks with positions from there on
    and needs ``sums``, the table to renew.
    """
    dev = _cuda_index("K", K, 3)
    if dev != torch.cuda.current_device():
        with torch.cuda.device(dev):
            return gattn_block_sums(K, seq_k, block, lens, since, sums, stream)
    Nk, Hkv, D = K.shape
    S = _sequences(seq_k, seq_k, lens, dev)
    if since is not None:
        _want("since", since, (S,), torch.int32, dev)
        if sums is None:
            raise ValueError("since needs sums, the table to renew")
    shape = (gattn_block_count(Nk, S, block), Hkv, D)
    handle, other = _stream_of(dev, stream)
    if sums is None:
        sums = _new(dev, other, shape, torch.float64)
    else:
        _want("sums", sums, shape, torch.float64, dev)
    desc = _BLOCK_PACK.pack(S, 0, Nk, Hkv, Hkv, D, _dtype_code(K.dtype), block, 1, 1, 0, 0.0, 0,
                            seq_k.data_ptr(), seq_k.data_ptr(), _at(lens) or 0, 0, 0)
    _check((_lib or load_library()).gattn_block_sums(desc, K.data_ptr(), _at(since),
                                                     sums.data_ptr(), handle),
           "gattn_block_sums")
    return sums


def gattn_block_select(Q: torch.Tensor, sums: torch.Tensor, seq_q: torch.Tensor,
                       seq_k: torch.Tensor, topk: int, block: int, q_block: int, nk: int,
                       len_k=None, causal: bool = False, max_len_k: int = 0, idx=None,
                       workspace=None, stream=None) -> torch.Tensor:
    """The topk blocks of highest score of every unit and key head: int32 [units, Hkv, topk].

    ``nk`` is the number of key rows that ``sums`` was built from and
    ``max_len_k`` the most keys of one sequence (0: nk).
    """
    dev = _cuda_index("Q", Q, 3)
    if dev != torch.cuda.current_device():
        with torch.cuda.device(dev):
            return gattn_block_select(Q, sums, seq_q, seq_k, topk, block, q_block, nk, len_k,
                                      causal, max_len_k, idx, workspace, stream)
    Nq, H, D = Q.shape
    Hkv = sums.shape[1] if sums.dim() == 3 else 0
    S = _sequences(seq_q, seq_k, len_k, dev)
    _want("sums", sums, (gattn_block_count(nk, S, block), Hkv, D), torch.float64, dev)
    shape = (gattn_block_units(Nq, S, q_block), Hkv, topk)
    handle, other = _stream_of(dev, stream)
    if idx is None:
        idx = _new(dev, other, shape, torch.int32)
    else:
        _want("idx", idx, shape, torch.int32, dev)
    desc = _BLOCK_PACK.pack(S, Nq, nk, H, Hkv, D, _dtype_code(Q.dtype), block, q_block, topk,
                            1 if causal else 0, 0.0, max_len_k, seq_q.data_ptr(),
                            seq_k.data_ptr(), _at(len_k) or 0, 0, 0)
    ws = _workspace(workspace, dev, other, "gattn_block_select_workspace_size", desc,
                    (S, Nq, nk, H, Hkv, D, Q.dtype, block, q_block, topk))
    _check((_lib or load_library()).gattn_block_select(desc, Q.data_ptr(), sums.data_ptr(),
                                                       idx.data_ptr(), _at(ws), _bytes(ws), handle),
           "gattn_block_select")
    return idx


def _block_attn(Q, K, V, idx, seq_q, seq_k, block, q_block, scale, causal, len_k):
    """Checks of the forward and backward: (device, descriptor, key of their workspaces)."""
    dev = _cuda_index("Q", Q, 3)
    Nq, H, D = Q.shape
    if K.dim() != 3 or idx.dim() != 3:
        raise ValueError("need Q [Nq, H, D], K and V [Nk, Hkv, D] and idx [units, Hkv, topk]")
    Nk, Hkv, _ = K.shape
    _want("K", K, (Nk, Hkv, D), Q.dtype, dev)
    _want("V", V, (Nk, Hkv, D), Q.dtype, dev)
    S = _sequences(seq_q, seq_k, len_k, dev)
    units, topk = gattn_block_units(Nq, S, q_block), idx.shape[2]
    su, sh, sl = idx.stride()
    if (idx.get_device() != dev or idx.dtype != torch.int32 or idx.shape[0] != units
            or idx.shape[1] != Hkv or (topk > 1 and sl != 1)):
        raise ValueError(f"idx must be int32 of shape ({units}, {Hkv}, topk) on device {dev}, "
                         "each list contiguous")
    if su == 0 and sh == 0 and units * Hkv > 1:
        raise ValueError("idx repeats one list for all units and heads; make it contiguous")
    desc = _BLOCK_PACK.pack(S, Nq, Nk, H, Hkv, D, _dtype_code(Q.dtype), block, q_block, topk,
                            1 if causal else 0, scale, 0, seq_q.data_ptr(), seq_k.data_ptr(),
                            _at(len_k) or 0, su, sh)
    return dev, desc, (S, Nq, Nk, H, Hkv, D, Q.dtype, block, q_block, topk)


def gattn_block_fwd(Q, K, V, idx, seq_q, seq_k, block: int, q_block: int, scale: float = 0.0,
                    causal: bool = False, len_k=None, out=None, lse=None, workspace=None,
                    stream=None):
    """Softmax attention over the blocks that idx lists: (out [Nq, H, D], lse fp32 [Nq, H]).

    Rows of no sequence are not written; tensors that the call allocates hold
    anything there.
    """
    dev, desc, key = _block_attn(Q, K, V, idx, seq_q, seq_k, block, q_block, scale, causal, len_k)
    if dev != torch.cuda.current_device():
        with torch.cuda.device(dev):
            return gattn_block_fwd(Q, K, V, idx, seq_q, seq_k, block, q_block, scale, causal,
                                   len_k, out, lse, workspace, stream)
    handle, other = _stream_of(dev, stream)
    if out is None:
        out = _like(Q, other)
    else:
        _want("out", out, Q.shape, Q.dtype, dev)
    if lse is None:
        lse = _new(dev, other, Q.shape[:2], torch.float32)
    else:
        _want("lse", lse, Q.shape[:2], torch.float32, dev)
    ws = _workspace(workspace, dev, other, "gattn_block_fwd_workspace_size", desc, key)
    _check((_lib or load_library()).gattn_block_fwd(
        desc, Q.data_ptr(), K.data_ptr(), V.data_ptr(), idx.data_ptr(), out.data_ptr(),
        lse.data_ptr(), _at(ws), _bytes(ws), handle), "gattn_block_fwd")
    return out, lse


def gattn_block_bwd(Q, K, V, idx, seq_q, seq_k, out, dout, lse, block: int, q_block: int,
                    scale: float = 0.0, causal: bool = False, len_k=None, dQ=None, dK=None,
                    dV=None, workspace=None, stream=None):
    """Gradients (dQ, dK, dV) of gattn_block_fwd; rows of no sequence are not written."""
    dev, desc, key = _block_attn(Q, K, V, idx, seq_q, seq_k, block, q_block, scale, causal, len_k)
    if dev != torch.cuda.current_device():
        with torch.cuda.device(dev):
            return gattn_block_bwd(Q, K, V, idx, seq_q, seq_k, out, dout, lse, block, q_block,
                                   scale, causal, len_k, dQ, dK, dV, workspace, stream)
    _want("out", out, Q.shape, Q.dtype, dev)
    _want("dout", dout, Q.shape, Q.dtype, dev)
    _want("lse", lse, Q.shape[:2], torch.float32, dev)
    handle, other = _stream_of(dev, stream)
    grads = []
    for name, t, like in (("dQ", dQ, Q), ("dK", dK, K), ("dV", dV, K)):
        if t is None:
            t = _like(like, other)
        else:
            _want(name, t, like.shape, like.dtype, dev)
        grads.append(t)
    ws = _workspace(workspace, dev, other, "gattn_block_bwd_workspace_size", desc, key)
    _check((_lib or load_library()).gattn_block_bwd(
        desc, Q.data_ptr(), K.data_ptr(), V.data_ptr(), idx.data_ptr(), out.data_ptr(),
        dout.data_ptr(), lse.data_ptr(), grads[0].data_ptr(), grads[1].data_ptr(),
        grads[2].data_ptr(), _at(ws), _bytes(ws), handle), "gattn_block_bwd")
    return tuple(grads)


def gattn_block_check_errors() -> None:
    """Raise GattnError(GATTN_ERR_TIMEOUT) if a block-attention kernel gave up a bounded wait."""
    _check(load_library().gattn_block_check_errors(), "gattn_block_check_errors")


def gattn_block_set_wait_test(fail_first_wait: bool) -> None:
    """Test hook of the bounded-wait failure path: while set, block-attention kernels (bf16) give
    up at once, so the next gattn_block_check_errors raises GATTN_ERR_TIMEOUT."""
    _check(load_library().gattn_block_set_wait_test(int(bool(fail_first_wait))),
           "gattn_block_set_wait_test")


NORM = {"rms": 0, "layer": 1}


def _norm_desc(res, gate, w_post, b_post, w_pre, b_pre, alpha, kind, eps):
    """Checks of the norm's forward and backward: (device, descriptor, N, F)."""
    dev = _cuda_index("res", res, 2)
    if kind not in NORM:
        raise ValueError(f"unknown norm kind {kind!r}")
    N, F = res.shape
    mode = 0
    if gate is not None:
        mode = 1 if gate.dim() == 1 else 2
        _want("gate", gate, (F,) if mode == 1 else (N, F),
              torch.float32 if mode == 1 else res.dtype, dev)
    for name, t in (("w_post", w_post), ("b_post", b_post), ("w_pre", w_pre), ("b_pre", b_pre)):
        if t is not None:
            _want(name, t, (F,), torch.float32, dev)
    desc = _NORM_PACK.pack(N, F, _dtype_code(res.dtype), NORM[kind], mode, alpha, eps,
                           _at(w_post) or 0, _at(b_post) or 0, _at(w_pre) or 0, _at(b_pre) or 0)
    return dev, desc, N, F


def gattn_norm_fwd(res, x=None, gate=None, w_post=None, b_post=None, w_pre=None, b_pre=None,
                   alpha: float = 1.0, kind: str = "rms", eps: float = 1e-6, h=None, y=None,
                   stats=None, stream=None):
    """h = res + alpha * gate * norm(x; w_post, b_post), y = norm(h; w_pre, b_pre).

    res, x: [N, F]; gate: [N, F] in their dtype, or fp32 [F], or None for 1;
    weights and biases fp32 [F].  Without w_post the first norm is left out,
    without w_pre the second (y is None), without x h is res itself.  Returns
    (h, y, stats); stats (fp32 [N, 4]) goes to gattn_norm_bwd.
    """
    dev, desc, N, F = _norm_desc(res, gate, w_post, b_post, w_pre, b_pre, alpha, kind, eps)
    if dev != torch.cuda.current_device():
        with torch.cuda.device(dev):
            return gattn_norm_fwd(res, x, gate, w_post, b_post, w_pre, b_pre, alpha, kind, eps,
                                  h, y, stats, stream)
    handle, other = _stream_of(dev, stream)
    shape, dtype = res.shape, res.dtype
    if x is None:
        h = res
    else:
        _want("x", x, shape, dtype, dev)
        if h is None:
            h = _like(res, other)
        else:
            _want("h", h, shape, dtype, dev)
    if w_pre is None:
        y = None
    elif y is None:
        y = _like(res, other)
    else:
        _want("y", y, shape, dtype, dev)
    if stats is None:
        stats = _new(dev, other, (N, 4), torch.float32)
    else:
        _want("stats", stats, (N, 4), torch.float32, dev)
    _check((_lib or load_library()).gattn_norm_fwd(
        desc, res.data_ptr(), _at(x), _at(gate), None if x is None else h.data_ptr(), _at(y),
        stats.data_ptr(), handle), "gattn_norm_fwd")
    return h, y, stats


def gattn_norm_bwd(res, stats, dh=None, dy=None, x=None, gate=None, w_post=None, b_post=None,
                   w_pre=None, b_pre=None, alpha: float = 1.0, kind: str = "rms",
                   workspace=None, stream=None) -> dict:
    """Gradients of gattn_norm_fwd from dh (of h, or None) and dy (of y), at the forward's
    res, x, gate and stats.

    Returns a dict of dres, dx, dgate, dw_post, db_post, dw_pre, db_pre; None
    where the operand is absent.
    """
    dev, desc, N, F = _norm_desc(res, gate, w_post, b_post, w_pre, b_pre, alpha, kind, 0.0)
    if dev != torch.cuda.current_device():
        with torch.cuda.device(dev):
            return gattn_norm_bwd(res, stats, dh, dy, x, gate, w_post, b_post, w_pre, b_pre,
                                  alpha, kind, workspace, stream)
    for name, t in (("dh", dh), ("dy", dy), ("x", x)):
        if t is not None:
            _want(name, t, (N, F), res.dtype, dev)
    _want("stats", stats, (N, 4), torch.float32, dev)
    handle, other = _stream_of(dev, stream)
    g = {"dres": _like(res, other), "dx": None if x is None else _like(x, other),
         "dgate": None if gate is None else _like(gate, other)}
    for n, t in (("dw_post", w_post), ("db_post", b_post), ("dw_pre", w_pre), ("db_pre", b_pre)):
        g[n] = None if t is None else _like(t, other)
    ws = _workspace(workspace, dev, other, "gattn_norm_workspace_size", desc, (N, F, res.dtype))
    _check((_lib or load_library()).gattn_norm_bwd(
        desc, res.data_ptr(), stats.data_ptr(), _at(dh), _at(dy), _at(x), _at(gate),
        *[_at(t) for t in g.values()], _at(ws), _bytes(ws), handle), "gattn_norm_bwd")
    return g


# ----------------------------------------------------------------------------
# rotary positions, and a cache of keys and values in 4 or 8 bits
# ----------------------------------------------------------------------------
_ROTARY_PACK = struct.Struct("@9if5P4q")            # _RotaryDesc
_CACHE_PACK = struct.Struct("@11ifi4x3P4q3P")       # _CacheDesc
assert _ROTARY_PACK.size == ctypes.sizeof(_RotaryDesc)
assert _CACHE_PACK.size == ctypes.sizeof(_CacheDesc)
ROTARY_LAYOUT = {"half": 0, "interleaved": 1}
ROTARY_SCALING = {"none": 0, "linear": 1, "base": 2, "ramp": 3}
_CODES = {torch.float32: GATTN_F32, torch.bfloat16: GATTN_BF16}
_INT32, _F32, _empty, _empty_like = torch.int32, torch.float32, torch.empty, torch.empty_like
_device = torch._C._cuda_getDevice              # of tensors that are on a GPU already
_raw_stream = torch._C._cuda_getCurrentRawStream


def _offsets(name, t, n, dev):
    """_want for the int32 vectors of a call, without a call's way to its message."""
    if (t.get_device() != dev or t.dtype is not _INT32 or t.numel() != n or t.dim() != 1
            or not t.is_contiguous()):
        _want(name, t, (n,), _INT32, dev)


def _seq_args(seq_q, seq_k, len_k, dev):
    """Checked offsets and lengths (each but one may be None): S."""
    S = (seq_q if seq_k is None else seq_k).numel() - 1
    if S < 0:
        raise ValueError("seq_q and seq_k need S + 1 entries and len_k S")
    if seq_q is not None:
        _offsets("seq_q", seq_q, S + 1, dev)
    if seq_k is not None:
        _offsets("seq_k", seq_k, S + 1, dev)
    if len_k is not None:
        _offsets("len_k", len_k, S, dev)
    return S


def _row_stride(name, t, H, D, dtype, dev):
    """Elements between the rows of t [N, H, D], whose heads lie side by side (as in a slice of
    a joint projection)."""
    if (t.get_device() != dev or t.dtype is not dtype or t.dim() != 3 or t.size(1) != H
            or t.size(2) != D):
        raise ValueError(f"{name} must be a CUDA tensor, {dtype}, of shape (N, {H}, {D}), on "
                         f"device {dev}")
    if t.is_contiguous():
        return H * D
    sn, sh, sd = t.stride()
    if (D > 1 and sd != 1) or (H > 1 and sh != D):
        raise ValueError(f"{name}: the heads of a row must be contiguous")
    if t.shape[0] <= 1:
        return H * D
    if sn < H * D:
        raise ValueError(f"{name}: rows must not overlap")
    return sn


def gattn_rotary_freqs(width: int, theta: float = 10000.0, scaling: str = "none",
                       factor: float = 1.0, orig_len: float = 0.0, low: float = 1.0,
                       high: float = 32.0, device="cuda") -> torch.Tensor:
    """Frequencies of the width / 2 pairs of a head for gattn_rotary, int64 [width / 2]: turns
    per position in units of 2^-64 (include/gattn.h).  ``scaling``: "none", or for contexts
    longer than those of training "linear", "base" or "ramp" (with ``orig_len``)."""
    if scaling not in ROTARY_SCALING:
        raise ValueError(f"scaling must be one of {tuple(ROTARY_SCALING)}, got {scaling!r}")
    out = (ctypes.c_uint64 * max(width // 2, 1))()
    _check(load_library().gattn_rotary_freqs(width, theta, ROTARY_SCALING[scaling], factor,
                                             orig_len, low, high, ctypes.addressof(out)),
           "gattn_rotary_freqs")
    return torch.from_numpy(np.frombuffer(out, dtype=np.int64).copy()).to(device)


def gattn_rotary(Q: torch.Tensor, freqs: torch.Tensor, K=None, layout: str = "half", pos=None,
                 seq_q=None, seq_k=None, len_k=None, amp: float = 1.0, inverse: bool = False,
                 out_q=None, out_k=None, stream=None):
    """Q [N, H, D] and K [N, Hkv, D] (or None) with the first 2 * len(freqs) elements of every
    head turned by the rows' positions: (Q', K').

    Positions are ``pos`` (int32 [N]), or those of the rows of sequences as the block and cache
    attention counts them (``seq_q``, and the keys' ``seq_k`` and ``len_k`` where sequences hold
    more than the new rows).  Rows of Q and K may lie apart, as slices of a joint projection do;
    ``out_q`` and ``out_k`` may be Q and K themselves.  ``inverse`` turns back, as a backward does.
    Rows of no sequence are not written.
    """
    dev = Q.get_device()
    if dev < 0 or Q.dim() != 3:
        raise ValueError(f"Q must be a CUDA tensor [N, H, D], has the shape {tuple(Q.shape)}")
    if dev != _device():
        with torch.cuda.device(dev):
            return gattn_rotary(Q, freqs, K, layout, pos, seq_q, seq_k, len_k, amp, inverse, out_q,
                                out_k, stream)
    N, H, D = Q.shape
    dt = Q.dtype
    order = ROTARY_LAYOUT.get(layout)
    if order is None:
        raise ValueError(f"layout must be one of {tuple(ROTARY_LAYOUT)}, got {layout!r}")
    pairs = freqs.numel()
    if freqs.get_device() != dev or freqs.dtype is not torch.int64 or not freqs.is_contiguous():
        _want("freqs", freqs, (pairs,), torch.int64, dev)
    qs = qos = H * D
    if not Q.is_contiguous():
        qs = _row_stride("Q", Q, H, D, dt, dev)
    Hkv = ks = kos = 0
    if K is not None:
        if K.dim() != 3 or K.size(0) != N:
            raise ValueError(f"K must have the {N} rows of Q, has the shape {tuple(K.shape)}")
        Hkv = K.size(1)
        kos = Hkv * D
        ks = _row_stride("K", K, Hkv, D, dt, dev)
    elif out_k is not None:
        raise ValueError("out_k needs K")
    S = p_pos = p_sq = p_sk = p_len = 0
    if pos is not None:
        if seq_q is not None or seq_k is not None or len_k is not None:
            raise ValueError("give pos or sequences, not both")
        _offsets("pos", pos, N, dev)
        p_pos = pos.data_ptr()
    else:
        if seq_q is None:
            raise ValueError("positions need pos or seq_q")
        S = _seq_args(seq_q, seq_k, len_k, dev)
        p_sq = seq_q.data_ptr()
        if seq_k is not None:
            p_sk = seq_k.data_ptr()
        if len_k is not None:
            p_len = len_k.data_ptr()
    other = None
    if stream is None:
        handle = _raw_stream(dev)
    else:
        handle, other = _stream_of(dev, stream)
    if out_q is None:
        if other is not None:
            out_q = _new(dev, other, Q.shape, dt)
        else:
            out_q = _empty_like(Q) if qs == qos else _empty((N, H, D), dtype=dt, device=dev)
    else:
        if out_q.shape != Q.shape:
            raise ValueError(f"out_q must have the shape {tuple(Q.shape)}")
        qos = _row_stride("out_q", out_q, H, D, dt, dev)
    if K is None:
        p_k = p_ko = None
    else:
        if out_k is None:
            if other is not None:
                out_k = _new(dev, other, K.shape, dt)
            else:
                out_k = _empty_like(K) if ks == kos else _empty((N, Hkv, D), dtype=dt, device=dev)
        else:
            if out_k.shape != K.shape:
                raise ValueError(f"out_k must have the shape {tuple(K.shape)}")
            kos = _row_stride("out_k", out_k, Hkv, D, dt, dev)
        p_k, p_ko = K.data_ptr(), out_k.data_ptr()
    code = _CODES.get(dt)
    desc = _ROTARY_PACK.pack(N, H, Hkv, D, _dtype_code(dt) if code is None else code, 2 * pairs,
                             order, 1 if inverse else 0, S, amp, freqs.data_ptr(), p_pos, p_sq,
                             p_sk, p_len, qs, ks, qos, kos)
    status = (_lib or load_library()).gattn_rotary(desc, Q.data_ptr(), p_k, out_q.data_ptr(), p_ko,
                                                   handle)
    if status:
        _check(status, "gattn_rotary")
    return out_q, out_k


class Cache:
    """Keys and values in 4 or 8 bits (include/gattn.h): ``k`` and ``v`` uint8
    [Hkv, rows, D * bits / 8], ``par`` bf16 [Hkv, rows, 4]."""

    __slots__ = ("k", "v", "par", "bits", "rows", "Hkv", "D", "device")

    def __init__(self, k: torch.Tensor, v: torch.Tensor, par: torch.Tensor, bits: int):
        if bits not in (4, 8):
            raise ValueError(f"bits must be 4 or 8, got {bits}")
        dev = _cuda_index("k", k, 3)
        self.Hkv, self.rows, row = k.shape
        _want("k", k, k.shape, torch.uint8, dev)
        _want("v", v, k.shape, torch.uint8, dev)
        _want("par", par, (self.Hkv, self.rows, 4), torch.bfloat16, dev)
        self.D = row * 8 // bits
        self.k, self.v, self.par, self.bits, self.device = k, v, par, bits, dev


def gattn_cache_new(rows: int, Hkv: int, D: int, bits: int = 4, device="cuda") -> Cache:
    """An empty cache with room for ``rows`` rows of all sequences together."""
    if D not in (32, 64, 128):
        raise ValueError(f"D must be 32, 64 or 128, got {D}")
    if bits not in (4, 8):
        raise ValueError(f"bits must be 4 or 8, got {bits}")
    k, v = (torch.zeros(Hkv, rows, D * bits // 8, dtype=torch.uint8, device=device)
            for _ in range(2))
    return Cache(k, v, torch.zeros(Hkv, rows, 4, dtype=torch.bfloat16, device=device), bits)


def _cache_desc(c, S, N, H, dtype, block, topk, causal, scale, max_len_k, seq_q, seq_k, len_k,
                su=0, sh=0, ks=0, vs=0):
    code = _CODES.get(dtype)
    return _CACHE_PACK.pack(S, N, c.rows, H, c.Hkv, c.D, _dtype_code(dtype) if code is None else code,
                            c.bits, block, topk, 1 if causal else 0, scale, max_len_k,
                            0 if seq_q is None else seq_q.data_ptr(), seq_k.data_ptr(),
                            0 if len_k is None else len_k.data_ptr(), su, sh, ks, vs,
                            c.k.data_ptr(), c.v.data_ptr(), c.par.data_ptr())


def gattn_cache_write(cache: Cache, K: torch.Tensor, V: torch.Tensor, seq_q: torch.Tensor,
                      seq_k: torch.Tensor, len_k=None, stream=None) -> None:
    """Append the rows of K and V [N, Hkv, D] to their sequences: ``len_k`` counts them already.

    Rows of K and V may lie apart (16-byte aligned), as slices of a joint projection do.
    """
    dev = cache.device
    if dev != _device():
        with torch.cuda.device(dev):
            return gattn_cache_write(cache, K, V, seq_q, seq_k, len_k, stream)
    ks = _row_stride("K", K, cache.Hkv, cache.D, K.dtype, dev)
    vs = _row_stride("V", V, cache.Hkv, cache.D, K.dtype, dev)
    if V.shape[0] != K.shape[0]:
        raise ValueError("K and V must have the same rows")
    S = _seq_args(seq_q, seq_k, len_k, dev)
    handle = _raw_stream(dev) if stream is None else _stream_of(dev, stream)[0]
    desc = _cache_desc(cache, S, K.shape[0], cache.Hkv, K.dtype, 64, 0, False, 0.0, 0, seq_q, seq_k,
                       len_k, 0, 0, ks, vs)
    status = (_lib or load_library()).gattn_cache_write(desc, K.data_ptr(), V.data_ptr(), handle)
    if status:
        _check(status, "gattn_cache_write")


def gattn_cache_read(cache: Cache, seq_q: torch.Tensor, seq_k: torch.Tensor, len_k=None, since=None,
                     rows=None, dtype=torch.bfloat16, K=None, V=None, stream=None):
    """Rows of the cache in ``dtype``: (K, V), each [rows, Hkv, D].

    Row i of sequence s's [seq_q[s], seq_q[s+1]) is the one at position i + len_k[s] - lq (the
    rows that gattn_cache_write appended), or i + since[s].  Rows without such a position are
    not written; tensors that the call allocates hold anything there.  ``rows`` is needed where
    neither K nor V is given.
    """
    dev = cache.device
    if dev != _device():
        with torch.cuda.device(dev):
            return gattn_cache_read(cache, seq_q, seq_k, len_k, since, rows, dtype, K, V, stream)
    S = _seq_args(seq_q, seq_k, len_k, dev)
    if since is not None:
        _offsets("since", since, S, dev)
    given = K if K is not None else V
    if given is not None:
        rows, dtype = given.shape[0], given.dtype
    elif rows is None:
        raise ValueError("rows is needed where neither K nor V is given")
    shape = (rows, cache.Hkv, cache.D)
    handle, other = (_raw_stream(dev), None) if stream is None else _stream_of(dev, stream)
    if given is None:
        if other is None:
            K = _empty(shape, dtype=dtype, device=dev)
            V = _empty_like(K)
        else:
            K, V = _new(dev, other, shape, dtype), _new(dev, other, shape, dtype)
    else:
        for name, t in (("K", K), ("V", V)):
            if t is not None:
                _want(name, t, shape, dtype, dev)
    desc = _cache_desc(cache, S, rows, cache.Hkv, dtype, 64, 0, False, 0.0, 0, seq_q, seq_k, len_k)
    status = (_lib or load_library()).gattn_cache_read(desc, _at(since), _at(K), _at(V), handle)
    if status:
        _check(status, "gattn_cache_read")
    return K, V


def gattn_cache_sums(cache: Cache, seq_k: torch.Tensor, block: int, lens=None, since=None, sums=None,
                     stream=None) -> torch.Tensor:
    """gattn_block_sums of the cached keys: fp64 sums [blocks, Hkv, D] of what they stand for."""
    dev = cache.device
    if dev != _device():
        with torch.cuda.device(dev):
            return gattn_cache_sums(cache, seq_k, block, lens, since, sums, stream)
    S = _seq_args(None, seq_k, lens, dev)
    if since is not None:
        _offsets("since", since, S, dev)
        if sums is None:
            raise ValueError("since needs sums, the table to renew")
    shape = (gattn_block_count(cache.rows, S, block), cache.Hkv, cache.D)
    handle, other = (_raw_stream(dev), None) if stream is None else _stream_of(dev, stream)
    if sums is None:
        sums = _new(dev, other, shape, torch.float64)
    else:
        _want("sums", sums, shape, torch.float64, dev)
    desc = _cache_desc(cache, S, 0, cache.Hkv, torch.float32, block, 0, False, 0.0, 0, None, seq_k,
                       lens)
    status = (_lib or load_library()).gattn_cache_sums(desc, _at(since), sums.data_ptr(), handle)
    if status:
        _check(status, "gattn_cache_sums")
    return sums


def gattn_cache_fwd(Q: torch.Tensor, cache: Cache, seq_q: torch.Tensor, seq_k: torch.Tensor,
                    len_k=None, idx=None, block: int = 64, scale: float = 0.0,
                    causal: bool = False, max_len_k: int = 0, out=None, lse=None, workspace=None,
                    stream=None):
    """Softmax attention of every row of Q [N, H, D] over the cache: (out, lse fp32 [N, H]).

    ``idx`` (int32 [N, Hkv, topk]) names blocks of each row's own sequence, as for
    gattn_block_fwd with q_block = 1; without it the whole sequence is read.  ``max_len_k`` is the
    most rows of one sequence (0: all rows of the cache): a close bound lets short caches be
    split well.  Rows of no sequence are not written.
    """
    dev = _cuda_index("Q", Q, 3)
    if dev != _device():
        with torch.cuda.device(dev):
            return gattn_cache_fwd(Q, cache, seq_q, seq_k, len_k, idx, block, scale, causal,
                                   max_len_k, out, lse, workspace, stream)
    N, H, D = Q.shape
    if cache.device != dev or cache.D != D:
        raise ValueError(f"Q [N, H, {D}] on device {dev} needs a cache of that width there")
    S = _seq_args(seq_q, seq_k, len_k, dev)
    topk = su = sh = 0
    if idx is not None:
        if idx.dim() != 3:
            raise ValueError("idx must be [N, Hkv, topk]")
        units, topk = N if S else 0, idx.shape[2]
        su, sh, sl = idx.stride()
        if (idx.get_device() != dev or idx.dtype != torch.int32 or idx.shape[0] != units
                or idx.shape[1] != cache.Hkv or topk < 1 or (topk > 1 and sl != 1)):
            raise ValueError(f"idx must be int32 of shape ({units}, {cache.Hkv}, topk) on device "
                             f"{dev}, each list contiguous")
        if su == 0 and sh == 0 and units * cache.Hkv > 1:
            raise ValueError("idx repeats one list for all rows and heads; make it contiguous")
    handle, other = (_raw_stream(dev), None) if stream is None else _stream_of(dev, stream)
    if out is None:
        out = _empty_like(Q) if other is None else _new(dev, other, Q.shape, Q.dtype)
    else:
        _want("out", out, Q.shape, Q.dtype, dev)
    if lse is None:
        lse = _empty((N, H), dtype=_F32, device=dev) if other is None else \
            _new(dev, other, (N, H), _F32)
    else:
        _want("lse", lse, (N, H), _F32, dev)
    desc = _cache_desc(cache, S, N, H, Q.dtype, block, topk, causal, scale, max_len_k, seq_q, seq_k,
                       len_k, su, sh)
    ws = _workspace(workspace, dev, other, "gattn_cache_fwd_workspace_size", desc,
                    (S > 0, N, cache.rows, H, cache.Hkv, D, cache.bits, Q.dtype, block, topk,
                     max_len_k))
    status = (_lib or load_library()).gattn_cache_fwd(desc, Q.data_ptr(), _at(idx), out.data_ptr(),
                                                      lse.data_ptr(), _at(ws), _bytes(ws), handle)
    if status:
        _check(status, "gattn_cache_fwd")
    return out, lse
