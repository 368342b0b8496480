"""GB300 (sm_103a) sparse x dense matrix multiply: C = A_sparse @ B_dense.

Thin Python binding over the C ABI of ``libspmm_gb300.so`` (declared in
``include/spmm_gb300.h``).  Every step of the computation runs in the CUDA
library; this module only allocates outputs with torch and passes pointers,
sizes and the current CUDA stream.  There is no CPU fallback: a missing
library raises.

Format containers hold device tensors:
  BCSR(M, K, bh, bw, nnzb, dtype, row_ptr, col_idx, vals)
  Mat24(M, K, dtype, vals, meta)
  Slide(M, K, n, dtype, vals, meta)   ((2n-2):2n lifted into 2:4 windows)
  TVW(M, K, tile_rows, dtype, n_tiles, Kp, tile_ptr, cols, vals, meta)
  CSR(M, K, nnz, dtype, row_ptr, col, val)
  WCSR(...)  (see include/spmm_gb300.h for the field meanings)
  Route(T, k, n_keys, order, pos, offsets)   (one-hot rows sorted by key)
  Rows8(rows, cols, dtype, q, scale)   (rows held in 8 bits)

Beyond C = A B for those formats: spmm_slide ((2n-2):2n as overlapping 2:4
windows), spmm_bcsr_permuted (BCSR after a Reverse Cuthill-McKee order from
rcm_order), spmm_sddmm (A B sampled at a CSR pattern) and the pruning
builders spmm_prune_24 / spmm_prune_tvw.  One-hot operators (tokens by expert or
by vocabulary row): spmm_build_route, spmm_dispatch, spmm_combine and their
gradients, spmm_embed and spmm_embed_grad, and the experts' products
spmm_experts / spmm_experts_dx / spmm_experts_dw between them.  Around those, for
a gated mixture of experts: the router spmm_topk, the gated feed-forward block
spmm_experts_gated, activation checkpoints in 8 bits (spmm_pack_rows,
spmm_unpack_rows, save="packed"), and the gradients spmm_topk_grad,
spmm_gated_grad and spmm_experts_gated_grad.

Calls are not recorded by autograd: a result has no history even where an operand
requires grad.  A backward pass calls the gradient operators itself, by hand
(examples/moe_layer.py) or in a torch.autograd.Function of the caller's.  Results
must not overlap operands, and operands live on the current device.
"""
from __future__ import annotations

import ctypes as C
from dataclasses import dataclass, field
from typing import Optional

import torch

from . import _lib
from ._lib import SpmmError

__all__ = ["BCSR", "Mat24", "Slide", "TVW", "CSR", "WCSR", "SpmmError", "spmm_bcsr", "spmm_build_bcsr_count",
           "spmm_build_bcsr_fill", "build_bcsr", "spmm_compress_24", "spmm_prune_24", "spmm_widen_24", "spmm_24", "spmm_24_workspace_size",
           "spmm_build_tvw", "spmm_prune_tvw", "spmm_tvw", "spmm_build_wcsr_workspace_size", "spmm_build_wcsr_count",
           "spmm_build_wcsr_fill", "build_wcsr", "spmm_wcsr", "spmm_wcsr_workspace_size",
           "spmm_build_slide", "spmm_slide", "spmm_slide_workspace_size",
           "spmm_sddmm", "rcm_order", "spmm_permute_sym", "spmm_permute_rows", "spmm_bcsr_permuted", "spmm_bcsr_permuted_workspace_size",
           "Route", "spmm_build_route", "spmm_build_route_workspace_size", "spmm_dispatch", "spmm_dispatch_grad",
           "spmm_combine", "spmm_combine_grad", "spmm_embed", "spmm_embed_grad", "spmm_embed_grad_workspace_size",
           "spmm_experts", "spmm_experts_dx", "spmm_experts_dw", "spmm_experts_grad",
           "Rows8", "spmm_topk", "spmm_topk_grad", "spmm_pack_rows", "spmm_unpack_rows",
           "spmm_experts_gated", "spmm_gated_grad", "spmm_experts_gated_grad", "spmm_experts_gated_grad_workspace_size",
           "last_device_error", "selftest_timeout", "library_path", "trace_enable", "trace_read"]

_DT = {torch.bfloat16: _lib.SPMM_BF16, torch.float16: _lib.SPMM_F16, torch.int8: _lib.SPMM_I8,
       torch.float8_e4m3fn: _lib.SPMM_E4M3, torch.float8_e5m2: _lib.SPMM_E5M2}


def library_path() -> str:
    return _lib.LIB_PATH


def _code(dtype) -> int:
    if dtype not in _DT:
        raise TypeError(f"unsupported dtype {dtype}")
    return _DT[dtype]


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None or t.numel() == 0 else C.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return C.c_void_p(s.cuda_stream)


def _check_dev(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("all operands must be CUDA tensors (this library has no CPU path)")


# ------------------------------------------------------------------ formats
@dataclass
class BCSR:
    M: int
    K: int
    bh: int
    bw: int
    nnzb: int
    dtype: torch.dtype
    row_ptr: torch.Tensor
    col_idx: torch.Tensor
    vals: torch.Tensor

    def c(self) -> _lib.BcsrT:
        return _lib.BcsrT(self.M, self.K, self.bh, self.bw, self.nnzb, _code(self.dtype), _ptr(self.row_ptr),
                          _ptr(self.col_idx), _ptr(self.vals))


@dataclass
class Mat24:
    M: int
    K: int
    dtype: torch.dtype
    vals: torch.Tensor
    meta: torch.Tensor
    vals16: Optional[torch.Tensor] = None  # int8: vals widened to fp16 once (spmm_widen_24)

    def c(self) -> _lib.T24:
        return _lib.T24(self.M, self.K, _code(self.dtype), _ptr(self.vals), _ptr(self.meta), _ptr(self.vals16))


@dataclass
class Slide:
    """(2n-2):2n operand lifted into n - 1 overlapping 2:4 windows per group of 2n
    (window planes); K is the original depth, vals/meta span K' = 2 K (n-1) / n."""
    M: int
    K: int
    n: int
    dtype: torch.dtype
    vals: torch.Tensor
    meta: torch.Tensor

    @property
    def K_lifted(self) -> int:
        return 4 * (self.n - 1) * (self.K // (2 * self.n))

    def c(self) -> _lib.SlideT:
        return _lib.SlideT(self.M, self.K, self.n, _code(self.dtype), _ptr(self.vals), _ptr(self.meta))


@dataclass
class TVW:
    M: int
    K: int
    tile_rows: int
    dtype: torch.dtype
    n_tiles: int
    Kp: int
    tile_ptr: torch.Tensor
    cols: torch.Tensor
    vals: torch.Tensor
    meta: torch.Tensor

    def c(self) -> _lib.TvwT:
        return _lib.TvwT(self.M, self.K, self.tile_rows, _code(self.dtype), self.n_tiles, self.Kp,
                         _ptr(self.tile_ptr), _ptr(self.cols), _ptr(self.vals), _ptr(self.meta))


@dataclass
class CSR:
    M: int
    K: int
    nnz: int
    dtype: torch.dtype
    row_ptr: torch.Tensor
    col: torch.Tensor
    val: torch.Tensor

    def c(self) -> _lib.CsrT:
        return _lib.CsrT(self.M, self.K, self.nnz, _code(self.dtype), _ptr(self.row_ptr), _ptr(self.col),
                         _ptr(self.val))


@dataclass
class WCSR:
    M: int
    K: int
    nnz: int
    h: int
    S: int
    dtype: torch.dtype
    n_windows: int
    n_wcols: int
    n_units: int
    wcol_ptr: torch.Tensor
    wcols: torch.Tensor
    wnz_ptr: torch.Tensor
    unit_ptr: torch.Tensor
    unit_win: torch.Tensor
    unit_nz_ptr: torch.Tensor
    lrow: torch.Tensor
    slot: torch.Tensor
    val: torch.Tensor
    workspace: Optional[torch.Tensor] = field(default=None, repr=False)

    def c(self) -> _lib.WcsrT:
        return _lib.WcsrT(self.M, self.K, self.nnz, self.h, self.S, _code(self.dtype), self.n_windows,
                          self.n_wcols, self.n_units, _ptr(self.wcol_ptr), _ptr(self.wcols), _ptr(self.wnz_ptr),
                          _ptr(self.unit_ptr), _ptr(self.unit_win), _ptr(self.unit_nz_ptr), _ptr(self.lrow),
                          _ptr(self.slot), _ptr(self.val))


# ------------------------------------------------------------------ utilities
def last_device_error() -> int:
    """Read and clear the sticky device error word (SPMM_DEVERR_* bits)."""
    v = C.c_int32(0)
    _lib.call("spmm_last_device_error", C.byref(v))
    return v.value


def selftest_timeout(timeout_ns: int = 1_000_000, stream=None) -> None:
    _lib.call("spmm_selftest_timeout", C.c_uint64(timeout_ns), _stream(stream))


def trace_enable(on: bool = True) -> None:
    """Record CUDA events around every library kernel launch (see spmm_trace_read)."""
    _lib.call("spmm_trace_enable", 1 if on else 0)


def trace_read(kernel: int):
    """(launches, total_ms) of one kernel kind since tracing was enabled."""
    n, ms = C.c_int64(0), C.c_double(0.0)
    _lib.call("spmm_trace_read", kernel, C.byref(n), C.byref(ms))
    return n.value, ms.value


def _out(C_, M, N, dtype, device):
    if C_ is None:
        return torch.empty((M, N), dtype=dtype, device=device)
    return C_


# ------------------------------------------------------------------ BCSR
def spmm_build_bcsr_count(dense: torch.Tensor, bh: int, bw: int, stream=None):
    _check_dev(dense)
    M, K = dense.shape
    row_ptr = torch.empty(M // bh + 1 if bh > 0 else 1, dtype=torch.int32, device=dense.device)
    n = C.c_int64(0)
    _lib.call("spmm_build_bcsr_count", _ptr(dense), M, K, dense.stride(0), bh, bw, _code(dense.dtype),
              _ptr(row_ptr), C.byref(n), _stream(stream))
    return row_ptr, n.value


def spmm_build_bcsr_fill(dense: torch.Tensor, bh: int, bw: int, row_ptr: torch.Tensor, nnzb: int,
                         stream=None) -> BCSR:
    _check_dev(dense, row_ptr)
    M, K = dense.shape
    col_idx = torch.empty(max(nnzb, 1), dtype=torch.int32, device=dense.device)[:nnzb]
    vals = torch.empty((max(nnzb, 1), bh, bw), dtype=dense.dtype, device=dense.device)[:nnzb]
    _lib.call("spmm_build_bcsr_fill", _ptr(dense), M, K, dense.stride(0), bh, bw, _code(dense.dtype),
              _ptr(row_ptr), _ptr(col_idx), _ptr(vals), _stream(stream))
    return BCSR(M, K, bh, bw, nnzb, dense.dtype, row_ptr, col_idx, vals)


def build_bcsr(dense: torch.Tensor, bh: int, bw: int, stream=None) -> BCSR:
    row_ptr, n = spmm_build_bcsr_count(dense, bh, bw, stream)
    return spmm_build_bcsr_fill(dense, bh, bw, row_ptr, n, stream)


def spmm_bcsr(A: BCSR, B: torch.Tensor, C_: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    _check_dev(B, C_)
    N = B.shape[1]
    out = _out(C_, A.M, N, torch.float32, B.device)
    a = A.c()
    _lib.call("spmm_bcsr", C.byref(a), _ptr(B), B.stride(0), _ptr(out), out.stride(0), N, _stream(stream))
    return out


# ------------------------------------------------------------------ SDDMM
def spmm_sddmm(S: CSR, A: torch.Tensor, Bt: torch.Tensor, out: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
    """out[e] = A[i] . Bt[j] for every stored (i, j) of the CSR pattern S, in pattern
    order: fp32 for fp16/bf16 operands, exact int32 for int8 (S.dtype torch.int8)."""
    _check_dev(A, Bt, out)
    K = A.shape[1]
    if out is None:
        odt = torch.int32 if S.dtype == torch.int8 else torch.float32
        out = torch.empty(S.nnz, dtype=odt, device=A.device)
    s = S.c()
    _lib.call("spmm_sddmm", C.byref(s), K, _ptr(A), A.stride(0), _ptr(Bt), Bt.stride(0), _ptr(out), _stream(stream))
    return out


# ------------------------------------------------------------------ permutation before BCSR
def rcm_order(n: int, row_ptr, col) -> torch.Tensor:
    """Reverse Cuthill-McKee order (host) of an n x n CSR pattern given as host
    arrays (numpy or CPU tensors); returns perm as a CPU int32 tensor."""
    rp = torch.as_tensor(row_ptr, dtype=torch.int32).contiguous()
    cl = torch.as_tensor(col, dtype=torch.int32).contiguous()
    if rp.is_cuda or cl.is_cuda:
        raise ValueError("rcm_order takes host arrays")
    perm = torch.empty(n, dtype=torch.int32)
    _lib.call("spmm_rcm_order", n, _ptr(rp), _ptr(cl), _ptr(perm))
    return perm


def spmm_permute_sym(dense: torch.Tensor, perm: torch.Tensor, stream=None) -> torch.Tensor:
    """out[i][j] = dense[perm[i]][perm[j]] (P A P^T) on the device."""
    _check_dev(dense, perm)
    n = dense.shape[0]
    out = torch.empty((n, n), dtype=dense.dtype, device=dense.device)
    _lib.call("spmm_permute_sym", _ptr(dense), n, dense.stride(0), _code(dense.dtype), _ptr(perm), _ptr(out),
              out.stride(0), _stream(stream))
    return out


def spmm_permute_rows(src: torch.Tensor, perm: torch.Tensor, scatter: bool = False,
                      out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Row gather (out[i] = src[perm[i]]) or scatter (out[perm[i]] = src[i])."""
    _check_dev(src, perm, out)
    rows, cols = src.shape
    if out is None:
        out = torch.empty_like(src)
    _lib.call("spmm_permute_rows", _ptr(src), src.stride(0), _ptr(out), out.stride(0), rows, cols,
              src.element_size(), _ptr(perm), 1 if scatter else 0, _stream(stream))
    return out


def spmm_bcsr_permuted_workspace_size(A: BCSR, N: int) -> int:
    n = C.c_size_t(0)
    a = A.c()
    _lib.call("spmm_bcsr_permuted_workspace_size", C.byref(a), N, C.byref(n))
    return n.value


def spmm_bcsr_permuted(A: BCSR, perm: torch.Tensor, B: torch.Tensor, C_: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """C = A B where A is given as the BCSR of P A P^T and perm (device int32)."""
    _check_dev(perm, B, C_, workspace)
    N = B.shape[1]
    out = _out(C_, A.M, N, torch.float32, B.device)
    if workspace is None:
        workspace = torch.empty(spmm_bcsr_permuted_workspace_size(A, N), dtype=torch.uint8, device=B.device)
    a = A.c()
    _lib.call("spmm_bcsr_permuted", C.byref(a), _ptr(perm), _ptr(B), B.stride(0), _ptr(out), out.stride(0), N,
              _ptr(workspace), workspace.numel(), _stream(stream))
    return out


# ------------------------------------------------------------------ 2:4
def spmm_compress_24(dense: torch.Tensor, stream=None) -> Mat24:
    _check_dev(dense)
    M, K = dense.shape
    vals = torch.empty((M, K // 2), dtype=dense.dtype, device=dense.device)
    meta = torch.empty((M, K // 8), dtype=torch.uint8, device=dense.device)
    _lib.call("spmm_compress_24", _ptr(dense), M, K, dense.stride(0), _code(dense.dtype), _ptr(vals),
              _ptr(meta), _stream(stream))
    return Mat24(M, K, dense.dtype, vals, meta)


def spmm_prune_24(dense: torch.Tensor, stream=None) -> Mat24:
    """Magnitude-prune a dense (M x K) matrix into 2:4 (two largest |a| per group of 4)."""
    _check_dev(dense)
    M, K = dense.shape
    vals = torch.empty((M, K // 2), dtype=dense.dtype, device=dense.device)
    meta = torch.empty((M, K // 8), dtype=torch.uint8, device=dense.device)
    _lib.call("spmm_prune_24", _ptr(dense), M, K, dense.stride(0), _code(dense.dtype), _ptr(vals),
              _ptr(meta), _stream(stream))
    return Mat24(M, K, dense.dtype, vals, meta)


def spmm_24_workspace_size(A: Mat24, N: int) -> int:
    n = C.c_size_t(0)
    a = A.c()
    _lib.call("spmm_24_workspace_size", C.byref(a), N, C.byref(n))
    return n.value


def spmm_widen_24(A: Mat24, stream=None) -> Mat24:
    """int8 2:4 operand: the same operand with its values widened to fp16 once
    (vals16), so that spmm_24 widens only B on each call."""
    v16 = torch.empty((A.M, A.K // 2), dtype=torch.float16, device=A.vals.device)
    a = A.c()
    _lib.call("spmm_widen_24", C.byref(a), _ptr(v16), _stream(stream))
    return Mat24(A.M, A.K, A.dtype, A.vals, A.meta, v16)


def spmm_24(A: Mat24, B: torch.Tensor, C_: Optional[torch.Tensor] = None,
            workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    _check_dev(B, C_, workspace)
    N = B.shape[1]
    odt = torch.int32 if A.dtype == torch.int8 else torch.float32
    out = _out(C_, A.M, N, odt, B.device)
    need = spmm_24_workspace_size(A, N)
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=B.device)
    a = A.c()
    _lib.call("spmm_24", C.byref(a), _ptr(B), B.stride(0), _ptr(out), out.stride(0), N, _ptr(workspace),
              0 if workspace is None else workspace.numel() * workspace.element_size(), _stream(stream))
    return out


# ------------------------------------------------------------------ (2n-2):2n
def spmm_build_slide(dense: torch.Tensor, n: int, stream=None) -> Slide:
    """Decompose a dense (2n-2):2n matrix into its lifted 2:4 operand (n - 1
    overlapping windows per group of 2n, window-plane order)."""
    _check_dev(dense)
    M, K = dense.shape
    Kl = 4 * (n - 1) * (K // (2 * n)) if n > 0 else 0
    vals = torch.empty((M, Kl // 2), dtype=dense.dtype, device=dense.device)
    meta = torch.empty((M, Kl // 8), dtype=torch.uint8, device=dense.device)
    _lib.call("spmm_build_slide", _ptr(dense), M, K, dense.stride(0), _code(dense.dtype), n, _ptr(vals),
              _ptr(meta), _stream(stream))
    return Slide(M, K, n, dense.dtype, vals, meta)


def spmm_slide_workspace_size(A: Slide, N: int) -> int:
    n = C.c_size_t(0)
    a = A.c()
    _lib.call("spmm_slide_workspace_size", C.byref(a), N, C.byref(n))
    return n.value


def spmm_slide(A: Slide, B: torch.Tensor, C_: Optional[torch.Tensor] = None,
               workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """C = A @ B for a lifted (2n-2):2n operand; B holds the original K rows."""
    _check_dev(B, C_, workspace)
    N = B.shape[1]
    odt = torch.int32 if A.dtype == torch.int8 else torch.float32
    out = _out(C_, A.M, N, odt, B.device)
    need = spmm_slide_workspace_size(A, N)
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=B.device)
    a = A.c()
    _lib.call("spmm_slide", C.byref(a), _ptr(B), B.stride(0), _ptr(out), out.stride(0), N, _ptr(workspace),
              0 if workspace is None else workspace.numel() * workspace.element_size(), _stream(stream))
    return out


# ------------------------------------------------------------------ TVW
def spmm_build_tvw(dense: torch.Tensor, tile_rows: int, tile_ptr: torch.Tensor, cols: torch.Tensor,
                   Kp: Optional[int] = None, stream=None) -> TVW:
    _check_dev(dense, tile_ptr, cols)
    M, K = dense.shape
    n_tiles = (M + tile_rows - 1) // tile_rows
    if Kp is None:
        kt = int((tile_ptr[1:] - tile_ptr[:-1]).max().item()) if n_tiles else 0
        Kp = max(128, -(-kt // 128) * 128)
    vals = torch.empty((M, Kp // 2), dtype=dense.dtype, device=dense.device)
    meta = torch.empty((M, Kp // 8), dtype=torch.uint8, device=dense.device)
    _lib.call("spmm_build_tvw", _ptr(dense), M, K, dense.stride(0), _code(dense.dtype), tile_rows, _ptr(tile_ptr),
              _ptr(cols), n_tiles, Kp, _ptr(vals), _ptr(meta), _stream(stream))
    return TVW(M, K, tile_rows, dense.dtype, n_tiles, Kp, tile_ptr, cols, vals, meta)



def spmm_prune_tvw(dense: torch.Tensor, tile_rows: int, tile_ptr: torch.Tensor, cols: torch.Tensor,
                   Kp: Optional[int] = None, stream=None) -> TVW:
    """Magnitude-prune a dense matrix into TVW (kept columns given; 2:4 by magnitude inside)."""
    _check_dev(dense, tile_ptr, cols)
    M, K = dense.shape
    n_tiles = (M + tile_rows - 1) // tile_rows
    if Kp is None:
        kt = int((tile_ptr[1:] - tile_ptr[:-1]).max().item()) if n_tiles else 0
        Kp = max(128, -(-kt // 128) * 128)
    vals = torch.empty((M, Kp // 2), dtype=dense.dtype, device=dense.device)
    meta = torch.empty((M, Kp // 8), dtype=torch.uint8, device=dense.device)
    _lib.call("spmm_prune_tvw", _ptr(dense), M, K, dense.stride(0), _code(dense.dtype), tile_rows, _ptr(tile_ptr),
              _ptr(cols), n_tiles, Kp, _ptr(vals), _ptr(meta), _stream(stream))
    return TVW(M, K, tile_rows, dense.dtype, n_tiles, Kp, tile_ptr, cols, vals, meta)


def spmm_tvw(A: TVW, B: torch.Tensor, C_: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    _check_dev(B, C_)
    N = B.shape[1]
    out = _out(C_, A.M, N, torch.float32, B.device)
    a = A.c()
    _lib.call("spmm_tvw", C.byref(a), _ptr(B), B.stride(0), _ptr(out), out.stride(0), N, _stream(stream))
    return out


# ------------------------------------------------------------------ WCSR
def spmm_build_wcsr_workspace_size(A: CSR, h: int) -> int:
    n = C.c_size_t(0)
    a = A.c()
    _lib.call("spmm_build_wcsr_workspace_size", C.byref(a), h, C.byref(n))
    return n.value


def spmm_build_wcsr_count(A: CSR, h: int, S: int, workspace: torch.Tensor, stream=None):
    _check_dev(workspace)
    tw, tu = C.c_int64(0), C.c_int64(0)
    a = A.c()
    _lib.call("spmm_build_wcsr_count", C.byref(a), h, S, _ptr(workspace), workspace.numel(), C.byref(tw),
              C.byref(tu), _stream(stream))
    return tw.value, tu.value


def spmm_build_wcsr_fill(A: CSR, h: int, S: int, workspace: torch.Tensor, n_wcols: int, n_units: int,
                         stream=None) -> WCSR:
    dev = A.row_ptr.device
    nw = (A.M + h - 1) // h

    def i32(n):
        return torch.empty(n, dtype=torch.int32, device=dev)

    W = WCSR(A.M, A.K, A.nnz, h, S, A.dtype, nw, n_wcols, n_units, i32(nw + 1), i32(max(n_wcols, 1))[:n_wcols],
             i32(nw + 1), i32(nw + 1), i32(max(n_units, 1))[:n_units], i32(n_units + 1),
             torch.empty(max(A.nnz, 1), dtype=torch.uint8, device=dev)[:A.nnz], i32(max(A.nnz, 1))[:A.nnz],
             torch.empty(max(A.nnz, 1), dtype=A.dtype, device=dev)[:A.nnz])
    w = W.c()
    a = A.c()
    _lib.call("spmm_build_wcsr_fill", C.byref(a), h, S, _ptr(workspace), workspace.numel(), C.byref(w),
              _stream(stream))
    return W


def build_wcsr(A: CSR, h: int = 16, S: int = 32, stream=None) -> WCSR:
    ws = torch.empty(max(1, spmm_build_wcsr_workspace_size(A, h)), dtype=torch.uint8, device=A.row_ptr.device)
    tw, tu = spmm_build_wcsr_count(A, h, S, ws, stream)
    return spmm_build_wcsr_fill(A, h, S, ws, tw, tu, stream)


def spmm_wcsr_workspace_size(A: WCSR, N: int) -> int:
    n = C.c_size_t(0)
    a = A.c()
    _lib.call("spmm_wcsr_workspace_size", C.byref(a), N, C.byref(n))
    return n.value


def spmm_wcsr(A: WCSR, B: torch.Tensor, C_: Optional[torch.Tensor] = None,
              workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """C = A B for a row-window operand (tensor-core window products).  The
    workspace (kept on A when not given) needs no clearing between calls."""
    _check_dev(B, C_, workspace)
    N = B.shape[1]
    out = _out(C_, A.M, N, torch.float32, B.device)
    if workspace is None:
        need = spmm_wcsr_workspace_size(A, N)
        if A.workspace is None or A.workspace.numel() < need:
            A.workspace = torch.zeros(max(need, 1), dtype=torch.uint8, device=B.device)
        workspace = A.workspace
    a = A.c()
    _lib.call("spmm_wcsr", C.byref(a), _ptr(B), B.stride(0), _ptr(out), out.stride(0), N, _ptr(workspace),
              workspace.numel(), _stream(stream))
    return out


# ------------------------------------------------------------------ one-hot operators
_ROW_DT = {torch.bfloat16: _lib.SPMM_BF16, torch.float16: _lib.SPMM_F16, torch.float32: _lib.SPMM_F32}
_ID_BYTES = {torch.int32: 4, torch.int64: 8}


class Route:
    """T x k ids sorted by value: order (flat indices, dropped ones last), pos
    (place of each flat index, -1 if dropped), offsets (first place per key) and,
    for k = 1, keys (the sorted ids, n_keys if dropped).  All int32 on the device;
    pos has the ids' shape.  A route does not change after it is built: its C
    struct holds the tensors' addresses, so assigning to a field raises.  Copies
    and pickles build a struct of their own."""

    def __init__(self, T: int, k: int, n_keys: int, order: torch.Tensor, pos: torch.Tensor, offsets: torch.Tensor,
                 keys: Optional[torch.Tensor] = None):
        ref = C.byref(_lib.RouteT(T, k, n_keys, order.data_ptr(), pos.data_ptr(), offsets.data_ptr(),
                                  None if keys is None else keys.data_ptr()))
        self.__dict__.update(T=T, k=k, n_keys=n_keys, n_rows=T * k, order=order, pos=pos, offsets=offsets, keys=keys,
                             device=order.device, shape=pos.shape, _ref=ref)

    def __setattr__(self, name, value):
        raise AttributeError(f"cannot assign to {name}: a route does not change after it is built")

    def __delattr__(self, name):
        raise AttributeError(f"cannot delete {name}: a route does not change after it is built")

    def __reduce__(self):
        return Route, (self.T, self.k, self.n_keys, self.order, self.pos, self.offsets, self.keys)

    def c(self) -> _lib.RouteT:
        return self._ref._obj


# At decoding sizes the kernels take 2-4 us, so the wrappers below spend as little
# as they can: addresses go to ctypes as integers, the stream handle comes without
# a Stream object (3 us), and a route's struct is built once.
def _row_code(dtype) -> int:
    code = _ROW_DT.get(dtype)
    if code is None:
        raise TypeError(f"unsupported row dtype {dtype}")
    return code


def _handle(stream, device):
    """The raw handle of the call's stream.  The library launches on the current device, so operands or a
    stream of another one are refused."""
    current = torch._C._cuda_getDevice()
    if device.index != current:
        raise ValueError(f"operands are on {device}, but the current device is cuda:{current} (torch.cuda.set_device)")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(current)
    if stream.device_index != current:
        raise ValueError(f"the stream belongs to cuda:{stream.device_index}, but the current device is cuda:{current}")
    return stream.cuda_stream


def _empty(like: torch.Tensor, shape, dtype, stream):
    """A new tensor on like's device whose memory belongs to the stream the kernel runs on."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def _rows(t: torch.Tensor, what: str, rows: int, H: int, dtype, device) -> int:
    """Check a rows x H operand of the type on the device; returns its row pitch."""
    if t.device != device or not t.is_cuda:
        raise ValueError(f"{what} must be on {device} (this library has no CPU path)")
    if t.dtype is not dtype:
        raise TypeError(f"{what} must be {dtype}, not {t.dtype}")
    if t.shape != (rows, H):
        raise ValueError(f"{what} must be {rows} x {H}, not {tuple(t.shape)}")
    ld, inner = t.stride()
    if inner != 1 and H > 1 and rows > 0:
        raise ValueError(f"{what} must have contiguous rows")
    return ld if rows > 1 else H


def _weights(t: torch.Tensor, what: str, E: int, N: int, K: int, dtype, device):
    """Check an E x N x K operand; returns its row and expert pitches."""
    if t.device != device or not t.is_cuda:
        raise ValueError(f"{what} must be on {device} (this library has no CPU path)")
    if t.dtype is not dtype:
        raise TypeError(f"{what} must be {dtype}, not {t.dtype}")
    if t.shape != (E, N, K):
        raise ValueError(f"{what} must be {E} x {N} x {K}, not {tuple(t.shape)}")
    if K > 1 and t.stride(2) != 1:
        raise ValueError(f"{what} must have contiguous rows")
    ldw = t.stride(1) if N > 1 else K
    return ldw, (t.stride(0) if E > 1 else N * ldw)


def _route_w(R: Route, w: torch.Tensor, device) -> int:
    if w.device != device or w.dtype is not torch.float32:
        raise TypeError(f"w must be float32 on {device}")
    if w.shape != R.shape or not w.is_contiguous():
        raise ValueError(f"w must be a contiguous tensor of the ids' shape {tuple(R.shape)}")
    return w.data_ptr()


def spmm_build_route_workspace_size(T: int, k: int, n_keys: int) -> int:
    if k >= 1 << 31:  # the C entry takes 32 bits, of which ctypes would keep the lower ones
        raise SpmmError("spmm_build_route_workspace_size", 8)
    n = C.c_size_t(0)
    _lib.call("spmm_build_route_workspace_size", T, k, n_keys, C.byref(n))
    return n.value


def _workspace(workspace: Optional[torch.Tensor], need: int, like: torch.Tensor, stream):
    """(tensor, address, bytes) of the caller's workspace, or of a new one if one is needed."""
    if workspace is None:
        if not need:
            return None, None, 0
        workspace = _empty(like, need, torch.uint8, stream)
    elif workspace.device != like.device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {like.device}")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def spmm_build_route(ids: torch.Tensor, n_keys: int, workspace: Optional[torch.Tensor] = None,
                     stream=None) -> Route:
    """Sort ids (T, or T x k; int32 or int64) by value.  Negative ids are dropped
    choices; ids >= n_keys are dropped too and set SPMM_DEVERR_INDEX."""
    _check_dev(ids)
    if ids.dtype not in _ID_BYTES:
        raise TypeError(f"ids must be int32 or int64, not {ids.dtype}")
    shape = ids.shape
    if len(shape) not in (1, 2):
        raise ValueError("ids must be T or T x k")
    T, k = shape[0], (1 if len(shape) == 1 else shape[1])
    if k > 1 and T > 0 and ids.stride(1) != 1:
        raise ValueError("ids must have contiguous rows")
    need = spmm_build_route_workspace_size(T, k, n_keys)
    ws, ws_ptr, ws_bytes = _workspace(workspace, need, ids, stream)
    i32 = torch.int32
    R = Route(T, k, n_keys, _empty(ids, T * k, i32, stream), _empty(ids, shape, i32, stream),
              _empty(ids, n_keys + 1, i32, stream), _empty(ids, T, i32, stream) if k == 1 else None)
    _lib.call("spmm_build_route", ids.data_ptr(), _ID_BYTES[ids.dtype], ids.stride(0) if T > 1 else k, R._ref, ws_ptr,
              ws_bytes, _handle(stream, ids.device))
    return R


def spmm_dispatch(R: Route, x: torch.Tensor, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """xs[p] = x[order[p] // k] for the kept places, zero rows after them."""
    H, dev, dt, rows = x.shape[-1], R.device, x.dtype, R.n_rows
    code, ldx = _row_code(dt), _rows(x, "x", R.T, H, dt, dev)
    if out is None:
        out, ldo = _empty(x, (rows, H), dt, stream), H
    else:
        ldo = _rows(out, "out", rows, H, dt, dev)
    _lib.call("spmm_dispatch", R._ref, x.data_ptr(), ldx, out.data_ptr(), ldo, H, code, _handle(stream, dev))
    return out


def spmm_combine(R: Route, ys: torch.Tensor, w: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
    """y[t] = sum_j w[t, j] ys[pos[t, j]] over the kept choices (w fp32; None: weights of 1)."""
    H, dev, dt = ys.shape[-1], R.device, ys.dtype
    code, ldys = _row_code(dt), _rows(ys, "ys", R.n_rows, H, dt, dev)
    w_ptr = None if w is None else _route_w(R, w, dev)
    if out is None:
        out, ldo = _empty(ys, (R.T, H), dt, stream), H
    else:
        ldo = _rows(out, "out", R.T, H, dt, dev)
    _lib.call("spmm_combine", R._ref, ys.data_ptr(), ldys, w_ptr, out.data_ptr(), ldo, H, code, _handle(stream, dev))
    return out


def spmm_dispatch_grad(R: Route, dxs: torch.Tensor, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Gradient of spmm_dispatch: dx[t] = sum_j dxs[pos[t, j]] (spmm_combine with weights of 1)."""
    return spmm_combine(R, dxs, None, out, stream)


def spmm_combine_grad(R: Route, dy: torch.Tensor, ys: torch.Tensor, w: torch.Tensor,
                      out: Optional[torch.Tensor] = None, stream=None):
    """Gradients of spmm_combine: (dys, dw) with dys[pos[t, j]] = w[t, j] dy[t] (zero
    rows past the kept places) and dw[t, j] = <dy[t], ys[pos[t, j]]>, fp32, of w's shape."""
    H, dev, dt, rows = dy.shape[-1], R.device, dy.dtype, R.n_rows
    code, lddy, ldys = _row_code(dt), _rows(dy, "dy", R.T, H, dt, dev), _rows(ys, "ys", rows, H, dt, dev)
    w_ptr = _route_w(R, w, dev)
    if out is None:
        out, ldo = _empty(dy, (rows, H), dt, stream), H
    else:
        ldo = _rows(out, "out", rows, H, dt, dev)
    dw = _empty(w, w.shape, torch.float32, stream)
    _lib.call("spmm_combine_grad", R._ref, dy.data_ptr(), lddy, ys.data_ptr(), ldys, w_ptr, out.data_ptr(), ldo,
              dw.data_ptr(), H, code, _handle(stream, dev))
    return out, dw


def spmm_embed(table: torch.Tensor, ids: torch.Tensor, scale: float = 1.0, out: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
    """out[t] = scale * table[ids[t]]; a negative id (padding) gives a zero row, an id
    past the table as well and sets SPMM_DEVERR_INDEX."""
    V, H, dev, dt = table.shape[0], table.shape[-1], table.device, table.dtype
    code, ldt = _row_code(dt), _rows(table, "table", V, H, dt, dev)
    id_bytes = _ID_BYTES.get(ids.dtype)
    if id_bytes is None:
        raise TypeError(f"ids must be int32 or int64, not {ids.dtype}")
    if ids.dim() != 1 or ids.device != dev or not ids.is_contiguous():
        raise ValueError(f"ids must be a contiguous vector on {dev}")
    T = ids.shape[0]
    if out is None:
        out, ldo = _empty(table, (T, H), dt, stream), H
    else:
        ldo = _rows(out, "out", T, H, dt, dev)
    _lib.call("spmm_embed", table.data_ptr(), V, H, ldt, code, ids.data_ptr(), id_bytes, T, scale, out.data_ptr(), ldo,
              _handle(stream, dev))
    return out


def spmm_embed_grad_workspace_size(R: Route, H: int) -> int:
    n = C.c_size_t(0)
    _lib.call("spmm_embed_grad_workspace_size", R._ref, H, C.byref(n))
    return n.value


def spmm_embed_grad(R: Route, dy: torch.Tensor, scale: float = 1.0, out: Optional[torch.Tensor] = None,
                    accumulate: bool = False, workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Gradient of spmm_embed for the table, from the route of the ids (k = 1, n_keys
    = V): scale * the sum of dy over each row's tokens.  Every row is written, or
    with accumulate the sums are added to out.  out is dy's type (default) or fp32."""
    H, dev, dt = dy.shape[-1], R.device, dy.dtype
    code, lddy = _row_code(dt), _rows(dy, "dy", R.T, H, dt, dev)
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs out")
        out, ldo = _empty(dy, (R.n_keys, H), dt, stream), H
    else:
        ldo = _rows(out, "out", R.n_keys, H, out.dtype, dev)
    ws, ws_ptr, ws_bytes = _workspace(workspace, spmm_embed_grad_workspace_size(R, H), dy, stream)
    _lib.call("spmm_embed_grad", R._ref, dy.data_ptr(), lddy, H, code, scale, 1 if accumulate else 0, out.data_ptr(),
              ldo, _row_code(out.dtype), ws_ptr, ws_bytes, _handle(stream, dev))
    return out


def spmm_experts(R: Route, xs: torch.Tensor, W: torch.Tensor, out: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
    """ys[p] = W[e] xs[p] for the rows p of expert e (W is E x N x K, R.n_keys = E);
    zero rows past the kept places.  bf16 or fp16."""
    dev, dt, rows = R.device, xs.dtype, R.n_rows
    N, K = W.shape[-2], W.shape[-1]
    code, ldx = _row_code(dt), _rows(xs, "xs", rows, K, dt, dev)
    ldw, lde = _weights(W, "W", R.n_keys, N, K, dt, dev)
    if out is None:
        out, ldo = _empty(xs, (rows, N), dt, stream), N
    else:
        ldo = _rows(out, "out", rows, N, dt, dev)
    _lib.call("spmm_experts", R._ref, xs.data_ptr(), ldx, W.data_ptr(), ldw, lde, N, K, code, out.data_ptr(), ldo,
              _handle(stream, dev))
    return out


def spmm_experts_dx(R: Route, dys: torch.Tensor, W: torch.Tensor, out: Optional[torch.Tensor] = None,
                    stream=None) -> torch.Tensor:
    """dxs[p] = W[e]^T dys[p] for the rows p of expert e; zero rows past the kept places."""
    dev, dt, rows = R.device, dys.dtype, R.n_rows
    N, K = W.shape[-2], W.shape[-1]
    code, ldy = _row_code(dt), _rows(dys, "dys", rows, N, dt, dev)
    ldw, lde = _weights(W, "W", R.n_keys, N, K, dt, dev)
    if out is None:
        out, ldo = _empty(dys, (rows, K), dt, stream), K
    else:
        ldo = _rows(out, "out", rows, K, dt, dev)
    _lib.call("spmm_experts_dx", R._ref, dys.data_ptr(), ldy, W.data_ptr(), ldw, lde, N, K, code, out.data_ptr(), ldo,
              _handle(stream, dev))
    return out


def spmm_experts_dw(R: Route, dys: torch.Tensor, xs: torch.Tensor, out: Optional[torch.Tensor] = None,
                    stream=None) -> torch.Tensor:
    """dW[e] = sum of dys[p] xs[p]^T over the rows p of expert e (E x N x K; zeros for an unused expert)."""
    dev, dt, rows, E = R.device, dys.dtype, R.n_rows, R.n_keys
    N, K = dys.shape[-1], xs.shape[-1]
    code, ldy, ldx = _row_code(dt), _rows(dys, "dys", rows, N, dt, dev), _rows(xs, "xs", rows, K, dt, dev)
    if out is None:
        out = _empty(dys, (E, N, K), dt, stream)
    ldw, lde = _weights(out, "out", E, N, K, dt, dev)
    _lib.call("spmm_experts_dw", R._ref, dys.data_ptr(), ldy, xs.data_ptr(), ldx, N, K, code, out.data_ptr(), ldw, lde,
              _handle(stream, dev))
    return out


def spmm_experts_grad(R: Route, dys: torch.Tensor, xs: torch.Tensor, W: torch.Tensor, stream=None):
    """Both gradients of spmm_experts: (dxs, dW)."""
    return spmm_experts_dx(R, dys, W, stream=stream), spmm_experts_dw(R, dys, xs, stream=stream)


# ------------------------------------------------------------------ gated experts
_ACTS = {"silu": _lib.ACT_SILU, "gelu": _lib.ACT_GELU, "gelu_tanh": _lib.ACT_GELU_TANH}


class Rows8:
    """rows x cols values of dtype held in 8 bits: 16 consecutive values of a row share
    a power of two, value = q 2^(scale - 127) (scale 255: NaN).  q is int8, rows x
    cols, scale uint8, rows x ceil(cols / 16); both may be views of wider rows.  Like a
    Route it holds its tensors' addresses, so assigning to a field raises."""

    def __init__(self, rows: int, cols: int, dtype: torch.dtype, q: torch.Tensor, scale: torch.Tensor):
        groups = -(-cols // 16)
        for t, what, dt, n in ((q, "q", torch.int8, cols), (scale, "scale", torch.uint8, groups)):
            if not t.is_cuda or t.device != q.device:
                raise ValueError("q and scale must be on one CUDA device (this library has no CPU path)")
            if t.dtype is not dt or t.shape != (rows, n):
                raise ValueError(f"{what} must be {rows} x {n} of {dt}")
            if n > 1 and rows > 0 and t.stride(1) != 1:
                raise ValueError(f"{what} must have contiguous rows")
        self._hold(rows, cols, dtype, q, q.stride(0) if rows > 1 else groups * 16, scale,
                   scale.stride(0) if rows > 1 else groups)

    def _hold(self, rows, cols, dtype, q, ldq, scale, lds):
        self.__dict__.update(rows=rows, cols=cols, dtype=dtype, q=q, scale=scale, device=q.device,
                             _ref=C.byref(_lib.Rows8T(rows, cols, q.data_ptr(), ldq, scale.data_ptr(), lds)))

    def __setattr__(self, name, value):
        raise AttributeError(f"cannot assign to {name}: 8-bit rows hold their tensors' addresses")

    def __delattr__(self, name):
        raise AttributeError(f"cannot delete {name}: 8-bit rows hold their tensors' addresses")

    def __reduce__(self):
        return Rows8, (self.rows, self.cols, self.dtype, self.q, self.scale)

    def c(self) -> _lib.Rows8T:
        return self._ref._obj


def _rows8(like: torch.Tensor, rows: int, cols: int, dtype, stream) -> Rows8:
    """Unwritten 8-bit rows; the pitch of q is a multiple of 16, so that every row moves in wide pieces."""
    groups = (cols + 15) // 16
    ldq = groups * 16
    if stream is None:  # (slicing a wider tensor costs the host twice as much)
        q = torch.empty_strided((rows, cols), (ldq, 1), dtype=torch.int8, device=like.device)
    else:
        with torch.cuda.stream(stream):
            q = torch.empty_strided((rows, cols), (ldq, 1), dtype=torch.int8, device=like.device)
    P = Rows8.__new__(Rows8)
    P._hold(rows, cols, dtype, q, ldq, _empty(like, (rows, groups), torch.uint8, stream), groups)
    return P


def _act(act: str) -> int:
    code = _ACTS.get(act)
    if code is None:
        raise ValueError(f"act must be one of {', '.join(_ACTS)}, not {act!r}")
    return code


def spmm_topk(logits: torch.Tensor, k: int, renorm: bool = True, id_dtype=torch.int64, stream=None):
    """The router: (ids, w) of each token's k largest logits (T x E; bf16, fp16 or
    fp32), largest first, equal ones by ascending index.  w (fp32) is the softmax over
    the chosen logits, or with renorm=False their entries of the softmax over all E.
    -inf is never chosen: id -1 (dropped by spmm_build_route) and weight 0 take its
    place.  NaN ranks first and makes the token's weights NaN.  k <= 32, E <= 1024."""
    _check_dev(logits)
    T, E = logits.shape
    dev = logits.device
    code, ldl = _row_code(logits.dtype), _rows(logits, "logits", T, E, logits.dtype, dev)
    id_bytes = _ID_BYTES.get(id_dtype)
    if id_bytes is None:
        raise TypeError(f"ids must be int32 or int64, not {id_dtype}")
    if not 0 < k <= E:
        raise ValueError(f"k must be between 1 and {E}, not {k}")
    ids, w = _empty(logits, (T, k), id_dtype, stream), _empty(logits, (T, k), torch.float32, stream)
    _lib.call("spmm_topk", logits.data_ptr(), T, E, ldl, code, k, 1 if renorm else 0, ids.data_ptr(), id_bytes, w.data_ptr(),
              _handle(stream, dev))
    return ids, w


def spmm_topk_grad(logits: torch.Tensor, ids: torch.Tensor, w: torch.Tensor, dw: torch.Tensor, renorm: bool = True,
                   out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Gradient of spmm_topk's weights for the logits (T x E of their type; every entry
    written), from its ids and w and the gradient dw of w.  A negative id is a dropped
    choice; an id >= E as well and sets SPMM_DEVERR_INDEX."""
    _check_dev(logits)
    T, E = logits.shape
    dev = logits.device
    code, ldl = _row_code(logits.dtype), _rows(logits, "logits", T, E, logits.dtype, dev)
    id_bytes = _ID_BYTES.get(ids.dtype)
    if id_bytes is None:
        raise TypeError(f"ids must be int32 or int64, not {ids.dtype}")
    if ids.dim() != 2 or ids.shape[0] != T or ids.device != dev or not ids.is_contiguous():
        raise ValueError(f"ids must be a contiguous {T} x k tensor on {dev}")
    for t, what in ((w, "w"), (dw, "dw")):
        if t.device != dev or t.dtype is not torch.float32:
            raise TypeError(f"{what} must be float32 on {dev}")
        if t.shape != ids.shape or not t.is_contiguous():
            raise ValueError(f"{what} must be a contiguous tensor of the ids' shape {tuple(ids.shape)}")
    k = ids.shape[1]
    if not 0 < k <= E:
        raise ValueError(f"k must be between 1 and {E}, not {k}")
    if out is None:
        out, ldo = _empty(logits, (T, E), logits.dtype, stream), E
    else:
        ldo = _rows(out, "out", T, E, logits.dtype, dev)
    _lib.call("spmm_topk_grad", logits.data_ptr(), T, E, ldl, code, k, 1 if renorm else 0, ids.data_ptr(), id_bytes,
              w.data_ptr(), dw.data_ptr(), out.data_ptr(), ldo, _handle(stream, dev))
    return out


def spmm_pack_rows(x: torch.Tensor, out: Optional[Rows8] = None, stream=None) -> Rows8:
    """A checkpoint of rows x (bf16, fp16 or fp32) in 8 bits: Rows8, 17/16 bytes a value.
    A value is off by at most half a unit of its group, 1/255 to 1/127.5 of the
    group's largest magnitude."""
    _check_dev(x)
    rows, cols = x.shape
    code, ldx = _row_code(x.dtype), _rows(x, "x", rows, cols, x.dtype, x.device)
    if out is None:
        out = _rows8(x, rows, cols, x.dtype, stream)
    elif (out.rows, out.cols, out.dtype, out.device) != (rows, cols, x.dtype, x.device):
        raise ValueError(f"out must hold {rows} x {cols} values of {x.dtype} on {x.device}")
    _lib.call("spmm_pack_rows", x.data_ptr(), ldx, code, out._ref, _handle(stream, x.device))
    return out


def spmm_unpack_rows(P: Rows8, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The rows that P holds, of P.dtype (or of out's type).  fp16: 65536, as which the largest
    values are held, reads as 65504; larger ones become infinity."""
    dev = P.device
    if out is None:
        out, ldo = _empty(P.q, (P.rows, P.cols), P.dtype, stream), P.cols
    else:
        ldo = _rows(out, "out", P.rows, P.cols, out.dtype, dev)
    _lib.call("spmm_unpack_rows", P._ref, out.data_ptr(), ldo, _row_code(out.dtype), _handle(stream, dev))
    return out


def spmm_experts_gated(R: Route, xs: torch.Tensor, W: torch.Tensor, act: str = "silu", save: Optional[str] = None,
                       out: Optional[torch.Tensor] = None, stream=None):
    """h[p] = act(g) u with [g u] = W[e] xs[p] for the rows p of expert e: W is E x 2N x
    K, the gate's N rows before the up projection's; act is silu, gelu or gelu_tanh;
    zero rows past the kept places.  bf16 or fp16, N a multiple of 16.  A training step
    keeps [g u] (T k x 2N) for spmm_experts_gated_grad: save="rows" returns (h, gu)
    with gu of xs's type, save="packed" (h, Rows8) with gu in 8 bits.  h has the same bits
    whatever is saved, but for fp16 with save="packed", whose last bits can differ (the
    depth is summed in two halves)."""
    dev, dt, rows = R.device, xs.dtype, R.n_rows
    N, K = W.shape[-2] // 2, W.shape[-1]
    code, ldx, actc = _row_code(dt), _rows(xs, "xs", rows, K, dt, dev), _act(act)
    ldw, lde = _weights(W, "W", R.n_keys, 2 * N, K, dt, dev)
    if save not in (None, "rows", "packed"):
        raise ValueError(f"save must be None, 'rows' or 'packed', not {save!r}")
    if out is None:
        out, ldo = _empty(xs, (rows, N), dt, stream), N
    else:
        ldo = _rows(out, "out", rows, N, dt, dev)
    gu = _empty(xs, (rows, 2 * N), dt, stream) if save == "rows" else None
    packed = _rows8(xs, rows, 2 * N, dt, stream) if save == "packed" else None
    _lib.call("spmm_experts_gated", R._ref, xs.data_ptr(), ldx, W.data_ptr(), ldw, lde, N, K, code, actc, out.data_ptr(), ldo,
              None if gu is None else gu.data_ptr(), 2 * N, None if packed is None else packed._ref,
              _handle(stream, dev))
    return out if save is None else (out, gu if packed is None else packed)


def spmm_gated_grad(R: Route, dh: torch.Tensor, gu, act: str = "silu", with_h: bool = False,
                    out: Optional[torch.Tensor] = None, stream=None):
    """Gradient of h = act(g) u for [g u], from the kept gu (rows or Rows8) and the
    gradient dh: dgu (T k x 2N), zero rows past the kept places.  with_h returns (dgu,
    h): h again, which the gradient of the projection after it needs."""
    dev, dt, rows = R.device, dh.dtype, R.n_rows
    N = dh.shape[-1]
    code, ldd, actc = _row_code(dt), _rows(dh, "dh", rows, N, dt, dev), _act(act)
    gu_ptr, ldgu, packed = _kept(gu, rows, N, dt, dev)
    if out is None:
        out, ldo = _empty(dh, (rows, 2 * N), dt, stream), 2 * N
    else:
        ldo = _rows(out, "out", rows, 2 * N, dt, dev)
    h = _empty(dh, (rows, N), dt, stream) if with_h else None
    _lib.call("spmm_gated_grad", R._ref, dh.data_ptr(), ldd, gu_ptr, ldgu, packed, N, code, actc, out.data_ptr(), ldo,
              None if h is None else h.data_ptr(), N, _handle(stream, dev))
    return (out, h) if with_h else out


def _kept(gu, rows: int, N: int, dtype, device):
    """(address, pitch, 8-bit struct) of what a forward call kept of [g u]."""
    if isinstance(gu, Rows8):
        if (gu.rows, gu.cols, gu.dtype, gu.device) != (rows, 2 * N, dtype, device):
            raise ValueError(f"gu must hold {rows} x {2 * N} values of {dtype} on {device}")
        return None, 2 * N, gu._ref
    return gu.data_ptr(), _rows(gu, "gu", rows, 2 * N, dtype, device), None


def spmm_experts_gated_grad_workspace_size(R: Route, N: int, K: int, packed_rows: bool) -> int:
    n = C.c_size_t(0)
    _lib.call("spmm_experts_gated_grad_workspace_size", R._ref, N, K, 1 if packed_rows else 0, C.byref(n))
    return n.value


def spmm_experts_gated_grad(R: Route, dh: torch.Tensor, xs, W: torch.Tensor, gu, act: str = "silu",
                            workspace: Optional[torch.Tensor] = None, stream=None):
    """The gradients (dgu, dxs, dW) of spmm_experts_gated from the gradient dh of h: xs
    (rows, or the Rows8 checkpoint of them) and W as in the forward call, gu what it saved.
    dxs and dW are products of dgu as it is rounded."""
    dev, dt, rows = R.device, dh.dtype, R.n_rows
    N, K = dh.shape[-1], W.shape[-1]
    code, ldd, actc = _row_code(dt), _rows(dh, "dh", rows, N, dt, dev), _act(act)
    gu_ptr, ldgu, packed = _kept(gu, rows, N, dt, dev)
    ldw, lde = _weights(W, "W", R.n_keys, 2 * N, K, dt, dev)
    if isinstance(xs, Rows8):
        if (xs.rows, xs.cols, xs.dtype, xs.device) != (rows, K, dt, dev):
            raise ValueError(f"xs must hold {rows} x {K} values of {dt} on {dev}")
        xs_ptr, ldx, xs8 = None, K, xs._ref
    else:
        xs_ptr, ldx, xs8 = xs.data_ptr(), _rows(xs, "xs", rows, K, dt, dev), None
    need = spmm_experts_gated_grad_workspace_size(R, N, K, xs8 is not None)
    dgu, dxs = _empty(dh, (rows, 2 * N), dt, stream), _empty(dh, (rows, K), dt, stream)
    dW = _empty(dh, (R.n_keys, 2 * N, K), dt, stream)
    ws, ws_ptr, ws_bytes = _workspace(workspace, need, dh, stream)
    _lib.call("spmm_experts_gated_grad", R._ref, dh.data_ptr(), ldd, xs_ptr, ldx, xs8, W.data_ptr(), ldw, lde, gu_ptr, ldgu,
              packed, N, K, code, actc, dgu.data_ptr(), 2 * N, dxs.data_ptr(), K, dW.data_ptr(), K, 2 * N * K, ws_ptr, ws_bytes,
              _handle(stream, dev))
    return dgu, dxs, dW
