"""Thin ctypes binding of ``libpararnn.so`` (the C ABI in ``include/pararnn.h``).

Argument marshalling only: every step of the solve runs in the library's CUDA
kernels.  PyTorch supplies device memory and the current stream.  There is no
CPU path: if the library is missing or a tensor is not on a CUDA device, the
call raises.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libpararnn.so")

DEER, QUASI, ELK, QUASI_ELK = 0, 1, 2, 3
MODES = {"DEER": DEER, "QUASI": QUASI, "ELK": ELK, "QUASI_ELK": QUASI_ELK}
GRU_DENSE, GRU_DIAG, LSTM_DIAG = 0, 1, 2
F32, BF16 = 0, 1
ACTIVATIONS = {"none": 0, "silu": 1, "gelu": 2}
STATUS = {0: "OK", 1: "NOT_CONVERGED", 2: "DIVERGED", 3: "INVALID_ARG", 4: "CUDA_ERROR",
          5: "TIMEOUT"}
EXPORTS = ("pararnn_workspace_size", "pararnn_newton_solve", "pararnn_newton_solve_async",
           "pararnn_input_projection", "pararnn_newton_iterate_async",
           "pararnn_affine_scan_workspace_size", "pararnn_affine_scan",
           "pararnn_affine_scan_status", "pararnn_status_string", "pararnn_newton_solve_host",
           "pararnn_host_workspace_size", "pararnn_adjoint", "pararnn_adjoint_workspace_size",
           "pararnn_adjoint_status", "pararnn_newton_solve_guess_async", "pararnn_newton_solve_chunked",
           "pararnn_chunked_workspace_size", "pararnn_lstm_solve", "pararnn_lstm_workspace_size",
           "pararnn_newton_solve_reuse", "pararnn_reuse_workspace_size", "pararnn_lstm_solve_host",
           "pararnn_lstm_host_workspace_size", "pararnn_adjoint_host", "pararnn_adjoint_host_workspace_size",
           "pararnn_newton_solve_trace", "pararnn_test_withheld_publish", "pararnn_adjoint_exact",
           "pararnn_adjoint_exact_workspace_size", "pararnn_newton_solve_host_streamed",
           "pararnn_host_streamed_workspace_size", "pararnn_lstm_solve_host_streamed",
           "pararnn_lstm_host_streamed_workspace_size", "pararnn_affine_scan_host",
           "pararnn_affine_scan_host_workspace_size", "pararnn_linear_attention",
           "pararnn_linear_attention_workspace_size", "pararnn_linear_attention_backward",
           "pararnn_linear_attention_backward_workspace_size", "pararnn_linear_attention_step",
           "pararnn_group_norm", "pararnn_group_norm_workspace_size", "pararnn_group_norm_backward",
           "pararnn_group_norm_backward_workspace_size")


class Cell(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int), ("din", ctypes.c_int), ("d", ctypes.c_int),
                ("x_dtype", ctypes.c_int), ("w_dtype", ctypes.c_int)]


class Params(ctypes.Structure):
    _fields_ = [("w_ih", ctypes.c_void_p), ("b_ih", ctypes.c_void_p),
                ("w_hh", ctypes.c_void_p), ("b_hh", ctypes.c_void_p)]


class Info(ctypes.Structure):
    _fields_ = [("iters", ctypes.c_int), ("status", ctypes.c_int),
                ("delta", ctypes.c_float), ("residual", ctypes.c_float)]


class Rows(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("stride_b", ctypes.c_longlong), ("stride_t", ctypes.c_longlong),
                ("stride_h", ctypes.c_longlong)]


class AttentionShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("B", "T", "H", "Hkv", "dk", "dv", "dtype")] + [("scale", ctypes.c_float)]


class NormShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("N", "S", "C", "groups", "x_dtype", "y_dtype", "act")] + [
        ("eps", ctypes.c_float)]


_lib = None


def lib() -> ctypes.CDLL:
    """Load the library once; raise if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(
                f"{_LIB_PATH} is missing: build it with `python -m newton_solve_nonlinear_b200.build`")
        L = ctypes.CDLL(_LIB_PATH)
        vp, ci, cf, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        L.pararnn_workspace_size.argtypes = [ctypes.POINTER(Cell), ci, ci, ci]
        L.pararnn_workspace_size.restype = sz
        solve_args = [ctypes.POINTER(Cell), ctypes.POINTER(Params), vp, vp, ci, ci, ci, cf, cf, ci,
                      vp, vp, vp, sz, vp]
        L.pararnn_newton_solve.argtypes = solve_args
        L.pararnn_newton_solve.restype = ci
        L.pararnn_newton_solve_async.argtypes = solve_args
        L.pararnn_newton_solve_async.restype = ci
        L.pararnn_input_projection.argtypes = [ctypes.POINTER(Cell), ctypes.POINTER(Params), vp, ci,
                                               ci, vp, vp]
        L.pararnn_input_projection.restype = ci
        L.pararnn_newton_iterate_async.argtypes = solve_args
        L.pararnn_newton_iterate_async.restype = ci
        L.pararnn_affine_scan_workspace_size.argtypes = [ci, ci, ci, ci]
        L.pararnn_affine_scan_workspace_size.restype = sz
        L.pararnn_affine_scan.argtypes = [vp, vp, vp, ci, ci, ci, ci, vp, vp, sz, vp]
        L.pararnn_affine_scan.restype = ci
        L.pararnn_affine_scan_status.argtypes = [vp, vp]
        L.pararnn_affine_scan_status.restype = ci
        L.pararnn_affine_scan_host.argtypes = [vp, vp, vp, ci, ci, ci, ci, vp, ci, vp, sz, vp]
        L.pararnn_affine_scan_host.restype = ci
        L.pararnn_affine_scan_host_workspace_size.argtypes = [ci, ci, ci, ci, ci]
        L.pararnn_affine_scan_host_workspace_size.restype = sz
        L.pararnn_newton_solve_host.argtypes = [ctypes.POINTER(Cell), ctypes.POINTER(Params), vp, vp,
                                                ci, ci, ci, cf, cf, ci, vp, vp, ci, vp, sz, vp]
        L.pararnn_newton_solve_host.restype = ci
        L.pararnn_host_workspace_size.argtypes = [ctypes.POINTER(Cell), ci, ci, ci, ci]
        L.pararnn_host_workspace_size.restype = sz
        L.pararnn_newton_solve_host_streamed.argtypes = L.pararnn_newton_solve_host.argtypes
        L.pararnn_newton_solve_host_streamed.restype = ci
        L.pararnn_host_streamed_workspace_size.argtypes = [ctypes.POINTER(Cell), ci, ci, ci, ci]
        L.pararnn_host_streamed_workspace_size.restype = sz
        L.pararnn_adjoint.argtypes = [ctypes.POINTER(Cell), ctypes.POINTER(Params), vp, vp, vp, vp, ci, ci,
                                      vp, vp, vp, vp, vp, sz, vp]
        L.pararnn_adjoint.restype = ci
        L.pararnn_adjoint_workspace_size.argtypes = [ctypes.POINTER(Cell), ci, ci]
        L.pararnn_adjoint_workspace_size.restype = sz
        L.pararnn_adjoint_status.argtypes = [vp, vp]
        L.pararnn_adjoint_status.restype = ci
        L.pararnn_newton_solve_guess_async.argtypes = [ctypes.POINTER(Cell), ctypes.POINTER(Params), vp, vp, vp,
                                                       ci, ci, ci, cf, cf, ci, vp, vp, vp, sz, vp]
        L.pararnn_newton_solve_guess_async.restype = ci
        L.pararnn_newton_solve_chunked.argtypes = [ctypes.POINTER(Cell), ctypes.POINTER(Params), vp, vp, ci, ci,
                                                   ci, ci, cf, cf, ci, vp, ctypes.POINTER(Info), vp, sz, vp]
        L.pararnn_newton_solve_chunked.restype = ci
        L.pararnn_chunked_workspace_size.argtypes = [ctypes.POINTER(Cell), ci, ci, ci, ci]
        L.pararnn_chunked_workspace_size.restype = sz
        L.pararnn_lstm_solve.argtypes = [ctypes.POINTER(Cell), ctypes.POINTER(Params), vp, vp, vp, ci, ci, cf, ci,
                                         vp, vp, ctypes.POINTER(Info), vp, sz, vp]
        L.pararnn_lstm_solve.restype = ci
        L.pararnn_lstm_workspace_size.argtypes = [ctypes.POINTER(Cell), ci, ci]
        L.pararnn_lstm_workspace_size.restype = sz
        L.pararnn_newton_solve_reuse.argtypes = [ctypes.POINTER(Cell), ctypes.POINTER(Params), vp, vp, ci, ci, ci,
                                                 cf, ci, vp, ctypes.POINTER(Info), vp, sz, vp]
        L.pararnn_newton_solve_reuse.restype = ci
        L.pararnn_reuse_workspace_size.argtypes = [ctypes.POINTER(Cell), ci, ci]
        L.pararnn_reuse_workspace_size.restype = sz
        L.pararnn_lstm_solve_host.argtypes = [ctypes.POINTER(Cell), ctypes.POINTER(Params), vp, vp, vp, ci, ci, cf, ci,
                                              vp, vp, ctypes.POINTER(Info), ci, vp, sz, vp]
        L.pararnn_lstm_solve_host.restype = ci
        L.pararnn_lstm_host_workspace_size.argtypes = [ctypes.POINTER(Cell), ci, ci, ci]
        L.pararnn_lstm_host_workspace_size.restype = sz
        L.pararnn_lstm_solve_host_streamed.argtypes = L.pararnn_lstm_solve_host.argtypes
        L.pararnn_lstm_solve_host_streamed.restype = ci
        L.pararnn_lstm_host_streamed_workspace_size.argtypes = [ctypes.POINTER(Cell), ci, ci, ci]
        L.pararnn_lstm_host_streamed_workspace_size.restype = sz
        L.pararnn_adjoint_host.argtypes = [ctypes.POINTER(Cell), ctypes.POINTER(Params), vp, vp, vp, vp, ci, ci,
                                           vp, vp, vp, vp, ci, vp, sz, vp]
        L.pararnn_adjoint_host.restype = ci
        L.pararnn_adjoint_host_workspace_size.argtypes = [ctypes.POINTER(Cell), ci, ci, ci]
        L.pararnn_adjoint_host_workspace_size.restype = sz
        L.pararnn_newton_solve_trace.argtypes = [ctypes.POINTER(Cell), ctypes.POINTER(Params), vp, vp, ci, ci, ci,
                                                 cf, cf, ci, vp, ctypes.POINTER(Info), vp, ci, vp, sz, vp]
        L.pararnn_newton_solve_trace.restype = ci
        L.pararnn_test_withheld_publish.argtypes = [ctypes.POINTER(Cell), ctypes.POINTER(Params), vp, vp, ci, ci,
                                                    ci, cf, vp, ctypes.POINTER(Info), ctypes.c_longlong, vp, sz, vp]
        L.pararnn_test_withheld_publish.restype = ci
        L.pararnn_adjoint_exact.argtypes = [ctypes.POINTER(Cell), ctypes.POINTER(Params), vp, vp, vp, vp, ci, ci,
                                            vp, vp, vp, vp, vp, sz, vp]
        L.pararnn_adjoint_exact.restype = ci
        L.pararnn_adjoint_exact_workspace_size.argtypes = [ctypes.POINTER(Cell), ci, ci]
        L.pararnn_adjoint_exact_workspace_size.restype = sz
        shape_p, rows_p, norm_p = ctypes.POINTER(AttentionShape), ctypes.POINTER(Rows), ctypes.POINTER(NormShape)
        L.pararnn_linear_attention_workspace_size.argtypes = [shape_p, rows_p, rows_p, rows_p]
        L.pararnn_linear_attention_workspace_size.restype = sz
        L.pararnn_linear_attention_backward_workspace_size.argtypes = [shape_p, rows_p, rows_p, rows_p, rows_p]
        L.pararnn_linear_attention_backward_workspace_size.restype = sz
        L.pararnn_linear_attention.argtypes = [shape_p, rows_p, rows_p, rows_p, vp, vp, vp, vp, vp, vp, sz, vp]
        L.pararnn_linear_attention.restype = ci
        L.pararnn_linear_attention_backward.argtypes = [shape_p, rows_p, rows_p, rows_p, vp, rows_p, vp, vp, vp, vp, vp,
                                                        vp, vp, vp, sz, vp]
        L.pararnn_linear_attention_backward.restype = ci
        L.pararnn_linear_attention_step.argtypes = [shape_p, rows_p, rows_p, rows_p, vp, vp, vp, ci, vp, vp, vp]
        L.pararnn_linear_attention_step.restype = ci
        for name in ("pararnn_group_norm_workspace_size", "pararnn_group_norm_backward_workspace_size"):
            getattr(L, name).argtypes = [norm_p]
            getattr(L, name).restype = sz
        L.pararnn_group_norm.argtypes = [norm_p, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.pararnn_group_norm.restype = ci
        L.pararnn_group_norm_backward.argtypes = [norm_p, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.pararnn_group_norm_backward.restype = ci
        L.pararnn_status_string.argtypes = [ci]
        L.pararnn_status_string.restype = ctypes.c_char_p
        _lib = L
    return _lib


def _dtype_code(t: torch.dtype) -> int:
    if t == torch.float32:
        return F32
    if t == torch.bfloat16:
        return BF16
    raise TypeError(f"unsupported dtype {t}")


def _dev(t: torch.Tensor, name: str) -> int:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _stream(stream) -> int:
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def make_cell(kind: str, din: int, d: int, dtype: torch.dtype) -> Cell:
    code = {"dense": GRU_DENSE, "diag": GRU_DIAG, "lstm_diag": LSTM_DIAG}[kind]
    return Cell(code, din, d, _dtype_code(dtype), _dtype_code(dtype))


def lstm_workspace_size(din: int, d: int, B: int, T: int, dtype: torch.dtype = torch.float32) -> int:
    cell = make_cell("lstm_diag", din, d, dtype)
    return int(lib().pararnn_lstm_workspace_size(ctypes.byref(cell), B, T))


def lstm_solve(w_ih, b_ih, u, b_hh, x, c0, h0, *, tol: float, max_iters: int = 0, out=None, workspace=None,
               stream=None):
    """Evaluate the diagonal-recurrence LSTM over x [B, T, Din] by exact Newton.
    Weights: w_ih [4D, Din] (x's dtype), b_ih, u, b_hh [4D] fp32; c0, h0 [B, D].
    Returns (c, h, SolveResult) with c, h [B, T, D] fp32 CUDA tensors."""
    B, T, din = x.shape
    d = h0.shape[1]
    cell = make_cell("lstm_diag", din, d, x.dtype)
    L = lib()
    need = int(L.pararnn_lstm_workspace_size(ctypes.byref(cell), B, T))
    if need == 0:
        raise ValueError("arguments rejected by pararnn_lstm_workspace_size")
    if workspace is None:
        workspace = alloc_workspace(need, x.device)
    c, h = out if out is not None else (torch.empty(B, T, d, dtype=torch.float32, device=x.device),
                                        torch.empty(B, T, d, dtype=torch.float32, device=x.device))
    params = Params(_dev(w_ih, "w_ih"), _dev(b_ih, "b_ih"), _dev(u, "u"), _dev(b_hh, "b_hh"))
    info = Info()
    rc = L.pararnn_lstm_solve(ctypes.byref(cell), ctypes.byref(params), _dev(x, "x"), _dev(c0, "c0"), _dev(h0, "h0"),
                              B, T, float(tol), int(max_iters), _dev(c, "c"), _dev(h, "h"), ctypes.byref(info),
                              _dev(workspace, "workspace"), workspace.numel(), _stream(stream))
    if rc in (3, 4):
        raise RuntimeError(f"pararnn_lstm_solve: {L.pararnn_status_string(rc).decode()}")
    return c, h, SolveResult(h, info.iters, STATUS[info.status], info.delta, info.residual)


def workspace_size(kind: str, din: int, d: int, B: int, T: int, mode: str,
                   dtype: torch.dtype = torch.float32) -> int:
    cell = make_cell(kind, din, d, dtype)
    return int(lib().pararnn_workspace_size(ctypes.byref(cell), B, T, MODES[mode]))


def alloc_workspace(nbytes: int, device=None) -> torch.Tensor:
    """A 256-byte aligned device buffer of at least ``nbytes`` bytes."""
    buf = torch.empty(nbytes + 256, dtype=torch.uint8, device=device or "cuda")
    off = (-buf.data_ptr()) % 256
    return buf[off:off + nbytes]


@dataclass
class SolveResult:
    h: torch.Tensor
    iters: int
    status: str
    delta: float
    residual: float
    trace: object = None  # [iters, 2] host tensor: max |dh| and max |r| per iteration (trace=True)


def newton_solve(w_ih, b_ih, w_hh, b_hh, x, h0, *, kind: str, mode: str, tol: float,
                 lam: float = 0.0, max_iters: int = 0, out=None, workspace=None,
                 stream=None, sync: bool = True, info_dev=None, h_init=None, jac_every: int = 1,
                 trace: bool = False):
    """Evaluate the GRU over x [B, T, Din] with the chosen Newton mode.

    All tensors must be contiguous CUDA tensors (x and w_ih fp32 or bf16, the
    rest fp32).  With ``sync`` the call waits and returns a SolveResult; with
    ``sync=False`` it only enqueues, writing the report into ``info_dev`` (an
    int32 CUDA tensor of 4 elements) and returns ``out``.  ``h_init`` [B, T, D]
    (fp32 CUDA) starts the iteration from that guess instead of zero.
    ``jac_every`` > 1 (mode DEER, dense cell, d <= 32) recomputes the Jacobian
    only every jac_every iterations (synchronous; no h_init).  ``trace`` (sync
    only) also returns every iteration's max |dh| and max |r| (SolveResult.trace)."""
    B, T, din = x.shape
    d = h0.shape[1]
    cell = make_cell(kind, din, d, x.dtype)
    if w_ih.dtype != x.dtype:
        raise TypeError("x and w_ih must have the same dtype")
    L = lib()
    if jac_every != 1:
        if mode != "DEER" or h_init is not None or not sync:
            raise ValueError("jac_every > 1 takes mode DEER, sync=True and no h_init")
        need = int(L.pararnn_reuse_workspace_size(ctypes.byref(cell), B, T))
        if need == 0:
            raise ValueError("arguments rejected by pararnn_reuse_workspace_size")
        if workspace is None:
            workspace = alloc_workspace(need, x.device)
        if out is None:
            out = torch.empty(B, T, d, dtype=torch.float32, device=x.device)
        params = Params(_dev(w_ih, "w_ih"), _dev(b_ih, "b_ih"), _dev(w_hh, "w_hh"), _dev(b_hh, "b_hh"))
        info = Info()
        rc = L.pararnn_newton_solve_reuse(ctypes.byref(cell), ctypes.byref(params), _dev(x, "x"), _dev(h0, "h0"),
                                          B, T, int(jac_every), float(tol), int(max_iters), _dev(out, "out"),
                                          ctypes.byref(info), _dev(workspace, "workspace"), workspace.numel(),
                                          _stream(stream))
        if rc in (3, 4):
            raise RuntimeError(f"pararnn_newton_solve_reuse: {L.pararnn_status_string(rc).decode()}")
        return SolveResult(out, info.iters, STATUS[info.status], info.delta, info.residual)
    m = MODES[mode]
    need = int(L.pararnn_workspace_size(ctypes.byref(cell), B, T, m))
    if need == 0:
        raise ValueError("arguments rejected by pararnn_workspace_size")
    if workspace is None:
        workspace = alloc_workspace(need, x.device)
    if out is None:
        out = torch.empty(B, T, d, dtype=torch.float32, device=x.device)
    params = Params(_dev(w_ih, "w_ih"), _dev(b_ih, "b_ih"), _dev(w_hh, "w_hh"), _dev(b_hh, "b_hh"))
    args = (ctypes.byref(cell), ctypes.byref(params), _dev(x, "x"), _dev(h0, "h0"), B, T, m,
            float(lam), float(tol), int(max_iters), _dev(out, "out"))
    if h_init is not None:
        own = info_dev is None
        if own:
            info_dev = torch.zeros(4, dtype=torch.int32, device=x.device)
        rc = L.pararnn_newton_solve_guess_async(ctypes.byref(cell), ctypes.byref(params), _dev(x, "x"),
                                                _dev(h0, "h0"), _dev(h_init, "h_init"), B, T, m, float(lam),
                                                float(tol), int(max_iters), _dev(out, "out"),
                                                _dev(info_dev, "info_dev"), _dev(workspace, "workspace"),
                                                workspace.numel(), _stream(stream))
        if rc != 0:
            raise RuntimeError(f"pararnn_newton_solve_guess_async: {L.pararnn_status_string(rc).decode()}")
        if not sync:
            return out
        rep = info_dev.cpu()  # waits for the solve
        return SolveResult(out, int(rep[0]), STATUS[int(rep[1])], float(rep[2:3].view(torch.float32)),
                           float(rep[3:4].view(torch.float32)))
    if sync and trace:
        cap = int(max_iters) if max_iters > 0 else T + 1
        tr = torch.full((cap, 2), float("nan"), dtype=torch.float32, device=x.device)
        info = Info()
        rc = L.pararnn_newton_solve_trace(*args, ctypes.byref(info), _dev(tr, "trace"), cap,
                                          _dev(workspace, "workspace"), workspace.numel(), _stream(stream))
        if rc in (3, 4):
            raise RuntimeError(f"pararnn_newton_solve_trace: {L.pararnn_status_string(rc).decode()}")
        return SolveResult(out, info.iters, STATUS[info.status], info.delta, info.residual,
                           tr[:info.iters].cpu())
    if sync:
        info = Info()
        rc = L.pararnn_newton_solve(*args, ctypes.byref(info), _dev(workspace, "workspace"),
                                    workspace.numel(), _stream(stream))
        if rc in (3, 4):
            raise RuntimeError(f"pararnn_newton_solve: {L.pararnn_status_string(rc).decode()}")
        return SolveResult(out, info.iters, STATUS[info.status], info.delta, info.residual)
    if info_dev is None:
        raise ValueError("sync=False needs info_dev (int32 CUDA tensor with 4 elements)")
    rc = L.pararnn_newton_solve_async(*args, _dev(info_dev, "info_dev"),
                                      _dev(workspace, "workspace"), workspace.numel(),
                                      _stream(stream))
    if rc != 0:
        raise RuntimeError(f"pararnn_newton_solve_async: {L.pararnn_status_string(rc).decode()}")
    return out


def _host(t: torch.Tensor, name: str) -> int:
    if t.is_cuda:
        raise ValueError(f"{name} must be a host tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def newton_solve_chunked(w_ih, b_ih, w_hh, b_hh, x, h0, *, kind: str, mode: str, tol: float, t_chunk: int,
                         lam: float = 0.0, max_iters: int = 0, out=None, workspace=None,
                         stream=None) -> "SolveResult":
    """The solve over consecutive time chunks of at most ``t_chunk`` steps (device
    memory grows with t_chunk, not T); the report sums iterations over chunks."""
    B, T, din = x.shape
    d = h0.shape[1]
    cell = make_cell(kind, din, d, x.dtype)
    L = lib()
    m = MODES[mode]
    need = int(L.pararnn_chunked_workspace_size(ctypes.byref(cell), B, T, int(t_chunk), m))
    if need == 0:
        raise ValueError("arguments rejected by pararnn_chunked_workspace_size")
    if workspace is None:
        workspace = alloc_workspace(need, x.device)
    if out is None:
        out = torch.empty(B, T, d, dtype=torch.float32, device=x.device)
    params = Params(_dev(w_ih, "w_ih"), _dev(b_ih, "b_ih"), _dev(w_hh, "w_hh"), _dev(b_hh, "b_hh"))
    info = Info()
    rc = L.pararnn_newton_solve_chunked(ctypes.byref(cell), ctypes.byref(params), _dev(x, "x"), _dev(h0, "h0"),
                                        B, T, int(t_chunk), m, float(lam), float(tol), int(max_iters),
                                        _dev(out, "out"), ctypes.byref(info), _dev(workspace, "workspace"),
                                        workspace.numel(), _stream(stream))
    if rc in (3, 4):
        raise RuntimeError(f"pararnn_newton_solve_chunked: {L.pararnn_status_string(rc).decode()}")
    return SolveResult(out, info.iters, STATUS[info.status], info.delta, info.residual)


def chunked_workspace_size(kind: str, din: int, d: int, B: int, T: int, t_chunk: int, mode: str,
                           dtype: torch.dtype = torch.float32) -> int:
    cell = make_cell(kind, din, d, dtype)
    return int(lib().pararnn_chunked_workspace_size(ctypes.byref(cell), B, T, int(t_chunk), MODES[mode]))


def host_workspace_size(kind: str, din: int, d: int, B: int, T: int, mode: str, parts: int,
                        dtype: torch.dtype = torch.float32) -> int:
    cell = make_cell(kind, din, d, dtype)
    return int(lib().pararnn_host_workspace_size(ctypes.byref(cell), B, T, MODES[mode], parts))


def newton_solve_host(w_ih, b_ih, w_hh, b_hh, x_host, h0_host, *, kind: str, mode: str, tol: float,
                      lam: float = 0.0, max_iters: int = 0, parts: int = 4, out=None,
                      workspace=None, device=None, stream=None) -> "SolveResult":
    """The solve from and to HOST tensors (x_host [B,T,Din], h0_host [B,D];
    ``out`` a host [B,T,D] fp32 tensor, page-locked for overlap).  The batch is
    solved in ``parts`` parts with copies overlapped with compute; weights are
    CUDA tensors.  Returns a SolveResult whose h is the host tensor and whose
    report is the worst part's."""
    B, T, din = x_host.shape
    d = h0_host.shape[1]
    parts = max(1, min(int(parts), B))
    cell = make_cell(kind, din, d, x_host.dtype)
    L = lib()
    m = MODES[mode]
    need = int(L.pararnn_host_workspace_size(ctypes.byref(cell), B, T, m, parts))
    if need == 0:
        raise ValueError("arguments rejected by pararnn_host_workspace_size")
    if workspace is None:
        workspace = alloc_workspace(need, w_hh.device if device is None else device)
    if out is None:
        out = torch.empty(B, T, d, dtype=torch.float32).pin_memory()
    params = Params(_dev(w_ih, "w_ih"), _dev(b_ih, "b_ih"), _dev(w_hh, "w_hh"), _dev(b_hh, "b_hh"))
    info = Info()
    rc = L.pararnn_newton_solve_host(ctypes.byref(cell), ctypes.byref(params), _host(x_host, "x_host"),
                                     _host(h0_host, "h0_host"), B, T, m, float(lam), float(tol),
                                     int(max_iters), _host(out, "out"), ctypes.byref(info), parts,
                                     _dev(workspace, "workspace"), workspace.numel(), _stream(stream))
    if rc in (3, 4):
        raise RuntimeError(f"pararnn_newton_solve_host: {L.pararnn_status_string(rc).decode()}")
    return SolveResult(out, info.iters, STATUS[info.status], info.delta, info.residual)


def host_streamed_workspace_size(kind: str, din: int, d: int, B: int, T: int, mode: str, parts: int,
                                 dtype: torch.dtype = torch.float32) -> int:
    cell = make_cell(kind, din, d, dtype)
    return int(lib().pararnn_host_streamed_workspace_size(ctypes.byref(cell), B, T, MODES[mode], parts))


def newton_solve_host_streamed(w_ih, b_ih, w_hh, b_hh, x_host, h0_host, *, kind: str, mode: str, tol: float,
                               lam: float = 0.0, max_iters: int = 0, parts: int = 7, out=None,
                               workspace=None, device=None, stream=None) -> "SolveResult":
    """The solve from and to HOST tensors with the sequence streamed through
    the device in ``parts`` time parts (whole batch in each; clamped to
    1 .. ceil(T / 128)), each part solved from the previous part's last states
    while the next part's inputs are copied in and the previous part's states
    out.  The report sums iterations over the parts."""
    B, T, din = x_host.shape
    d = h0_host.shape[1]
    parts = max(1, min(int(parts), (T + 127) // 128))
    cell = make_cell(kind, din, d, x_host.dtype)
    L = lib()
    m = MODES[mode]
    need = int(L.pararnn_host_streamed_workspace_size(ctypes.byref(cell), B, T, m, parts))
    if need == 0:
        raise ValueError("arguments rejected by pararnn_host_streamed_workspace_size")
    if workspace is None:
        workspace = alloc_workspace(need, w_hh.device if device is None else device)
    if out is None:
        out = torch.empty(B, T, d, dtype=torch.float32).pin_memory()
    params = Params(_dev(w_ih, "w_ih"), _dev(b_ih, "b_ih"), _dev(w_hh, "w_hh"), _dev(b_hh, "b_hh"))
    info = Info()
    rc = L.pararnn_newton_solve_host_streamed(ctypes.byref(cell), ctypes.byref(params), _host(x_host, "x_host"),
                                              _host(h0_host, "h0_host"), B, T, m, float(lam), float(tol),
                                              int(max_iters), _host(out, "out"), ctypes.byref(info), parts,
                                              _dev(workspace, "workspace"), workspace.numel(), _stream(stream))
    if rc in (3, 4):
        raise RuntimeError(f"pararnn_newton_solve_host_streamed: {L.pararnn_status_string(rc).decode()}")
    return SolveResult(out, info.iters, STATUS[info.status], info.delta, info.residual)


def lstm_solve_host(w_ih, b_ih, u, b_hh, x_host, c0_host, h0_host, *, tol: float, max_iters: int = 0,
                    parts: int = 4, out=None, workspace=None, device=None, stream=None):
    """The LSTM solve from and to HOST tensors (x_host [B,T,Din], c0_host and
    h0_host [B,D]; ``out`` a pair of host [B,T,D] fp32 tensors, page-locked for
    overlap), in ``parts`` parts with the copies overlapped with compute;
    weights are CUDA tensors.  Returns (c, h, SolveResult) with host c, h."""
    B, T, din = x_host.shape
    d = h0_host.shape[1]
    parts = max(1, min(int(parts), B))
    cell = make_cell("lstm_diag", din, d, x_host.dtype)
    L = lib()
    need = int(L.pararnn_lstm_host_workspace_size(ctypes.byref(cell), B, T, parts))
    if need == 0:
        raise ValueError("arguments rejected by pararnn_lstm_host_workspace_size")
    if workspace is None:
        workspace = alloc_workspace(need, u.device if device is None else device)
    c, h = out if out is not None else (torch.empty(B, T, d, dtype=torch.float32).pin_memory(),
                                        torch.empty(B, T, d, dtype=torch.float32).pin_memory())
    params = Params(_dev(w_ih, "w_ih"), _dev(b_ih, "b_ih"), _dev(u, "u"), _dev(b_hh, "b_hh"))
    info = Info()
    rc = L.pararnn_lstm_solve_host(ctypes.byref(cell), ctypes.byref(params), _host(x_host, "x_host"),
                                   _host(c0_host, "c0_host"), _host(h0_host, "h0_host"), B, T, float(tol),
                                   int(max_iters), _host(c, "c"), _host(h, "h"), ctypes.byref(info), parts,
                                   _dev(workspace, "workspace"), workspace.numel(), _stream(stream))
    if rc in (3, 4):
        raise RuntimeError(f"pararnn_lstm_solve_host: {L.pararnn_status_string(rc).decode()}")
    return c, h, SolveResult(h, info.iters, STATUS[info.status], info.delta, info.residual)


def lstm_solve_host_streamed(w_ih, b_ih, u, b_hh, x_host, c0_host, h0_host, *, tol: float, max_iters: int = 0,
                             parts: int = 7, out=None, workspace=None, device=None, stream=None):
    """The LSTM solve from and to HOST tensors with the sequence streamed
    through the device in ``parts`` time parts (clamped to 1 .. ceil(T / 128));
    the report sums iterations over the parts.  Returns (c, h, SolveResult)."""
    B, T, din = x_host.shape
    d = h0_host.shape[1]
    parts = max(1, min(int(parts), (T + 127) // 128))
    cell = make_cell("lstm_diag", din, d, x_host.dtype)
    L = lib()
    need = int(L.pararnn_lstm_host_streamed_workspace_size(ctypes.byref(cell), B, T, parts))
    if need == 0:
        raise ValueError("arguments rejected by pararnn_lstm_host_streamed_workspace_size")
    if workspace is None:
        workspace = alloc_workspace(need, u.device if device is None else device)
    c, h = out if out is not None else (torch.empty(B, T, d, dtype=torch.float32).pin_memory(),
                                        torch.empty(B, T, d, dtype=torch.float32).pin_memory())
    params = Params(_dev(w_ih, "w_ih"), _dev(b_ih, "b_ih"), _dev(u, "u"), _dev(b_hh, "b_hh"))
    info = Info()
    rc = L.pararnn_lstm_solve_host_streamed(ctypes.byref(cell), ctypes.byref(params), _host(x_host, "x_host"),
                                            _host(c0_host, "c0_host"), _host(h0_host, "h0_host"), B, T, float(tol),
                                            int(max_iters), _host(c, "c"), _host(h, "h"), ctypes.byref(info), parts,
                                            _dev(workspace, "workspace"), workspace.numel(), _stream(stream))
    if rc in (3, 4):
        raise RuntimeError(f"pararnn_lstm_solve_host_streamed: {L.pararnn_status_string(rc).decode()}")
    return c, h, SolveResult(h, info.iters, STATUS[info.status], info.delta, info.residual)


def lstm_host_streamed_workspace_size(din: int, d: int, B: int, T: int, parts: int,
                                      dtype: torch.dtype = torch.bfloat16) -> int:
    cell = make_cell("lstm_diag", din, d, dtype)
    return int(lib().pararnn_lstm_host_streamed_workspace_size(ctypes.byref(cell), B, T, parts))


def adjoint_workspace_size(d: int, B: int, T: int, kind: str = "diag") -> int:
    cell = make_cell(kind, 1, d, torch.float32)
    return int(lib().pararnn_adjoint_workspace_size(ctypes.byref(cell), B, T))


def adjoint_exact(w_hh, b_hh, P, h0, h, dh, *, workspace=None, out=None, stream=None) -> dict:
    """The exact backward pass of the dense GRU (full transposed Jacobian):
    w_hh [3D, D], b_hh [3D], P [B,T,3D], h0 [B,D], h and dh [B,T,D], all fp32
    CUDA.  Returns dict(dP, dh0, dw_hh, db_hh)."""
    B, T, d = h.shape
    cell = make_cell("dense", 1, d, torch.float32)
    L = lib()
    need = int(L.pararnn_adjoint_exact_workspace_size(ctypes.byref(cell), B, T))
    if need == 0:
        raise ValueError("arguments rejected by pararnn_adjoint_exact_workspace_size")
    if workspace is None:
        workspace = alloc_workspace(need, h.device)
    o = out or {}
    dP = o["dP"] if "dP" in o else torch.empty_like(P)
    dh0 = o["dh0"] if "dh0" in o else torch.empty_like(h0)
    dw = o["dw_hh"] if "dw_hh" in o else torch.empty_like(w_hh)
    db = o["db_hh"] if "db_hh" in o else torch.empty_like(b_hh)
    params = Params(None, None, _dev(w_hh, "w_hh"), _dev(b_hh, "b_hh"))
    rc = L.pararnn_adjoint_exact(ctypes.byref(cell), ctypes.byref(params), _dev(P, "P"), _dev(h0, "h0"),
                                 _dev(h, "h"), _dev(dh, "dh"), B, T, _dev(dP, "dP"), _dev(dh0, "dh0"),
                                 _dev(dw, "dw_hh"), _dev(db, "db_hh"), _dev(workspace, "workspace"),
                                 workspace.numel(), _stream(stream))
    if rc != 0:
        raise RuntimeError(f"pararnn_adjoint_exact: {L.pararnn_status_string(rc).decode()}")
    return dict(dP=dP, dh0=dh0, dw_hh=dw, db_hh=db)


def adjoint(w_hh, b_hh, P, h0, h, dh, *, workspace=None, out=None, stream=None, check: bool = False) -> dict:
    """Backward pass of the GRU through the states h: gradients w.r.t. the
    pre-activations P [B,T,3D], h0 [B,D], w_hh and b_hh [3D], given
    dh = dL/dh [B,T,D] (all fp32 CUDA).  w_hh [3D] is the diagonal cell (exact
    gradients); w_hh [3D, D] the dense cell, whose adjoint runs with the
    Jacobian's diagonal (D <= 64).  Returns dict(dP, dh0, dw_hh, db_hh)."""
    B, T, d = h.shape
    cell = make_cell("dense" if w_hh.dim() == 2 else "diag", 1, d, torch.float32)
    L = lib()
    need = int(L.pararnn_adjoint_workspace_size(ctypes.byref(cell), B, T))
    if need == 0:
        raise ValueError("arguments rejected by pararnn_adjoint_workspace_size")
    if workspace is None:
        workspace = alloc_workspace(need, h.device)
    o = out or {}
    dP = o["dP"] if "dP" in o else torch.empty_like(P)
    dh0 = o["dh0"] if "dh0" in o else torch.empty_like(h0)
    dw = o["dw_hh"] if "dw_hh" in o else torch.empty_like(w_hh)
    db = o["db_hh"] if "db_hh" in o else torch.empty_like(b_hh)
    params = Params(None, None, _dev(w_hh, "w_hh"), _dev(b_hh, "b_hh"))
    rc = L.pararnn_adjoint(ctypes.byref(cell), ctypes.byref(params), _dev(P, "P"), _dev(h0, "h0"), _dev(h, "h"),
                           _dev(dh, "dh"), B, T, _dev(dP, "dP"), _dev(dh0, "dh0"), _dev(dw, "dw_hh"),
                           _dev(db, "db_hh"), _dev(workspace, "workspace"), workspace.numel(), _stream(stream))
    if rc != 0:
        raise RuntimeError(f"pararnn_adjoint: {L.pararnn_status_string(rc).decode()}")
    if check:
        st = L.pararnn_adjoint_status(_dev(workspace, "workspace"), _stream(stream))
        if st != 0:
            raise RuntimeError(f"pararnn_adjoint: {STATUS.get(st, st)}")
    return dict(dP=dP, dh0=dh0, dw_hh=dw, db_hh=db)


def adjoint_host(w_hh, b_hh, P_host, h0_host, h_host, dh_host, *, parts: int = 4, out=None, workspace=None,
                 stream=None) -> dict:
    """The backward pass from and to HOST tensors (P_host [B,T,3D], h0_host
    [B,D], h_host and dh_host [B,T,D], page-locked for overlap), in ``parts``
    parts with the copies overlapped with compute; w_hh, b_hh CUDA tensors
    (w_hh [3D]: diagonal cell, [3D, D]: dense cell).  Returns dict(dP, dh0,
    dw_hh, db_hh) of host tensors."""
    B, T, d = h_host.shape
    parts = max(1, min(int(parts), B))
    cell = make_cell("dense" if w_hh.dim() == 2 else "diag", 1, d, torch.float32)
    L = lib()
    need = int(L.pararnn_adjoint_host_workspace_size(ctypes.byref(cell), B, T, parts))
    if need == 0:
        raise ValueError("arguments rejected by pararnn_adjoint_host_workspace_size")
    if workspace is None:
        workspace = alloc_workspace(need, w_hh.device)
    o = out or {}
    pinned = lambda key, shape: o[key] if key in o else torch.empty(shape, dtype=torch.float32).pin_memory()
    dP = pinned("dP", P_host.shape)
    dh0 = pinned("dh0", h0_host.shape)
    dw = pinned("dw_hh", w_hh.shape)
    db = pinned("db_hh", b_hh.shape)
    params = Params(None, None, _dev(w_hh, "w_hh"), _dev(b_hh, "b_hh"))
    rc = L.pararnn_adjoint_host(ctypes.byref(cell), ctypes.byref(params), _host(P_host, "P_host"),
                                _host(h0_host, "h0_host"), _host(h_host, "h_host"), _host(dh_host, "dh_host"), B, T,
                                _host(dP, "dP"), _host(dh0, "dh0"), _host(dw, "dw_hh"), _host(db, "db_hh"), parts,
                                _dev(workspace, "workspace"), workspace.numel(), _stream(stream))
    if rc != 0:
        raise RuntimeError(f"pararnn_adjoint_host: {L.pararnn_status_string(rc).decode()}")
    return dict(dP=dP, dh0=dh0, dw_hh=dw, db_hh=db)


def input_projection(x, w_ih, b_ih, *, d: int, kind: str = "dense", out=None, stream=None):
    """P = x W_ih^T + b_ih for every step: x [B,T,Din] -> P [B,T,3D] fp32."""
    B, T, din = x.shape
    cell = make_cell(kind, din, d, x.dtype)
    if out is None:
        out = torch.empty(B, T, 3 * d, dtype=torch.float32, device=x.device)
    params = Params(_dev(w_ih, "w_ih"), _dev(b_ih, "b_ih"), 0, 0)
    rc = lib().pararnn_input_projection(ctypes.byref(cell), ctypes.byref(params), _dev(x, "x"),
                                        B, T, _dev(out, "out"), _stream(stream))
    if rc != 0:
        raise RuntimeError(f"pararnn_input_projection: {STATUS.get(rc, rc)}")
    return out


def newton_iterate(P, w_hh, b_hh, h0, *, kind: str, din: int, mode: str, tol: float,
                   info_dev, lam: float = 0.0, max_iters: int = 0, out=None, workspace=None,
                   dtype=torch.float32, stream=None):
    """Enqueue the Newton loop on precomputed P [B,T,3D]; report into info_dev."""
    B, T, _ = P.shape
    d = h0.shape[1]
    cell = make_cell(kind, din, d, dtype)
    L = lib()
    m = MODES[mode]
    if workspace is None:
        workspace = alloc_workspace(int(L.pararnn_workspace_size(ctypes.byref(cell), B, T, m)),
                                    P.device)
    if out is None:
        out = torch.empty(B, T, d, dtype=torch.float32, device=P.device)
    params = Params(0, 0, _dev(w_hh, "w_hh"), _dev(b_hh, "b_hh"))
    rc = L.pararnn_newton_iterate_async(ctypes.byref(cell), ctypes.byref(params), _dev(P, "P"),
                                        _dev(h0, "h0"), B, T, m, float(lam), float(tol),
                                        int(max_iters), _dev(out, "out"), _dev(info_dev, "info"),
                                        _dev(workspace, "workspace"), workspace.numel(),
                                        _stream(stream))
    if rc != 0:
        raise RuntimeError(f"pararnn_newton_iterate_async: {STATUS.get(rc, rc)}")
    return out


def solve_workload(w, mode: str, *, lam: float = 0.0, tol=None, max_iters: int = 0,
                   device="cuda", **kw) -> SolveResult:
    """Move a ``inputs.Workload`` to the device and solve it."""
    dev = lambda t: t.to(device).contiguous()
    return newton_solve(dev(w.w_ih), dev(w.b_ih), dev(w.w_hh), dev(w.b_hh), dev(w.x), dev(w.h0),
                        kind=w.kind, mode=mode, tol=w.tol if tol is None else tol, lam=lam,
                        max_iters=max_iters, **kw)


def withheld_publish(w, mode: str, tile: int, *, out=None, workspace=None, device="cuda",
                     stream=None) -> SolveResult:
    """The testing hook pararnn_test_withheld_publish on a ``inputs.Workload``:
    the solve with look-back tile ``tile`` silent in the first iteration."""
    dev = lambda t: t.to(device).contiguous()
    x, h0 = dev(w.x), dev(w.h0)
    B, T, din = x.shape
    d = h0.shape[1]
    cell = make_cell(w.kind, din, d, x.dtype)
    L = lib()
    m = MODES[mode]
    need = int(L.pararnn_workspace_size(ctypes.byref(cell), B, T, m))
    if workspace is None:
        workspace = alloc_workspace(need, x.device)
    if out is None:
        out = torch.empty(B, T, d, dtype=torch.float32, device=x.device)
    w_ih, b_ih, w_hh, b_hh = dev(w.w_ih), dev(w.b_ih), dev(w.w_hh), dev(w.b_hh)
    params = Params(_dev(w_ih, "w_ih"), _dev(b_ih, "b_ih"), _dev(w_hh, "w_hh"), _dev(b_hh, "b_hh"))
    info = Info()
    rc = L.pararnn_test_withheld_publish(ctypes.byref(cell), ctypes.byref(params), _dev(x, "x"), _dev(h0, "h0"),
                                         B, T, m, float(w.tol), _dev(out, "out"), ctypes.byref(info), int(tile),
                                         _dev(workspace, "workspace"), workspace.numel(), _stream(stream))
    if rc in (3, 4):
        raise RuntimeError(f"pararnn_test_withheld_publish: {L.pararnn_status_string(rc).decode()}")
    return SolveResult(out, info.iters, STATUS[info.status], info.delta, info.residual)


def affine_scan(A, b, h0, *, out=None, workspace=None, stream=None, check: bool = False):
    """h_t = A_t h_{t-1} + b_t over t for every sequence.  A is [B,T,D]
    (diagonal) or [B,T,D,D] (dense); b [B,T,D]; h0 [B,D]; all fp32 CUDA."""
    B, T, D = b.shape
    dense = 1 if A.dim() == 4 else 0
    L = lib()
    need = int(L.pararnn_affine_scan_workspace_size(B, T, D, dense))
    if need == 0:
        raise ValueError("arguments rejected by pararnn_affine_scan_workspace_size")
    if workspace is None:
        workspace = alloc_workspace(need, b.device)
    if out is None:
        out = torch.empty_like(b)
    rc = L.pararnn_affine_scan(_dev(A, "A"), _dev(b, "b"), _dev(h0, "h0"), B, T, D, dense,
                               _dev(out, "out"), _dev(workspace, "workspace"), workspace.numel(),
                               _stream(stream))
    if rc != 0:
        raise RuntimeError(f"pararnn_affine_scan: {L.pararnn_status_string(rc).decode()}")
    if check:
        st = L.pararnn_affine_scan_status(_dev(workspace, "workspace"), _stream(stream))
        if st != 0:
            raise RuntimeError(f"pararnn_affine_scan: {STATUS.get(st, st)}")
    return out


def affine_scan_host(A_host, b_host, h0_host, *, parts: int = 7, out=None, workspace=None, device=None,
                     stream=None):
    """The affine scan from and to HOST tensors (A [B,T,D] or [B,T,D,D], b
    [B,T,D], h0 [B,D], fp32; page-locked for overlap), streamed through the
    device in ``parts`` time parts (clamped to 1 .. ceil(T / 128)), each part
    started from the previous part's last states.  Returns the host h."""
    B, T, D = b_host.shape
    dense = 1 if A_host.dim() == 4 else 0
    parts = max(1, min(int(parts), (T + 127) // 128))
    L = lib()
    need = int(L.pararnn_affine_scan_host_workspace_size(B, T, D, dense, parts))
    if need == 0:
        raise ValueError("arguments rejected by pararnn_affine_scan_host_workspace_size")
    if workspace is None:
        workspace = alloc_workspace(need, device or "cuda")
    if out is None:
        out = torch.empty(B, T, D, dtype=torch.float32).pin_memory()
    rc = L.pararnn_affine_scan_host(_host(A_host, "A_host"), _host(b_host, "b_host"), _host(h0_host, "h0_host"),
                                    B, T, D, dense, _host(out, "out"), parts, _dev(workspace, "workspace"),
                                    workspace.numel(), _stream(stream))
    if rc != 0:
        raise RuntimeError(f"pararnn_affine_scan_host: {L.pararnn_status_string(rc).decode()}")
    return out


# ---- sequence layers: linear attention with a decay for each head, group norm -------------------------------


def _context(t, stream):
    """What a call on ``t`` has to be made under: the caller's stream, so that the call's own allocations belong to it,
    or t's device where another one is current; None where neither applies."""
    if stream is not None:
        if stream.device != t.device:
            raise ValueError(f"stream must be one of {t.device}, got one of {stream.device}")
        return torch.cuda.stream(stream)
    if t.is_cuda and t.get_device() != torch.cuda.current_device():
        return torch.cuda.device(t.get_device())
    return None


def _current(t) -> int:
    """The current stream of t's device, as a cudaStream_t."""
    return torch._C._cuda_getCurrentRawStream(t.get_device())


def _refuse(t, name: str, like, shape, dtype):
    if t.get_device() != like.get_device():
        raise ValueError(f"{name} must be on {like.device}, got {t.device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous{'' if t.is_contiguous() else ' along its last axis'}")


def _like(t, name: str, like, shape, dtype):
    """The address of a dense tensor of this shape and type on like's device, None for None; else raises."""
    if t is None:
        return None
    if t.dtype != dtype or t.shape != shape or t.get_device() != like.get_device() or not t.is_contiguous():
        _refuse(t, name, like, shape, dtype)
    return t.data_ptr()


def _rows(t, name: str, like, shape):
    """A [B, T, heads, width] operand (or [B, heads, width]) of like's type, strided in all but the last axis."""
    st = t.stride()
    if (t.dtype != like.dtype or t.shape != shape or t.get_device() != like.get_device()
            or (st[-1] != 1 and shape[-1] != 1)):
        _refuse(t, name, like, shape, like.dtype)
    return Rows(t.data_ptr(), st[0], st[1] if len(st) == 4 else 0, st[-2])


_INT = 2 ** 31  # the C ABI counts in int


def _no_graph(name: str):
    """These calls record no graph, so a gradient through them would be lost without a word: it is refused."""
    raise ValueError(f"{name} records no graph for an operand that requires a gradient: call it under torch.no_grad(); "
                     "gradients come from the backward calls")


def _attention_shape(q, k, v, log_decay, scale, dims: int = 4, back: bool = False):
    if q.dim() != dims or k.dim() != dims or v.dim() != dims:
        raise ValueError("q, k and v must be " + ("[B, T, heads, width]" if dims == 4 else "[B, heads, width]"))
    lead = q.shape[:-2]
    B, T = lead[0], lead[1] if dims == 4 else 1
    (H, dk), Hkv, dv = q.shape[-2:], k.shape[-2], v.shape[-1]
    if not (0 < B < _INT and 0 < T < _INT and 0 < H < _INT and 0 < Hkv) or H % Hkv:
        if max(B, T, H) >= _INT:
            raise ValueError(f"B, T and the head counts must be below 2**31: got {B}, {T} and {H}")
        raise ValueError(f"B, T and the head counts must be positive, q's heads a multiple of k's: {H} and {Hkv}")
    if not (1 <= dk <= 128 and 1 <= dv <= 128):
        raise ValueError(f"head widths must be 1 to 128: got {dk} and {dv}")
    if log_decay.requires_grad and (back or torch.is_grad_enabled()):
        raise ValueError("log_decay is a constant of the model: it gets no gradient")
    shape = AttentionShape(B, T, H, Hkv, dk, dv, _dtype_code(q.dtype), dk ** -0.5 if scale is None else scale)
    if not q.is_cuda:
        raise ValueError("q must be a CUDA tensor")
    return (shape, _rows(q, "q", q, (*lead, H, dk)), _rows(k, "k", q, (*lead, Hkv, dk)),
            _rows(v, "v", q, (*lead, Hkv, dv)))


def _workspace(need: int, name: str, workspace, device):
    """(tensor, address, bytes) of a call's workspace; none is allocated where none is needed."""
    if need == 0:
        raise ValueError(f"arguments rejected by {name}_workspace_size")
    if workspace is None:
        if need == 1:
            return None, None, 0
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
        if workspace.data_ptr() % 256:
            workspace = alloc_workspace(need, device)
    elif workspace.device != device:
        raise ValueError(f"workspace must be on {device}, got {workspace.device}")
    return workspace, _dev(workspace, "workspace"), workspace.numel()


def _checked(rc: int, name: str):
    if rc != 0:
        raise RuntimeError(f"{name}: {lib().pararnn_status_string(rc).decode()}")


def linear_attention(q, k, v, log_decay, *, s0=None, lengths=None, scale=None, out=None, workspace=None, stream=None):
    """Linear attention with a decay for each head over whole sequences:
    S_t = exp(log_decay) S_(t-1) + k_t v_t^T, o_t = scale * S_t^T q_t.

    q [B,T,H,dk], k [B,T,Hkv,dk], v [B,T,Hkv,dv] (fp32 or bf16 CUDA; views with
    any strides whose last axis is contiguous; Hkv divides H), log_decay [H]
    fp32 <= 0, s0 [B,H,dk,dv] fp32 the state before (zero if None), lengths [B]
    int32 (tokens behind them are not read, outputs there are zero), scale
    dk**-0.5 if None.  Returns (o [B,T,H,dv] of q's type, the last state
    [B,H,dk,dv] fp32); ``out`` gives both tensors (the state's may be s0).
    Records no graph: operands that require a gradient are taken under
    ``torch.no_grad()`` only, and ``linear_attention_backward`` has the gradients."""
    under = _context(q, stream)
    if under is not None:
        with under:
            return linear_attention(q, k, v, log_decay, s0=s0, lengths=lengths, scale=scale, out=out, workspace=workspace)
    if torch.is_grad_enabled() and (q.requires_grad or k.requires_grad or v.requires_grad
                                    or (s0 is not None and s0.requires_grad)):
        _no_graph("linear_attention")
    shape, rq, rk, rv = _attention_shape(q, k, v, log_decay, scale)
    B, T, H, dk, dv = shape.B, shape.T, shape.H, shape.dk, shape.dv
    o, s = out if out is not None else (q.new_empty((B, T, H, dv)), log_decay.new_empty((B, H, dk, dv)))
    L = lib()
    ws, ws_at, ws_bytes = _workspace(L.pararnn_linear_attention_workspace_size(shape, rq, rk, rv), "pararnn_linear_attention",
                                       workspace, q.device)
    _checked(L.pararnn_linear_attention(
        shape, rq, rk, rv, _like(log_decay, "log_decay", q, (H,), torch.float32),
        _like(s0, "s0", q, (B, H, dk, dv), torch.float32), _like(lengths, "lengths", q, (B,), torch.int32),
        _like(o, "out", q, (B, T, H, dv), q.dtype), _like(s, "out", q, (B, H, dk, dv), torch.float32),
        ws_at, ws_bytes, _current(q)), "pararnn_linear_attention")
    return o, s


def linear_attention_backward(q, k, v, log_decay, do, *, s0=None, ds=None, lengths=None, scale=None, workspace=None,
                              stream=None) -> dict:
    """The backward pass of ``linear_attention``: do [B,T,H,dv] = dL/do (q's
    type, strided as q), ds [B,H,dk,dv] fp32 the gradient of the last state
    (zero if None); the rest as given to the forward pass.  Returns dict(dq,
    dk, dv, ds0) of q's type (ds0 fp32, None without s0)."""
    under = _context(q, stream)
    if under is not None:
        with under:
            return linear_attention_backward(q, k, v, log_decay, do, s0=s0, ds=ds, lengths=lengths, scale=scale,
                                             workspace=workspace)
    shape, rq, rk, rv = _attention_shape(q, k, v, log_decay, scale, back=True)
    B, T, H, Hkv, dk, dv = shape.B, shape.T, shape.H, shape.Hkv, shape.dk, shape.dv
    rdo = _rows(do, "do", q, (B, T, H, dv))
    g = dict(dq=q.new_empty((B, T, H, dk)), dk=q.new_empty((B, T, Hkv, dk)), dv=q.new_empty((B, T, Hkv, dv)),
             ds0=None if s0 is None else s0.new_empty((B, H, dk, dv)))
    L = lib()
    ws, ws_at, ws_bytes = _workspace(L.pararnn_linear_attention_backward_workspace_size(shape, rq, rk, rv, rdo),
                                       "pararnn_linear_attention_backward", workspace, q.device)
    state = (B, H, dk, dv)
    _checked(L.pararnn_linear_attention_backward(
        shape, rq, rk, rv, _like(log_decay, "log_decay", q, (H,), torch.float32), rdo,
        _like(s0, "s0", q, state, torch.float32), _like(ds, "ds", q, state, torch.float32),
        _like(lengths, "lengths", q, (B,), torch.int32), g["dq"].data_ptr(), g["dk"].data_ptr(), g["dv"].data_ptr(),
        None if s0 is None else g["ds0"].data_ptr(), ws_at, ws_bytes, _current(q)),
        "pararnn_linear_attention_backward")
    return g


def linear_attention_step(q, k, v, log_decay, state, *, slots=None, scale=None, out_state=None, out=None, stream=None):
    """One token of every sequence: S = exp(log_decay) S + k v^T, o = scale S^T q.

    q [B,H,dk], k [B,Hkv,dk], v [B,Hkv,dv] as for ``linear_attention`` without
    the time axis; state [n,H,dk,dv] fp32 holds the states, row b's at slots[b]
    (int32 [B]; outside 0..n-1: no state, o is zero; the same slot twice: tokens
    in row order), or at b if None (n = B).  The states after the token go to
    ``out_state``, or replace those in ``state`` if None.  Returns o [B,H,dv].
    Records no graph, as ``linear_attention``."""
    under = _context(q, stream)
    if under is not None:
        with under:
            return linear_attention_step(q, k, v, log_decay, state, slots=slots, scale=scale, out_state=out_state, out=out)
    if torch.is_grad_enabled() and (q.requires_grad or k.requires_grad or v.requires_grad or state.requires_grad):
        _no_graph("linear_attention_step")
    if state.dim() != 4 or state.shape[0] < 1:
        raise ValueError("state must be [n, H, dk, dv]")
    n = state.shape[0]
    if n >= _INT:
        raise ValueError(f"states must be below 2**31: got {n}")
    shape, rq, rk, rv = _attention_shape(q, k, v, log_decay, scale, 3)
    B, H, dk, dv = shape.B, shape.H, shape.dk, shape.dv
    if slots is None and n != B:
        raise ValueError(f"state has {n} rows for {B} sequences: slots says which")
    if out is None:
        out = q.new_empty((B, H, dv))
    pool = (n, H, dk, dv)
    src = _like(state, "state", q, pool, torch.float32)
    _checked(lib().pararnn_linear_attention_step(
        shape, rq, rk, rv, _like(log_decay, "log_decay", q, (H,), torch.float32), src,
        _like(slots, "slots", q, (B,), torch.int32), n, _like(out, "out", q, (B, H, dv), q.dtype),
        src if out_state is None else _like(out_state, "out_state", q, pool, torch.float32), _current(q)),
        "pararnn_linear_attention_step")
    return out


def _norm_shape(x, groups, act, eps, y_dtype):
    if x.dim() < 2:
        raise ValueError("x must be [N, ..., C]")
    if act not in ACTIVATIONS:
        raise ValueError(f"act must be one of {sorted(ACTIVATIONS)}")
    N, C = x.shape[0], x.shape[-1]
    S = 1
    for n in x.shape[1:-1]:
        S *= n
    if min(N, S, C) < 1 or not 1 <= groups <= 2048 or C % groups:
        raise ValueError(f"x must not be empty and groups (1 to 2048) must divide its channels: {tuple(x.shape)}, {groups}")
    if max(N, S, C) >= _INT:
        raise ValueError(f"x's first, middle and last axes must be below 2**31: got {N}, {S} and {C}")
    return NormShape(N, S, C, groups, _dtype_code(x.dtype), _dtype_code(y_dtype), ACTIVATIONS[act], eps)


def group_norm(x, groups: int, weight=None, bias=None, *, gate=None, act: str = "silu", eps: float = 1e-5, lengths=None,
               out_dtype=None, out=None, workspace=None, stream=None):
    """Group norm, channels last: x [N, ..., C] is normalised over the rows
    between the first and the last axis and each group's channels, for every n;
    z = xhat * weight + bias, y = act(z), or z * act(gate) with a gate of x's
    shape and type.  [N, C] normalises each row's groups by themselves.

    x fp32 or bf16, contiguous CUDA; weight, bias [C] fp32; act "none", "silu" or
    "gelu"; lengths [N] int32: rows behind them (in the middle axes' order) are
    not read, do not count, and are zero in y.  Returns (y of ``out_dtype``, x's
    if None; stats [N, groups, 2] fp32: mean and 1 / sqrt(var + eps)).  Records
    no graph: operands that require a gradient are taken under ``torch.no_grad()``
    only, and ``group_norm_backward`` has the gradients."""
    under = _context(x, stream)
    if under is not None:
        with under:
            return group_norm(x, groups, weight, bias, gate=gate, act=act, eps=eps, lengths=lengths, out_dtype=out_dtype,
                              out=out, workspace=workspace)
    if torch.is_grad_enabled() and (x.requires_grad or (weight is not None and weight.requires_grad)
                                    or (bias is not None and bias.requires_grad)
                                    or (gate is not None and gate.requires_grad)):
        _no_graph("group_norm")
    y_dtype = out.dtype if out is not None else x.dtype if out_dtype is None else out_dtype
    shape = _norm_shape(x, groups, act, eps, y_dtype)
    channels = (shape.C,)
    y = out if out is not None else torch.empty(x.shape, dtype=y_dtype, device=x.device)
    stats = torch.empty(shape.N, groups, 2, dtype=torch.float32, device=x.device)
    L = lib()
    ws, ws_at, ws_bytes = _workspace(L.pararnn_group_norm_workspace_size(shape), "pararnn_group_norm", workspace, x.device)
    _checked(L.pararnn_group_norm(
        shape, _dev(x, "x"), _like(weight, "weight", x, channels, torch.float32),
        _like(bias, "bias", x, channels, torch.float32), _like(gate, "gate", x, x.shape, x.dtype),
        _like(lengths, "lengths", x, (shape.N,), torch.int32), _like(y, "out", x, x.shape, y_dtype), stats.data_ptr(),
        ws_at, ws_bytes, _current(x)), "pararnn_group_norm")
    return y, stats


def group_norm_backward(x, stats, dy, groups: int, weight=None, bias=None, *, gate=None, act: str = "silu",
                        lengths=None, workspace=None, stream=None) -> dict:
    """The backward pass of ``group_norm`` from dy [N, ..., C] = dL/dy (y's
    type) and the forward's stats; the rest as given to the forward pass.
    Returns dict(dx, dweight, dbias, dgate); dweight, dbias and dgate are None
    where the forward pass had no weight, bias or gate."""
    under = _context(x, stream)
    if under is not None:
        with under:
            return group_norm_backward(x, stats, dy, groups, weight, bias, gate=gate, act=act, lengths=lengths,
                                       workspace=workspace)
    shape = _norm_shape(x, groups, act, 0.0, dy.dtype)
    channels = (shape.C,)
    new = lambda t: None if t is None else torch.empty_like(t)
    ptr = lambda t: None if t is None else t.data_ptr()
    px = _dev(x, "x")
    pw = _like(weight, "weight", x, channels, torch.float32)
    pb = _like(bias, "bias", x, channels, torch.float32)
    pg = _like(gate, "gate", x, x.shape, x.dtype)
    g = dict(dx=torch.empty_like(x), dweight=new(weight), dbias=new(bias), dgate=new(gate))
    L = lib()
    ws, ws_at, ws_bytes = _workspace(L.pararnn_group_norm_backward_workspace_size(shape), "pararnn_group_norm_backward",
                                       workspace, x.device)
    _checked(L.pararnn_group_norm_backward(
        shape, px, _like(stats, "stats", x, (shape.N, groups, 2), torch.float32), _like(dy, "dy", x, x.shape, dy.dtype),
        pw, pb, pg, _like(lengths, "lengths", x, (shape.N,), torch.int32), ptr(g["dx"]), ptr(g["dweight"]),
        ptr(g["dbias"]), ptr(g["dgate"]), ws_at, ws_bytes, _current(x)), "pararnn_group_norm_backward")
    return g
