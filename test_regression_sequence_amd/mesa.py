"""Python binding of libmesa (ctypes).  Argument marshalling only.

Every step of the layer runs in the HIP library; this module passes device
pointers of torch tensors and the current HIP stream through the C ABI
declared in ``include/mesa.h``, and allocates outputs with torch.  There is no
fallback: if the library is missing, every call raises ``MesaError``.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

__all__ = [
    "MesaError", "lib", "library_path", "FwdDesc", "MESA_F32", "MESA_BF16",
    "workspace_bytes", "fwd_chunked", "fwd_chunked_noalloc", "fwd_chunked_prep", "fwd_scan", "fwd_solve", "decode_step", "abi_version",
    "status_string", "sym_state_floats", "sym_pack", "sym_unpack", "decode_step_symh",
    "lru_workspace_bytes", "lru_fwd", "lru_bwd", "lru_step",
    "rmsnorm", "rmsnorm_bwd", "rmsnorm_bwd_workspace_bytes",
    "qk_preprocess_bwd", "qk_preprocess_bwd_workspace_bytes",
    "delta_workspace_bytes", "delta_fwd", "delta_bwd", "delta_step", "grad_norm", "grad_clip",
]

MESA_F32 = 0
MESA_BF16 = 1
STATUS = {0: "MESA_OK", 1: "MESA_ERR_INVALID_ARG", 2: "MESA_ERR_UNSUPPORTED",
          3: "MESA_ERR_ALIGNMENT", 4: "MESA_ERR_WORKSPACE", 5: "MESA_ERR_HIP"}

_LIB: Optional[ctypes.CDLL] = None


class MesaError(RuntimeError):
    def __init__(self, msg, status: int | None = None):
        super().__init__(msg)
        self.status = status


class FwdDesc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("H", ctypes.c_int32), ("T", ctypes.c_int32),
                ("dk", ctypes.c_int32), ("dv", ctypes.c_int32), ("chunk", ctypes.c_int32),
                ("max_steps", ctypes.c_int32), ("tol", ctypes.c_float), ("in_dtype", ctypes.c_int)]


class LruDesc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("T", ctypes.c_int32), ("D", ctypes.c_int32), ("ld", ctypes.c_int32),
                ("c", ctypes.c_float), ("dtype", ctypes.c_int)]


class Rows(ctypes.Structure):
    _fields_ = [("b", ctypes.c_int64), ("h", ctypes.c_int64), ("t", ctypes.c_int64)]


class DeltaDesc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("H", ctypes.c_int32), ("Hk", ctypes.c_int32), ("T", ctypes.c_int32),
                ("dk", ctypes.c_int32), ("dv", ctypes.c_int32), ("dtype", ctypes.c_int),
                ("q", Rows), ("k", Rows), ("v", Rows), ("o", Rows), ("gamma", Rows), ("beta", Rows)]


class DeltaGradRows(ctypes.Structure):
    _fields_ = [("d_o", Rows), ("dq", Rows), ("dk", Rows), ("dv", Rows), ("dgamma", Rows), ("dbeta", Rows)]


def library_path() -> str:
    return os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmesa.so")


def lib() -> ctypes.CDLL:
    global _LIB
    if _LIB is None:
        path = library_path()
        if not os.path.exists(path):
            raise MesaError(f"{path} is not built; run `python -m test_regression_sequence_amd.build`")
        L = ctypes.CDLL(path)
        P, S, I32, F = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32, ctypes.c_float
        L.mesa_abi_version.restype = I32
        L.mesa_abi_version.argtypes = []
        L.mesa_status_string.restype = ctypes.c_char_p
        L.mesa_status_string.argtypes = [ctypes.c_int]
        L.mesa_fwd_workspace_bytes.restype = S
        L.mesa_fwd_workspace_bytes.argtypes = [ctypes.POINTER(FwdDesc)]
        L.mesa_fwd_chunked.restype = ctypes.c_int
        L.mesa_fwd_chunked.argtypes = [ctypes.POINTER(FwdDesc), P, P, P, P, P, P, P, P, P, P, P, P, P,
                                       P, S, P]
        L.mesa_fwd_chunked_warm.restype = ctypes.c_int
        L.mesa_fwd_chunked_warm.argtypes = list(L.mesa_fwd_chunked.argtypes)
        L.mesa_fwd_chunked_noalloc.restype = ctypes.c_int
        L.mesa_fwd_chunked_noalloc.argtypes = [ctypes.POINTER(FwdDesc)] + [P] * 13 + [P]
        L.mesa_fwd_chunked_prep.restype = ctypes.c_int
        L.mesa_fwd_chunked_prep.argtypes = [ctypes.POINTER(FwdDesc), P, P, P, P, P, I32, F] + [P] * 15 + [S, P]
        L.mesa_fwd_chunked_ex.restype = ctypes.c_int
        L.mesa_fwd_chunked_ex.argtypes = [ctypes.POINTER(FwdDesc), P, P, P, P, P, P, I32, P, P, P, P, P, P,
                                          P, P, S, P]
        L.mesa_fwd_scan.restype = ctypes.c_int
        L.mesa_fwd_scan.argtypes = [ctypes.POINTER(FwdDesc), P, P, P, P, P, P, P, P, P, S, P]
        L.mesa_fwd_solve.restype = ctypes.c_int
        L.mesa_fwd_solve.argtypes = [ctypes.POINTER(FwdDesc), P, P, P, P, P, P, P, P, P, P, S, P]
        L.mesa_decode_step.restype = ctypes.c_int
        L.mesa_decode_step.argtypes = [I32, I32, I32, I32, P, P, P, ctypes.c_int, P, P, P, P, P, P,
                                       P, P, I32, F, P]
        L.mesa_decode_step_symh.restype = ctypes.c_int
        L.mesa_decode_step_symh.argtypes = list(L.mesa_decode_step.argtypes)
        L.mesa_decode_step_warm.restype = ctypes.c_int
        L.mesa_decode_step_warm.argtypes = [I32, I32, I32, I32, P, P, P, ctypes.c_int, P, P, P, P, I32,
                                            P, P, P, P, I32, F, P]
        L.mesa_decode_step_ex.restype = ctypes.c_int
        L.mesa_decode_step_ex.argtypes = [I32, I32, I32, I32, P, P, P, ctypes.c_int, P, P, P, I32, P, I32,
                                          P, P, P, P, P, I32, F, P]
        L.mesa_bwd_workspace_bytes.restype = S
        L.mesa_bwd_workspace_bytes.argtypes = [ctypes.POINTER(FwdDesc)]
        L.mesa_bwd_chunked.restype = ctypes.c_int
        L.mesa_bwd_chunked.argtypes = [ctypes.POINTER(FwdDesc)] + [P] * 21 + [I32, P, S, P]
        L.mesa_bwd_chunked_ex.restype = ctypes.c_int
        L.mesa_bwd_chunked_ex.argtypes = [ctypes.POINTER(FwdDesc)] + [P] * 6 + [I32] + [P] * 15 + [I32, P, S, P]
        L.mesa_qk_preprocess.restype = ctypes.c_int
        L.mesa_qk_preprocess.argtypes = [I32, I32, I32, I32, I32, ctypes.c_int, P, P, P, P, P, P, F,
                                         P, P, P, P, P]
        L.mesa_sym_state_floats.restype = S
        L.mesa_sym_state_floats.argtypes = [I32]
        L.mesa_sym_pack.restype = ctypes.c_int
        L.mesa_sym_pack.argtypes = [I32, I32, P, P, P]
        L.mesa_sym_unpack.restype = ctypes.c_int
        L.mesa_sym_unpack.argtypes = [I32, I32, P, P, P]
        D = ctypes.POINTER(LruDesc)
        L.mesa_lru_workspace_bytes.restype = S
        L.mesa_lru_workspace_bytes.argtypes = [D]
        L.mesa_lru_fwd.restype = ctypes.c_int
        L.mesa_lru_fwd.argtypes = [D] + [P] * 9 + [S, P]
        L.mesa_lru_bwd.restype = ctypes.c_int
        L.mesa_lru_bwd.argtypes = [D] + [P] * 11 + [I32, P, P, I32, P, S, P]
        L.mesa_lru_step.restype = ctypes.c_int
        L.mesa_lru_step.argtypes = [I32, I32, I32, F, ctypes.c_int] + [P] * 7
        L.mesa_rmsnorm.restype = ctypes.c_int
        L.mesa_rmsnorm.argtypes = [I32, I32, ctypes.c_int, ctypes.c_int, P, P, P, F, ctypes.c_int, I32, P, P, P, P]
        L.mesa_rmsnorm_bwd_workspace_bytes.restype = S
        L.mesa_rmsnorm_bwd_workspace_bytes.argtypes = [I32, I32]
        L.mesa_rmsnorm_bwd.restype = ctypes.c_int
        L.mesa_rmsnorm_bwd.argtypes = [I32, I32, ctypes.c_int, ctypes.c_int, P, P, P, P, F, P, P, P, P, S, P]
        L.mesa_qk_preprocess_bwd_workspace_bytes.restype = S
        L.mesa_qk_preprocess_bwd_workspace_bytes.argtypes = [I32, I32, I32, I32, I32, ctypes.c_int]
        L.mesa_qk_preprocess_bwd.restype = ctypes.c_int
        L.mesa_qk_preprocess_bwd.argtypes = ([I32, I32, I32, I32, I32, ctypes.c_int] + [P] * 6 + [F] + [P] * 11
                                             + [S, P])
        D = ctypes.POINTER(DeltaDesc)
        L.mesa_delta_workspace_bytes.restype = S
        L.mesa_delta_workspace_bytes.argtypes = [D, I32]
        L.mesa_delta_fwd.restype = ctypes.c_int
        L.mesa_delta_fwd.argtypes = [D] + [P] * 9 + [I32, P, S, P]
        L.mesa_delta_bwd.restype = ctypes.c_int
        L.mesa_delta_bwd.argtypes = [D, ctypes.POINTER(DeltaGradRows)] + [P] * 15 + [I32, P, S, P]
        L.mesa_delta_step.restype = ctypes.c_int
        L.mesa_delta_step.argtypes = [D] + [P] * 8
        L.mesa_grad_clip_workspace_bytes.restype = S
        L.mesa_grad_clip_workspace_bytes.argtypes = []
        L.mesa_grad_norm.restype = ctypes.c_int
        L.mesa_grad_norm.argtypes = [I32] + [P] * 5 + [S, P]
        L.mesa_grad_clip.restype = ctypes.c_int
        L.mesa_grad_clip.argtypes = [I32] + [P] * 4 + [ctypes.c_double] * 2 + [P] * 3 + [S, P]
        _LIB = L
    return _LIB


def abi_version() -> int:
    return int(lib().mesa_abi_version())


def status_string(code: int) -> str:
    return lib().mesa_status_string(int(code)).decode()


def _check(code: int, what: str):
    if code != 0:
        raise MesaError(f"{what}: {STATUS.get(code, code)} ({status_string(code)})", code)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return MESA_F32
    if t.dtype == torch.bfloat16:
        return MESA_BF16
    raise MesaError(f"q/k/v must be float32 or bfloat16, got {t.dtype}")


def _need(t: torch.Tensor, name: str, shape, dtype=None):
    if not t.is_cuda:
        raise MesaError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise MesaError(f"{name} must be contiguous")
    if tuple(t.shape) != tuple(shape):
        raise MesaError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if dtype is not None and t.dtype != dtype:
        raise MesaError(f"{name} must be {dtype}, got {t.dtype}")


def make_desc(B, H, T, d, chunk, max_steps, tol, dtype_code) -> FwdDesc:
    return FwdDesc(B, H, T, d, d, chunk, max_steps, float(tol), dtype_code)


def workspace_bytes(B, H, T, d, chunk, max_steps=0, tol=0.0, dtype=torch.bfloat16) -> int:
    code = MESA_BF16 if dtype == torch.bfloat16 else MESA_F32
    desc = make_desc(B, H, T, d, chunk, max_steps, tol, code)
    return int(lib().mesa_fwd_workspace_bytes(ctypes.byref(desc)))


def fwd_chunked(q, k, v, gamma, beta, lam, *, chunk: int = 64, max_steps: int = 30,
                tol: float = 0.0, h0=None, g0=None, return_state: bool = False,
                return_steps: bool = True, return_x: bool = False, out=None,
                workspace: Optional[torch.Tensor] = None, stream=None, warm: bool = False) -> dict:
    """Chunked Mesa forward; q, k, v [B, H, T, d] (fp32 or bf16) on the GPU.

    gamma, beta [B, H, T] fp32; lam [H, d] fp32; h0, g0 optional [B, H, d, d]
    fp32.  Returns a dict with ``o`` [B, H, T, d] fp32 and, on request,
    ``steps`` [B, H, T] int32, ``x`` [B, H, T, d], ``h_final``, ``g_final``.
    ``out`` may pass preallocated result tensors (same keys).  ``warm`` calls
    ``mesa_fwd_chunked_warm``: token t's CG starts from token t-16's solution
    when both lie in one chunk (bf16 inputs).
    """
    return _fwd("warm" if warm else False, q, k, v, gamma, beta, lam, chunk=chunk, max_steps=max_steps, tol=tol, h0=h0,
                g0=g0, return_state=return_state, return_steps=return_steps, return_x=return_x,
                out=out, workspace=workspace, stream=stream)


NOALLOC_SCRATCH_BYTES = 64 << 20  # MESA_NOALLOC_SCRATCH_BYTES


def fwd_chunked_noalloc(q, k, v, gamma, beta, lam, *, chunk: int = 64, max_steps: int = 30,
                        tol: float = 0.0, h0=None, g0=None, return_state: bool = False,
                        return_steps: bool = True, return_x: bool = False, out=None,
                        stream=None) -> dict:
    """``fwd_chunked`` through ``mesa_fwd_chunked_noalloc``: the library uses its
    static per-GPU scratch (at most ``NOALLOC_SCRATCH_BYTES`` of workspace) and
    allocates nothing; pass ``out`` to allocate nothing here either."""
    return _fwd("noalloc", q, k, v, gamma, beta, lam, chunk=chunk, max_steps=max_steps, tol=tol, h0=h0,
                g0=g0, return_state=return_state, return_steps=return_steps, return_x=return_x,
                out=out, workspace=None, stream=stream)


def fwd_chunked_prep(q_raw, k_raw, v, gamma, beta, lam, w_q, w_k, *, q_hist=None, k_hist=None,
                     eps: float = 1e-6, chunk: int = 64, max_steps: int = 30, tol: float = 0.0,
                     h0=None, g0=None, return_state: bool = False, return_steps: bool = True,
                     return_x: bool = False, return_history: bool = False, out=None,
                     workspace: Optional[torch.Tensor] = None, stream=None) -> dict:
    """``fwd_chunked`` on raw bf16 q, k [B, H, T, d] with ``qk_preprocess`` fused
    into the forward (``mesa_fwd_chunked_prep``): taps w_q, w_k [H, d, W], raw
    histories q_hist, k_hist [B, H, W-1, d] (None: zeros).  The result equals
    ``qk_preprocess`` followed by ``fwd_chunked`` bit for bit; with
    return_history it also holds the next call's histories ``q_hist``,
    ``k_hist``.  bf16 inputs, chunk 64, d in {64, 128}, W in 1..4."""
    B, H, T, d = q_raw.shape
    W = w_q.shape[-1]
    _need(w_q, "w_q", (H, d, W), torch.float32)
    _need(w_k, "w_k", (H, d, W), torch.float32)
    for name, t in (("q_hist", q_hist), ("k_hist", k_hist)):
        if t is not None:
            _need(t, name, (B, H, W - 1, d), q_raw.dtype)
    prep = {"w_q": w_q, "w_k": w_k, "W": W, "eps": eps, "q_hist": q_hist, "k_hist": k_hist,
            "return_history": return_history}
    return _fwd("prep", q_raw, k_raw, v, gamma, beta, lam, chunk=chunk, max_steps=max_steps, tol=tol, h0=h0,
                g0=g0, return_state=return_state, return_steps=return_steps, return_x=return_x,
                out=out, workspace=workspace, stream=stream, prep=prep)


def fwd_chunked_ex(q, k, v, gamma, beta, lam, *, chunk: int = 64, max_steps: int = 30,
                   tol: float = 0.0, h0=None, g0=None, return_state: bool = False,
                   return_steps: bool = True, return_x: bool = False, out=None,
                   workspace: Optional[torch.Tensor] = None, stream=None) -> dict:
    """``fwd_chunked`` with ``lam`` either the diagonal [H, d] or a full
    symmetric positive definite matrix per head [H, d, d] (fp32, row-major);
    the full form needs bf16 inputs, chunk 64 and d in {64, 128}."""
    return _fwd(True, q, k, v, gamma, beta, lam, chunk=chunk, max_steps=max_steps, tol=tol, h0=h0,
                g0=g0, return_state=return_state, return_steps=return_steps, return_x=return_x,
                out=out, workspace=workspace, stream=stream)


def _fwd(ex: bool, q, k, v, gamma, beta, lam, *, chunk, max_steps, tol, h0, g0, return_state,
         return_steps, return_x, out, workspace, stream, prep=None) -> dict:
    B, H, T, d = q.shape
    code = _dtype_code(q)
    for name, t in (("q", q), ("k", k), ("v", v)):
        _need(t, name, (B, H, T, d), q.dtype)
    _need(gamma, "gamma", (B, H, T), torch.float32)
    _need(beta, "beta", (B, H, T), torch.float32)
    noalloc = ex == "noalloc"
    lam_full = ex is True and lam.dim() == 3
    _need(lam, "lam", (H, d, d) if lam_full else (H, d), torch.float32)
    for name, t in (("h0", h0), ("g0", g0)):
        if t is not None:
            _need(t, name, (B, H, d, d), torch.float32)
    desc = make_desc(B, H, T, d, chunk, max_steps, tol, code)
    L = lib()
    need = int(L.mesa_fwd_workspace_bytes(ctypes.byref(desc)))
    dev = q.device
    out = dict(out or {})
    res = {}
    res["o"] = out.get("o") if out.get("o") is not None else torch.empty((B, H, T, d), device=dev, dtype=torch.float32)
    if return_steps:
        res["steps"] = out.get("steps") if out.get("steps") is not None else torch.empty((B, H, T), device=dev, dtype=torch.int32)
    if return_x:
        res["x"] = out.get("x") if out.get("x") is not None else torch.empty((B, H, T, d), device=dev, dtype=torch.float32)
    if return_state:
        res["h_final"] = out.get("h_final") if out.get("h_final") is not None else torch.empty((B, H, d, d), device=dev, dtype=torch.float32)
        res["g_final"] = out.get("g_final") if out.get("g_final") is not None else torch.empty((B, H, d, d), device=dev, dtype=torch.float32)
    if prep is not None and prep["return_history"]:
        for key in ("q_hist", "k_hist"):
            res[key] = out.get(key) if out.get(key) is not None else torch.empty((B, H, prep["W"] - 1, d), device=dev, dtype=q.dtype)
    if noalloc:
        code_ = L.mesa_fwd_chunked_noalloc(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(gamma), _ptr(beta),
                                           _ptr(lam), _ptr(h0), _ptr(g0), _ptr(res["o"]), _ptr(res.get("h_final")),
                                           _ptr(res.get("g_final")), _ptr(res.get("steps")), _ptr(res.get("x")),
                                           _stream(stream))
        _check(code_, "mesa_fwd_chunked_noalloc")
        return res
    if workspace is None and need > 0:
        workspace = torch.empty(need, device=dev, dtype=torch.uint8)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rest = (_ptr(h0), _ptr(g0), _ptr(res["o"]), _ptr(res.get("h_final")), _ptr(res.get("g_final")),
            _ptr(res.get("steps")), _ptr(res.get("x")), _ptr(workspace), ctypes.c_size_t(wbytes),
            _stream(stream))
    head = (ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(gamma), _ptr(beta), _ptr(lam))
    if ex == "prep":
        code_ = L.mesa_fwd_chunked_prep(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(prep["w_q"]),
                                        _ptr(prep["w_k"]), int(prep["W"]), float(prep["eps"]), _ptr(prep["q_hist"]),
                                        _ptr(prep["k_hist"]), _ptr(gamma), _ptr(beta), _ptr(lam), *rest[:7],
                                        _ptr(res.get("q_hist")), _ptr(res.get("k_hist")), *rest[7:])
        _check(code_, "mesa_fwd_chunked_prep")
    elif ex == "warm":
        code_ = L.mesa_fwd_chunked_warm(*head, *rest)
        _check(code_, "mesa_fwd_chunked_warm")
    elif ex:
        code_ = L.mesa_fwd_chunked_ex(*head, 1 if lam_full else 0, *rest)
        _check(code_, "mesa_fwd_chunked_ex")
    else:
        code_ = L.mesa_fwd_chunked(*head, *rest)
        _check(code_, "mesa_fwd_chunked")
    return res


def fwd_scan(k, v, gamma, beta, *, chunk: int, workspace: torch.Tensor, h0=None, g0=None,
             h_final=None, g_final=None, stream=None):
    """State scan only: boundary states into ``workspace``, optional final states."""
    B, H, T, d = k.shape
    desc = make_desc(B, H, T, d, chunk, 0, 0.0, _dtype_code(k))
    wbytes = workspace.numel() * workspace.element_size()
    code_ = lib().mesa_fwd_scan(ctypes.byref(desc), _ptr(k), _ptr(v), _ptr(gamma), _ptr(beta),
                                _ptr(h0), _ptr(g0), _ptr(h_final), _ptr(g_final), _ptr(workspace),
                                ctypes.c_size_t(wbytes), _stream(stream))
    _check(code_, "mesa_fwd_scan")


def fwd_solve(q, k, v, gamma, beta, lam, *, chunk: int, max_steps: int, tol: float,
              workspace: torch.Tensor, o: torch.Tensor, steps=None, x=None, stream=None):
    """CG solve + read-out only, from the boundary states a preceding fwd_scan left in ``workspace``."""
    B, H, T, d = q.shape
    desc = make_desc(B, H, T, d, chunk, max_steps, tol, _dtype_code(q))
    wbytes = workspace.numel() * workspace.element_size()
    code_ = lib().mesa_fwd_solve(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(gamma), _ptr(beta),
                                 _ptr(lam), _ptr(o), _ptr(steps), _ptr(x), _ptr(workspace),
                                 ctypes.c_size_t(wbytes), _stream(stream))
    _check(code_, "mesa_fwd_solve")


def sym_state_floats(d: int) -> int:
    """Floats of one H state in the blocked upper-triangular layout (d in {64, 128})."""
    n = int(lib().mesa_sym_state_floats(int(d)))
    if n == 0:
        raise MesaError(f"no packed layout for d={d}", 2)
    return n


def sym_pack(full: torch.Tensor, stream=None) -> torch.Tensor:
    """[..., d, d] fp32 symmetric states -> [..., sym_state_floats(d)] blocked upper triangle."""
    d = full.shape[-1]
    lead = full.shape[:-2]
    count = int(full.numel() // (d * d))
    _need(full, "full", tuple(lead) + (d, d), torch.float32)
    out = torch.empty(tuple(lead) + (sym_state_floats(d),), device=full.device, dtype=torch.float32)
    _check(lib().mesa_sym_pack(count, d, _ptr(full), _ptr(out), _stream(stream)), "mesa_sym_pack")
    return out


def sym_unpack(packed: torch.Tensor, d: int, stream=None) -> torch.Tensor:
    """[..., sym_state_floats(d)] -> [..., d, d] fp32 (lower blocks mirrored)."""
    n = sym_state_floats(d)
    lead = packed.shape[:-1]
    _need(packed, "packed", tuple(lead) + (n,), torch.float32)
    count = int(packed.numel() // n)
    out = torch.empty(tuple(lead) + (d, d), device=packed.device, dtype=torch.float32)
    _check(lib().mesa_sym_unpack(count, d, _ptr(packed), _ptr(out), _stream(stream)), "mesa_sym_unpack")
    return out


def decode_step_symh(q, k, v, gamma, beta, lam, h_sym, g_state, *, max_steps: int = 32,
                     tol: float = 1e-4, return_steps: bool = True, return_x: bool = False,
                     out=None, stream=None) -> dict:
    """decode_step with h_sym [N, H, sym_state_floats(d)] in the blocked layout (updated in place)."""
    return decode_step(q, k, v, gamma, beta, lam, h_sym, g_state, max_steps=max_steps, tol=tol,
                       return_steps=return_steps, return_x=return_x, out=out, stream=stream,
                       _symh=True)


def decode_step(q, k, v, gamma, beta, lam, h_state, g_state, *, max_steps: int = 32,
                tol: float = 1e-4, return_steps: bool = True, return_x: bool = False,
                out=None, stream=None, _symh: bool = False) -> dict:
    """One recurrent step; q, k, v [N, H, d]; h_state, g_state [N, H, d, d] fp32, updated in place."""
    N, H, d = q.shape
    code = _dtype_code(q)
    for name, t in (("q", q), ("k", k), ("v", v)):
        _need(t, name, (N, H, d), q.dtype)
    _need(gamma, "gamma", (N, H), torch.float32)
    _need(beta, "beta", (N, H), torch.float32)
    _need(lam, "lam", (H, d), torch.float32)
    if _symh:
        _need(h_state, "h_sym", (N, H, sym_state_floats(d)), torch.float32)
    else:
        _need(h_state, "h_state", (N, H, d, d), torch.float32)
    _need(g_state, "g_state", (N, H, d, d), torch.float32)
    dev = q.device
    out = dict(out or {})
    res = {"o": out.get("o") if out.get("o") is not None else torch.empty((N, H, d), device=dev, dtype=torch.float32)}
    if return_steps:
        res["steps"] = out.get("steps") if out.get("steps") is not None else torch.empty((N, H), device=dev, dtype=torch.int32)
    if return_x:
        res["x"] = out.get("x") if out.get("x") is not None else torch.empty((N, H, d), device=dev, dtype=torch.float32)
    fn = lib().mesa_decode_step_symh if _symh else lib().mesa_decode_step
    code_ = fn(N, H, d, d, _ptr(q), _ptr(k), _ptr(v), code, _ptr(gamma), _ptr(beta),
               _ptr(lam), _ptr(h_state), _ptr(g_state), _ptr(res["o"]),
               _ptr(res.get("steps")), _ptr(res.get("x")), int(max_steps),
               float(tol), _stream(stream))
    _check(code_, "mesa_decode_step_symh" if _symh else "mesa_decode_step")
    return res


def decode_step_warm(q, k, v, gamma, beta, lam, h_state, g_state, x_state, *, packed_h: bool = False,
                     max_steps: int = 32, tol: float = 1e-4, return_steps: bool = True,
                     out=None, stream=None) -> dict:
    """decode_step with CG started from x_state [N, H, d] fp32, which is overwritten
    with this token's solution (the next step's start).  h_state is [N, H, d, d], or
    [N, H, sym_state_floats(d)] in the blocked layout when packed_h."""
    N, H, d = q.shape
    code = _dtype_code(q)
    for name, t in (("q", q), ("k", k), ("v", v)):
        _need(t, name, (N, H, d), q.dtype)
    _need(gamma, "gamma", (N, H), torch.float32)
    _need(beta, "beta", (N, H), torch.float32)
    _need(lam, "lam", (H, d), torch.float32)
    if packed_h:
        _need(h_state, "h_sym", (N, H, sym_state_floats(d)), torch.float32)
    else:
        _need(h_state, "h_state", (N, H, d, d), torch.float32)
    _need(g_state, "g_state", (N, H, d, d), torch.float32)
    _need(x_state, "x_state", (N, H, d), torch.float32)
    dev = q.device
    out = dict(out or {})
    res = {"o": out.get("o") if out.get("o") is not None else torch.empty((N, H, d), device=dev, dtype=torch.float32)}
    if return_steps:
        res["steps"] = out.get("steps") if out.get("steps") is not None else torch.empty((N, H), device=dev, dtype=torch.int32)
    code_ = lib().mesa_decode_step_warm(N, H, d, d, _ptr(q), _ptr(k), _ptr(v), code, _ptr(gamma), _ptr(beta),
                                        _ptr(lam), _ptr(h_state), 1 if packed_h else 0, _ptr(g_state),
                                        _ptr(x_state), _ptr(res["o"]), _ptr(res.get("steps")),
                                        int(max_steps), float(tol), _stream(stream))
    _check(code_, "mesa_decode_step_warm")
    return res


def qk_preprocess(q_raw, k_raw, w_q, w_k, *, q_hist=None, k_hist=None, eps: float = 1e-6,
                  return_history: bool = False, out=None, stream=None) -> dict:
    """Causal depthwise convolution of raw q, k [B, H, T, d] along time with taps
    w_q, w_k [H, d, W], then L2 normalisation per token.  q_hist, k_hist
    [B, H, W-1, d]: raw vectors before t = 0 (None: zeros).  Returns q, k (and,
    with return_history, the next call's histories q_hist, k_hist)."""
    B, H, T, d = q_raw.shape
    W = w_q.shape[-1]
    code = _dtype_code(q_raw)
    _need(q_raw, "q_raw", (B, H, T, d), q_raw.dtype)
    _need(k_raw, "k_raw", (B, H, T, d), q_raw.dtype)
    _need(w_q, "w_q", (H, d, W), torch.float32)
    _need(w_k, "w_k", (H, d, W), torch.float32)
    for name, t in (("q_hist", q_hist), ("k_hist", k_hist)):
        if t is not None:
            _need(t, name, (B, H, W - 1, d), q_raw.dtype)
    out = dict(out or {})
    dev = q_raw.device
    res = {}
    for key in ("q", "k"):
        res[key] = out.get(key) if out.get(key) is not None else torch.empty((B, H, T, d), device=dev, dtype=q_raw.dtype)
    if return_history:
        for key in ("q_hist", "k_hist"):
            res[key] = out.get(key) if out.get(key) is not None else torch.empty((B, H, W - 1, d), device=dev, dtype=q_raw.dtype)
    code_ = lib().mesa_qk_preprocess(B, H, T, d, W, code, _ptr(q_raw), _ptr(k_raw), _ptr(w_q), _ptr(w_k),
                                     _ptr(q_hist), _ptr(k_hist), float(eps), _ptr(res["q"]), _ptr(res["k"]),
                                     _ptr(res.get("q_hist")), _ptr(res.get("k_hist")), _stream(stream))
    _check(code_, "mesa_qk_preprocess")
    return res


def bwd_workspace_bytes(B, H, T, d, chunk, max_steps, tol, dtype_code=1) -> int:
    """Bytes of the backward's workspace (also a valid forward workspace)."""
    desc = make_desc(B, H, T, d, chunk, max_steps, tol, dtype_code)
    return int(lib().mesa_bwd_workspace_bytes(ctypes.byref(desc)))


def bwd_chunked(q, k, v, gamma, beta, lam, x, d_o, *, chunk: int = 64, max_steps: int = 30,
                tol: float = 0.0, h0=None, g0=None, d_hfinal=None, d_gfinal=None,
                state_grads: bool = False, return_steps: bool = False, out=None,
                workspace: Optional[torch.Tensor] = None, states_in_workspace: bool = False,
                stream=None) -> dict:
    """Backward of fwd_chunked: x is the forward's solutions (its return_x output),
    d_o [B, H, T, d] fp32 the gradient at o.  Returns dq, dk, dv [B, H, T, d],
    dgamma, dbeta [B, H, T], dlam [H, d] (fp32) and, with state_grads, dh0, dg0.
    states_in_workspace: the forward ran with ``workspace`` (bwd_workspace_bytes
    long) and left its boundary states there, so they are not recomputed."""
    return _bwd(False, q, k, v, gamma, beta, lam, x, d_o, chunk=chunk, max_steps=max_steps, tol=tol, h0=h0,
                g0=g0, d_hfinal=d_hfinal, d_gfinal=d_gfinal, state_grads=state_grads,
                return_steps=return_steps, out=out, workspace=workspace,
                states_in_workspace=states_in_workspace, stream=stream)


def bwd_chunked_ex(q, k, v, gamma, beta, lam, x, d_o, *, chunk: int = 64, max_steps: int = 30,
                   tol: float = 0.0, h0=None, g0=None, d_hfinal=None, d_gfinal=None,
                   state_grads: bool = False, return_steps: bool = False, out=None,
                   workspace: Optional[torch.Tensor] = None, states_in_workspace: bool = False,
                   stream=None) -> dict:
    """``bwd_chunked`` with ``lam`` the diagonal [H, d] or a full symmetric positive
    definite matrix per head [H, d, d]; with the full form ``dlam`` is [H, d, d],
    the partial derivative of each entry (-sum_t y_t x_t^T)."""
    return _bwd(True, q, k, v, gamma, beta, lam, x, d_o, chunk=chunk, max_steps=max_steps, tol=tol, h0=h0,
                g0=g0, d_hfinal=d_hfinal, d_gfinal=d_gfinal, state_grads=state_grads,
                return_steps=return_steps, out=out, workspace=workspace,
                states_in_workspace=states_in_workspace, stream=stream)


def _bwd(ex: bool, q, k, v, gamma, beta, lam, x, d_o, *, chunk, max_steps, tol, h0, g0, d_hfinal, d_gfinal,
         state_grads, return_steps, out, workspace, states_in_workspace, stream) -> dict:
    B, H, T, d = q.shape
    code = _dtype_code(q)
    for name, t in (("q", q), ("k", k), ("v", v)):
        _need(t, name, (B, H, T, d), q.dtype)
    _need(gamma, "gamma", (B, H, T), torch.float32)
    _need(beta, "beta", (B, H, T), torch.float32)
    noalloc = ex == "noalloc"
    lam_full = ex is True and lam.dim() == 3
    _need(lam, "lam", (H, d, d) if lam_full else (H, d), torch.float32)
    for name, t in (("x", x), ("d_o", d_o)):
        _need(t, name, (B, H, T, d), torch.float32)
    for name, t in (("h0", h0), ("g0", g0), ("d_hfinal", d_hfinal), ("d_gfinal", d_gfinal)):
        if t is not None:
            _need(t, name, (B, H, d, d), torch.float32)
    desc = make_desc(B, H, T, d, chunk, max_steps, tol, code)
    L = lib()
    need = int(L.mesa_bwd_workspace_bytes(ctypes.byref(desc)))
    dev = q.device
    out = dict(out or {})
    f32 = torch.float32

    def get(key, shape, dtype=f32):
        return out.get(key) if out.get(key) is not None else torch.empty(shape, device=dev, dtype=dtype)

    res = {key: get(key, (B, H, T, d)) for key in ("dq", "dk", "dv")}
    res.update(dgamma=get("dgamma", (B, H, T)), dbeta=get("dbeta", (B, H, T)), dlam=get("dlam", (H, d, d) if lam_full else (H, d)))
    if state_grads:
        res.update(dh0=get("dh0", (B, H, d, d)), dg0=get("dg0", (B, H, d, d)))
    if return_steps:
        res["adj_steps"] = get("adj_steps", (B, H, T), torch.int32)
    if workspace is None:
        workspace = torch.empty(max(need, 1), device=dev, dtype=torch.uint8)
    wbytes = workspace.numel() * workspace.element_size()
    head = (ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(gamma), _ptr(beta), _ptr(lam))
    rest = (_ptr(h0), _ptr(g0), _ptr(x), _ptr(d_o), _ptr(d_hfinal), _ptr(d_gfinal),
            _ptr(res["dq"]), _ptr(res["dk"]), _ptr(res["dv"]), _ptr(res["dgamma"]),
            _ptr(res["dbeta"]), _ptr(res["dlam"]), _ptr(res.get("dh0")), _ptr(res.get("dg0")),
            _ptr(res.get("adj_steps")), 1 if states_in_workspace else 0, _ptr(workspace),
            ctypes.c_size_t(wbytes), _stream(stream))
    if ex:
        code_ = L.mesa_bwd_chunked_ex(*head, 1 if lam_full else 0, *rest)
        _check(code_, "mesa_bwd_chunked_ex")
    else:
        code_ = L.mesa_bwd_chunked(*head, *rest)
        _check(code_, "mesa_bwd_chunked")
    return res


def decode_step_ex(q, k, v, gamma, beta, lam, h_state, g_state, *, x_state=None, packed_h: bool = False,
                   max_steps: int = 32, tol: float = 1e-4, return_steps: bool = True, return_x: bool = False,
                   out=None, stream=None) -> dict:
    """The general decode step: lam [H, d] (diagonal) or [H, d, d] (full symmetric
    positive definite); h_state full or packed (packed_h); x_state [N, H, d] for a
    warm start (overwritten with the solution) or None for a cold start."""
    N, H, d = q.shape
    code = _dtype_code(q)
    for name, t in (("q", q), ("k", k), ("v", v)):
        _need(t, name, (N, H, d), q.dtype)
    _need(gamma, "gamma", (N, H), torch.float32)
    _need(beta, "beta", (N, H), torch.float32)
    full = lam.dim() == 3
    _need(lam, "lam", (H, d, d) if full else (H, d), torch.float32)
    _need(h_state, "h_state", (N, H, sym_state_floats(d)) if packed_h else (N, H, d, d), torch.float32)
    _need(g_state, "g_state", (N, H, d, d), torch.float32)
    if x_state is not None:
        _need(x_state, "x_state", (N, H, d), torch.float32)
    dev = q.device
    out = dict(out or {})
    res = {"o": out.get("o") if out.get("o") is not None else torch.empty((N, H, d), device=dev, dtype=torch.float32)}
    if return_steps:
        res["steps"] = out.get("steps") if out.get("steps") is not None else torch.empty((N, H), device=dev, dtype=torch.int32)
    if return_x and x_state is None:
        res["x"] = out.get("x") if out.get("x") is not None else torch.empty((N, H, d), device=dev, dtype=torch.float32)
    code_ = lib().mesa_decode_step_ex(N, H, d, d, _ptr(q), _ptr(k), _ptr(v), code, _ptr(gamma), _ptr(beta),
                                      _ptr(lam), 1 if full else 0, _ptr(h_state), 1 if packed_h else 0,
                                      _ptr(g_state), _ptr(x_state), _ptr(res["o"]), _ptr(res.get("steps")),
                                      _ptr(res.get("x")), int(max_steps), float(tol), _stream(stream))
    _check(code_, "mesa_decode_step_ex")
    return res


# ---- operators around the layer ------------------------------------------------
#
# Every tensor of a call has to be on one device, the first argument's, and a
# given stream too; the call is launched there whatever device is current.  What
# a call allocates belongs to the stream it runs on, so that its memory is given
# on in that stream's order.  Tensors passed as `out` and workspaces may not overlap
# inputs or one another but where a call says so.

def _addr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _code_of(t: torch.Tensor, name: str) -> int:
    if t.dtype is torch.bfloat16:
        return MESA_BF16
    if t.dtype is torch.float32:
        return MESA_F32
    raise MesaError(f"{name} must be float32 or bfloat16, got {t.dtype}")


def _want(t: Optional[torch.Tensor], name: str, shape, dtype, dev):
    """t (None passes) is a dense tensor of this shape and type on dev."""
    if t is None or (t.shape == shape and t.dtype is dtype and t.device == dev and t.is_contiguous()):
        return
    _need(t, name, shape, dtype)
    raise MesaError(f"{name} is on {t.device}, expected {dev}")


def _home(t: torch.Tensor, name: str, dims: int, stream) -> torch.device:
    """The device of a call's first argument, which has `dims` dimensions."""
    if not t.is_cuda:
        raise MesaError(f"{name} must be a device tensor")
    if t.dim() != dims:
        raise MesaError(f"{name} has shape {tuple(t.shape)}, expected {dims} dimensions")
    if stream is not None and stream.device != t.device:
        raise MesaError(f"the stream belongs to {stream.device}, {name} is on {t.device}")
    return t.device


def _new(shape, dtype, dev, stream, like=None) -> torch.Tensor:
    """like: a tensor of this shape and type (as its twin in half the time, where it is dense)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return torch.empty(shape, device=dev, dtype=dtype)
    if like is not None and like.is_contiguous():
        return torch.empty_like(like)
    return torch.empty(shape, device=dev, dtype=dtype)


def _result(out: Optional[dict], key: str, shape, dtype, dev, stream, like=None) -> torch.Tensor:
    """out[key], checked, or a new tensor."""
    t = out.get(key) if out else None
    if t is None:
        return _new(shape, dtype, dev, stream, like)
    _want(t, key, shape, dtype, dev)
    return t


def _scratch(workspace: Optional[torch.Tensor], need, dev, stream):
    """(a workspace of need() bytes, or the given one; its bytes)"""
    if workspace is None:
        workspace = _new(need(), torch.uint8, dev, stream)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise MesaError(f"workspace must be contiguous and on {dev}")
    return workspace, workspace.numel() * workspace.element_size()


def _launch(what: str, dev, stream, *args):
    """The library's function `what` on the stream (None: dev's current one)."""
    fn = getattr(lib(), what)
    handle = torch._C._cuda_getCurrentRawStream(dev.index) if stream is None else stream.cuda_stream
    if dev.index == torch.cuda.current_device():
        code = fn(*args, handle)
    else:
        with torch.cuda.device(dev):
            code = fn(*args, handle)
    if code:
        _check(code, what)


def _token_stride(named, shape, dtype, dev) -> int:
    """The common token stride of [..., D] tensors: dense, or equal slices of wider
    rows (last index contiguous, every leading index of the row-major order)."""
    ld = None
    for name, t in named:
        if t.shape != shape or t.dtype is not dtype or t.device != dev:
            if tuple(t.shape) != tuple(shape):
                raise MesaError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
            raise MesaError(f"{name} must be {dtype} on {dev}, got {t.dtype} on {t.device}")
        if t.is_contiguous():
            own = shape[-1]
        else:
            tokens = shape[-2]
            own = t.stride(-2) if tokens > 1 else t.stride(0) if t.dim() == 3 else shape[-1]
            if t.stride(-1) != 1 or own < shape[-1] or (t.dim() == 3 and shape[0] > 1 and t.stride(0) != own * tokens):
                raise MesaError(f"{name} has strides {tuple(t.stride())}: rows must be slices of one row-major tensor")
        if ld is not None and own != ld:
            raise MesaError(f"{name} has token stride {own}, expected {ld}")
        ld = own
    return ld


def lru_workspace_bytes(B, T, D, *, dtype=torch.bfloat16) -> int:
    """Scratch bytes of lru_fwd and lru_bwd at these sizes."""
    desc = LruDesc(B, T, D, D, 1.0, MESA_BF16 if dtype == torch.bfloat16 else MESA_F32)
    return lib().mesa_lru_workspace_bytes(ctypes.byref(desc))


def lru_fwd(x, ga, gi, lam, *, c: float = 8.0, h0=None, lengths=None, return_state: bool = False, out=None,
            workspace: Optional[torch.Tensor] = None, stream=None) -> dict:
    """Gated linear recurrence over whole sequences; x, ga, gi [B, T, D] (fp32 or
    bf16, D >= 2): dense, or equal slices of one wider row-major tensor.

    a_t = exp(-c softplus(lam) sigmoid(ga_t)), h_t = a_t h_{t-1} +
    sqrt(1 - a_t^2) sigmoid(gi_t) x_t.  lam [D] fp32; h0 [B, D] fp32 or None;
    lengths [B] int32 or None (valid tokens; outputs behind them are zeros).
    Returns a dict with ``y`` [B, T, D] in x's dtype and, with return_state,
    ``h_final`` [B, D] fp32 (out["h_final"] may be h0 itself).  ``workspace``
    (lru_workspace_bytes long) keeps the states that ``lru_bwd`` can take over."""
    dev, dt, f32 = _home(x, "x", 3, stream), x.dtype, torch.float32
    shape = x.shape
    B, T, D = shape
    code, ld = _code_of(x, "x"), _token_stride((("x", x), ("ga", ga), ("gi", gi)), shape, dt, dev)
    _want(lam, "lam", (D,), f32, dev)
    _want(h0, "h0", (B, D), f32, dev)
    _want(lengths, "lengths", (B,), torch.int32, dev)
    res = {"y": _result(out, "y", shape, dt, dev, stream, x)}
    if return_state:
        res["h_final"] = _result(out, "h_final", (B, D), f32, dev, stream)
    workspace, wbytes = _scratch(workspace, lambda: lru_workspace_bytes(B, T, D, dtype=dt), dev, stream)
    _launch("mesa_lru_fwd", dev, stream, ctypes.byref(LruDesc(B, T, D, ld, c, code)), _addr(x), _addr(ga), _addr(gi),
            _addr(lam), _addr(h0), _addr(lengths), _addr(res["y"]), _addr(res.get("h_final")), _addr(workspace), wbytes)
    return res


def lru_bwd(x, ga, gi, lam, dy, *, c: float = 8.0, h0=None, lengths=None, d_hfinal=None, state_grads: bool = False,
            out=None, workspace: Optional[torch.Tensor] = None, states_in_workspace: bool = False,
            stream=None) -> dict:
    """Gradients of lru_fwd: dy [B, T, D] in x's dtype, d_hfinal [B, D] fp32 or None.
    Returns ``dx``, ``dga``, ``dgi`` in x's dtype, ``dlam`` [D] fp32 and, with
    state_grads, ``dh0`` [B, D] fp32.  ``out`` may hold dx, dga and dgi as equal
    slices of one wider tensor, and d_hfinal itself as dh0.  states_in_workspace: the forward ran with
    ``workspace`` and left its states there, so they are not formed again."""
    if states_in_workspace and workspace is None:
        raise MesaError("states_in_workspace needs the forward's workspace")
    dev, dt, f32 = _home(x, "x", 3, stream), x.dtype, torch.float32
    shape = x.shape
    B, T, D = shape
    code, ld = _code_of(x, "x"), _token_stride((("x", x), ("ga", ga), ("gi", gi)), shape, dt, dev)
    _want(lam, "lam", (D,), f32, dev)
    _want(h0, "h0", (B, D), f32, dev)
    _want(lengths, "lengths", (B,), torch.int32, dev)
    _want(dy, "dy", shape, dt, dev)
    _want(d_hfinal, "d_hfinal", (B, D), f32, dev)
    res = {}
    for key in ("dx", "dga", "dgi"):
        t = out.get(key) if out else None
        res[key] = _new(shape, dt, dev, stream, dy) if t is None else t
    ld_grad = _token_stride(res.items(), shape, dt, dev) if out else D
    res["dlam"] = _result(out, "dlam", (D,), f32, dev, stream, lam)
    if state_grads:
        res["dh0"] = _result(out, "dh0", (B, D), f32, dev, stream)
    workspace, wbytes = _scratch(workspace, lambda: lru_workspace_bytes(B, T, D, dtype=dt), dev, stream)
    _launch("mesa_lru_bwd", dev, stream, ctypes.byref(LruDesc(B, T, D, ld, c, code)), _addr(x), _addr(ga), _addr(gi),
            _addr(lam), _addr(h0), _addr(lengths), _addr(dy), _addr(d_hfinal), _addr(res["dx"]), _addr(res["dga"]),
            _addr(res["dgi"]), ld_grad, _addr(res["dlam"]), _addr(res.get("dh0")), 1 if states_in_workspace else 0,
            _addr(workspace), wbytes)
    return res


def lru_step(x, ga, gi, lam, h_state, *, c: float = 8.0, out=None, stream=None) -> dict:
    """One token of N sequences: x, ga, gi [N, D] (rows dense or slices of wider
    ones), h_state [N, D] fp32 updated in place.  Returns ``y`` [N, D] in x's dtype."""
    dev, dt = _home(x, "x", 2, stream), x.dtype
    shape = x.shape
    N, D = shape
    code, ld = _code_of(x, "x"), _token_stride((("x", x), ("ga", ga), ("gi", gi)), shape, dt, dev)
    _want(lam, "lam", (D,), torch.float32, dev)
    _want(h_state, "h_state", shape, torch.float32, dev)
    y = _result(out, "y", shape, dt, dev, stream, x)
    _launch("mesa_lru_step", dev, stream, N, D, ld, c, code, _addr(x), _addr(ga), _addr(gi), _addr(lam),
            _addr(h_state), _addr(y))
    return {"y": y}


def rmsnorm(x, w, *, residual=None, eps: float = 1e-6, quant_group: Optional[int] = None,
            return_residual: Optional[bool] = None, out=None, stream=None) -> dict:
    """Residual addition and RMS norm of the rows of x [R, D] (fp32 or bf16):
    s = x + residual, y = w s / sqrt(mean(s^2) + eps).  w [D] fp32; residual
    [R, D] in x's dtype or fp32, or None.

    quant_group None: ``y`` in x's dtype.  0 or 128: ``y`` as
    ``torch.float8_e4m3fn`` with fp32 ``scale`` [R, 1] (per row) or
    [R, ceil(D/128)] (per 128 channels).  ``residual`` is s in the residual's
    dtype (return_residual; default: when a residual is given).  ``out`` may pass
    result tensors; out["residual"] may be the residual itself."""
    dev, dt = _home(x, "x", 2, stream), x.dtype
    shape = x.shape
    R, D = shape
    code = _code_of(x, "x")
    _want(x, "x", shape, dt, dev)
    _want(w, "w", (D,), torch.float32, dev)
    res_dt, res_code = dt, code
    if residual is not None:
        res_dt, res_code = residual.dtype, _code_of(residual, "residual")
        _want(residual, "residual", shape, res_dt, dev)
    quant = quant_group is not None
    res = {"y": _result(out, "y", shape, torch.float8_e4m3fn if quant else dt, dev, stream,
                        None if quant else x)}
    if quant:
        groups = -(-D // quant_group) if quant_group > 0 else 1
        res["scale"] = _result(out, "scale", (R, groups), torch.float32, dev, stream)
    if residual is not None if return_residual is None else return_residual:
        res["residual"] = _result(out, "residual", shape, res_dt, dev, stream, x if residual is None else residual)
    _launch("mesa_rmsnorm", dev, stream, R, D, code, res_code, _addr(x), _addr(residual), _addr(w), eps,
            1 if quant else 0, quant_group or 0, _addr(res["y"]), _addr(res.get("scale")), _addr(res.get("residual")))
    return res


def rmsnorm_bwd_workspace_bytes(R, D) -> int:
    """Scratch bytes of rmsnorm_bwd."""
    return lib().mesa_rmsnorm_bwd_workspace_bytes(R, D)


def rmsnorm_bwd(s, w, dy, *, d_residual=None, eps: float = 1e-6, out=None,
                workspace: Optional[torch.Tensor] = None, stream=None) -> dict:
    """Gradients of rmsnorm at s [R, D] (the ``residual`` it returned, or x where
    there was none) and w: dy [R, D]; d_residual [R, D] in s's dtype or None, what
    reaches s along the residual stream.  Returns ``ds`` in s's dtype (the gradient
    of the residual and of x), ``dw`` [D] fp32 and, where dy is bf16 and s fp32,
    ``dx``: ds in bf16.  out["ds"] may be d_residual itself."""
    dev, dt = _home(s, "s", 2, stream), s.dtype
    shape = s.shape
    R, D = shape
    _want(s, "s", shape, dt, dev)
    _want(w, "w", (D,), torch.float32, dev)
    _want(dy, "dy", shape, dy.dtype, dev)
    _want(d_residual, "d_residual", shape, dt, dev)
    res = {"ds": _result(out, "ds", shape, dt, dev, stream, s),
           "dw": _result(out, "dw", (D,), torch.float32, dev, stream, w)}
    if dy.dtype != dt:
        res["dx"] = _result(out, "dx", shape, dy.dtype, dev, stream, dy)
    workspace, wbytes = _scratch(workspace, lambda: rmsnorm_bwd_workspace_bytes(R, D), dev, stream)
    _launch("mesa_rmsnorm_bwd", dev, stream, R, D, _code_of(dy, "dy"), _code_of(s, "s"), _addr(s), _addr(w),
            _addr(dy), _addr(d_residual), eps, _addr(res["ds"]), _addr(res.get("dx")), _addr(res["dw"]),
            _addr(workspace), wbytes)
    return res


def qk_preprocess_bwd_workspace_bytes(B, H, T, d, window, *, dtype=torch.bfloat16) -> int:
    """Scratch bytes of qk_preprocess_bwd."""
    code = MESA_BF16 if dtype == torch.bfloat16 else MESA_F32
    return lib().mesa_qk_preprocess_bwd_workspace_bytes(B, H, T, d, window, code)


def qk_preprocess_bwd(q_raw, k_raw, w_q, w_k, d_q, d_k, *, q_hist=None, k_hist=None, d_q_hist_out=None,
                      d_k_hist_out=None, eps: float = 1e-6, history_grads: bool = False, out=None,
                      workspace: Optional[torch.Tensor] = None, stream=None) -> dict:
    """Gradients of qk_preprocess: d_q, d_k [B, H, T, d] fp32 at its outputs (bwd_chunked's
    dq and dk), d_q_hist_out, d_k_hist_out [B, H, W-1, d] at its history outputs or None.
    Returns ``dq_raw``, ``dk_raw`` in the raw dtype, ``dw_q``, ``dw_k`` [H, d, W] fp32 and,
    with history_grads, ``dq_hist``, ``dk_hist``."""
    dev, dt, f32 = _home(q_raw, "q_raw", 4, stream), q_raw.dtype, torch.float32
    shape = q_raw.shape
    B, H, T, d = shape
    W = w_q.shape[-1]
    taps, hist = (H, d, W), (B, H, W - 1, d)
    code = _code_of(q_raw, "q_raw")
    _want(q_raw, "q_raw", shape, dt, dev)
    _want(k_raw, "k_raw", shape, dt, dev)
    _want(w_q, "w_q", taps, f32, dev)
    _want(w_k, "w_k", taps, f32, dev)
    _want(d_q, "d_q", shape, f32, dev)
    _want(d_k, "d_k", shape, f32, dev)
    _want(q_hist, "q_hist", hist, dt, dev)
    _want(k_hist, "k_hist", hist, dt, dev)
    _want(d_q_hist_out, "d_q_hist_out", hist, dt, dev)
    _want(d_k_hist_out, "d_k_hist_out", hist, dt, dev)
    res = {key: _result(out, key, shape, dt, dev, stream, q_raw) for key in ("dq_raw", "dk_raw")}
    res.update((key, _result(out, key, taps, f32, dev, stream, w_q)) for key in ("dw_q", "dw_k"))
    if history_grads:
        res.update((key, _result(out, key, hist, dt, dev, stream)) for key in ("dq_hist", "dk_hist"))
    workspace, wbytes = _scratch(workspace, lambda: qk_preprocess_bwd_workspace_bytes(B, H, T, d, W, dtype=dt), dev,
                                 stream)
    _launch("mesa_qk_preprocess_bwd", dev, stream, B, H, T, d, W, code, _addr(q_raw), _addr(k_raw), _addr(w_q),
            _addr(w_k), _addr(q_hist), _addr(k_hist), eps, _addr(d_q), _addr(d_k), _addr(d_q_hist_out),
            _addr(d_k_hist_out), _addr(res["dq_raw"]), _addr(res["dk_raw"]), _addr(res["dw_q"]), _addr(res["dw_k"]),
            _addr(res.get("dq_hist")), _addr(res.get("dk_hist")), _addr(workspace), wbytes)
    return res


def _rows(t: torch.Tensor) -> Rows:
    """The strides of [B, heads, T, d] (or [B, heads, T]) in elements."""
    st = t.stride()
    return Rows(st[0], st[1], st[2])


def _delta_in(t: torch.Tensor, name: str, shape, dtype, dev):
    """t [..., d] of this shape and type on dev, whose last index is contiguous."""
    if t.shape != shape:
        raise MesaError(f"{name} has shape {tuple(t.shape)}, expected {shape}")
    if t.dtype is not dtype or t.device != dev:
        raise MesaError(f"{name} must be {dtype} on {dev}, got {t.dtype} on {t.device}")
    if t.stride(-1) != 1 and t.numel():
        raise MesaError(f"{name} has strides {tuple(t.stride())}: the last index must be contiguous")


def _delta_desc(q, k, v, gamma, beta, stream):
    """(the descriptor but for o, the device, the type) of checked inputs."""
    dev, dt = _home(q, "q", 4, stream), q.dtype
    code = _code_of(q, "q")
    B, Hk, T, dk = q.shape
    if v.dim() != 4:
        raise MesaError(f"v has shape {tuple(v.shape)}, expected 4 dimensions")
    H, dv = v.shape[1], v.shape[3]
    _delta_in(q, "q", (B, Hk, T, dk), dt, dev)
    _delta_in(k, "k", (B, Hk, T, dk), dt, dev)
    _delta_in(v, "v", (B, H, T, dv), dt, dev)
    _delta_gate(gamma, "gamma", (B, H, T), dev)
    _delta_gate(beta, "beta", (B, H, T), dev)
    desc = DeltaDesc(B, H, Hk, T, dk, dv, code, _rows(q), _rows(k), _rows(v), Rows(0, 0, 0), _rows(gamma), _rows(beta))
    return desc, dev, dt


def _delta_gate(t: torch.Tensor, name: str, shape, dev):
    if t.shape != shape or t.dtype is not torch.float32 or t.device != dev:
        raise MesaError(f"{name} must be float32 {shape} on {dev}, got {t.dtype} {tuple(t.shape)} on {t.device}")


def _delta_out(out, key, like, dev, stream):
    """out[key], checked, or a new tensor that lies in memory as `like` does (dense where that shares rows)."""
    t = out.get(key) if out else None
    if t is not None:
        if like.dim() == 4:
            _delta_in(t, key, tuple(like.shape), like.dtype, dev)
        else:
            _delta_gate(t, key, tuple(like.shape), dev)
        return t
    if stream is not None:
        with torch.cuda.stream(stream):
            return torch.empty_like(like)
    return torch.empty_like(like)


def delta_workspace_bytes(q, k, v, gamma, beta, *, keep_states: bool = False) -> int:
    """Scratch bytes of delta_fwd for these inputs or, with keep_states, of a forward
    that leaves its states and of delta_bwd."""
    desc, _, _ = _delta_desc(q, k, v, gamma, beta, None)
    return lib().mesa_delta_workspace_bytes(ctypes.byref(desc), 1 if keep_states else 0)


def delta_fwd(q, k, v, gamma, beta, *, s0=None, lengths=None, return_state: bool = False, keep_states: bool = False,
              out=None, workspace: Optional[torch.Tensor] = None, stream=None) -> dict:
    """Gated delta rule over whole sequences: S_t = gamma_t S_{t-1} + beta_t (v_t -
    gamma_t S_{t-1} k_t) k_t^T, o_t = S_t q_t.

    q, k [B, Hk, T, dk], v [B, H, T, dv] (fp32 or bf16; H a multiple of Hk), gamma, beta
    [B, H, T] fp32: any strides whose last index (of q, k, v) is contiguous, so a
    transposed [B, T, H, d] tensor or a slice of a wider one is taken as it is.  s0
    [B, H, dv, dk] fp32 or None; lengths [B] int32 or None (valid tokens; outputs
    behind them are zeros).  Returns a dict with ``o`` [B, H, T, dv] in v's dtype and
    layout and, with return_state, ``s_final`` [B, H, dv, dk] fp32 (out["s_final"] may
    be s0 itself).  With keep_states, ``workspace`` (delta_workspace_bytes(...,
    keep_states=True) long) keeps the states that ``delta_bwd`` can take over."""
    desc, dev, dt = _delta_desc(q, k, v, gamma, beta, stream)
    f32 = torch.float32
    state = (desc.B, desc.H, desc.dv, desc.dk)
    _want(s0, "s0", state, f32, dev)
    _want(lengths, "lengths", (desc.B,), torch.int32, dev)
    if keep_states and workspace is None:
        raise MesaError("keep_states needs a workspace")
    res = {"o": _delta_out(out, "o", v, dev, stream)}
    desc.o = _rows(res["o"])
    if return_state:
        res["s_final"] = _result(out, "s_final", state, f32, dev, stream)
    keep = 1 if keep_states else 0
    workspace, wbytes = _scratch(workspace, lambda: lib().mesa_delta_workspace_bytes(ctypes.byref(desc), keep), dev,
                                 stream)
    _launch("mesa_delta_fwd", dev, stream, ctypes.byref(desc), _addr(q), _addr(k), _addr(v), _addr(gamma), _addr(beta),
            _addr(s0), _addr(lengths), _addr(res["o"]), _addr(res.get("s_final")), keep, _addr(workspace), wbytes)
    return res


def delta_bwd(q, k, v, gamma, beta, d_o, *, s0=None, lengths=None, d_sfinal=None, state_grads: bool = False, out=None,
              workspace: Optional[torch.Tensor] = None, states_in_workspace: bool = False, stream=None) -> dict:
    """Gradients of delta_fwd: d_o [B, H, T, dv] in v's dtype (any strides whose last
    index is contiguous), d_sfinal [B, H, dv, dk] fp32 or None.  Returns ``dq``, ``dk``,
    ``dv``, ``dgamma``, ``dbeta`` in the type and layout of q, k, v, gamma and beta and,
    with state_grads, ``ds0`` [B, H, dv, dk] fp32.  ``out`` may pass result tensors
    (slices of one wider tensor too), and d_sfinal itself as ds0.  states_in_workspace: the forward ran with keep_states and
    ``workspace`` and left its states there, so they are not formed again."""
    if states_in_workspace and workspace is None:
        raise MesaError("states_in_workspace needs the forward's workspace")
    desc, dev, dt = _delta_desc(q, k, v, gamma, beta, stream)
    f32 = torch.float32
    state = (desc.B, desc.H, desc.dv, desc.dk)
    _delta_in(d_o, "d_o", tuple(v.shape), dt, dev)
    _want(s0, "s0", state, f32, dev)
    _want(lengths, "lengths", (desc.B,), torch.int32, dev)
    _want(d_sfinal, "d_sfinal", state, f32, dev)
    res = {key: _delta_out(out, key, like, dev, stream)
           for key, like in (("dq", q), ("dk", k), ("dv", v), ("dgamma", gamma), ("dbeta", beta))}
    if state_grads:
        res["ds0"] = _result(out, "ds0", state, f32, dev, stream)
    rows = DeltaGradRows(_rows(d_o), *(_rows(res[key]) for key in ("dq", "dk", "dv", "dgamma", "dbeta")))
    workspace, wbytes = _scratch(workspace, lambda: lib().mesa_delta_workspace_bytes(ctypes.byref(desc), 1), dev, stream)
    _launch("mesa_delta_bwd", dev, stream, ctypes.byref(desc), ctypes.byref(rows), _addr(q), _addr(k), _addr(v),
            _addr(gamma), _addr(beta), _addr(s0), _addr(lengths), _addr(d_o), _addr(d_sfinal), _addr(res["dq"]),
            _addr(res["dk"]), _addr(res["dv"]), _addr(res["dgamma"]), _addr(res["dbeta"]), _addr(res.get("ds0")),
            1 if states_in_workspace else 0, _addr(workspace), wbytes)
    return res


def delta_step(q, k, v, gamma, beta, s_state, *, out=None, stream=None) -> dict:
    """One token of N sequences: q, k [N, Hk, dk], v [N, H, dv] (fp32 or bf16, last index
    contiguous), gamma, beta [N, H] fp32, s_state [N, H, dv, dk] fp32 updated in place.
    Returns ``o`` [N, H, dv] in v's dtype; out["o"] may be a slice of a wider tensor."""
    dev, dt = _home(q, "q", 3, stream), q.dtype
    code = _code_of(q, "q")
    N, Hk, dk = q.shape
    if v.dim() != 3:
        raise MesaError(f"v has shape {tuple(v.shape)}, expected 3 dimensions")
    _, H, dv = v.shape
    _delta_in(k, "k", (N, Hk, dk), dt, dev)
    _delta_in(v, "v", (N, H, dv), dt, dev)
    _delta_in(q, "q", (N, Hk, dk), dt, dev)
    _delta_gate(gamma, "gamma", (N, H), dev)
    _delta_gate(beta, "beta", (N, H), dev)
    _want(s_state, "s_state", (N, H, dv, dk), torch.float32, dev)
    if out and out.get("o") is not None:
        o = out["o"]
        _delta_in(o, "o", (N, H, dv), dt, dev)
    else:
        o = _new((N, H, dv), dt, dev, stream, v)
    rows = [Rows(*t.stride()[:2], 0) for t in (q, k, v, o, gamma, beta)]
    desc = DeltaDesc(N, H, Hk, 1, dk, dv, code, *rows)
    _launch("mesa_delta_step", dev, stream, ctypes.byref(desc), _addr(q), _addr(k), _addr(v), _addr(gamma), _addr(beta),
            _addr(s_state), _addr(o))
    return {"o": o}


_CODES = {torch.float32: MESA_F32, torch.bfloat16: MESA_BF16}
_device_index, _is_dense, _numel, _data_ptr = (torch.Tensor.get_device, torch.Tensor.is_contiguous, torch.Tensor.numel,
                                               torch.Tensor.data_ptr)


def _clip_lists(grads, out, stream):
    """(the device, count, and the arrays that the library takes) of checked gradients."""
    if not grads:
        raise MesaError("grads is empty")
    dev = grads[0].device
    if not grads[0].is_cuda:
        raise MesaError("grads must be device tensors")
    if stream is not None and stream.device != dev:
        raise MesaError(f"the stream belongs to {stream.device}, grads are on {dev}")
    n = len(grads)
    codes = [_CODES.get(g.dtype) for g in grads]
    if None in codes or set(map(_device_index, grads)) != {dev.index} or not all(map(_is_dense, grads)):
        i, g = next((i, g) for i, g in enumerate(grads)
                    if codes[i] is None or _device_index(g) != dev.index or not g.is_contiguous())
        raise MesaError(f"grads[{i}] must be dense float32 or bfloat16 on {dev}, got {g.dtype} on {g.device}")
    sizes = list(map(_numel, grads))
    at = (ctypes.c_void_p * n)(*map(_data_ptr, grads))
    to = at
    if out is not None and out is not grads:
        if len(out) != n:
            raise MesaError(f"out has {len(out)} tensors, grads {n}")
        for i, (g, o) in enumerate(zip(grads, out)):
            if o.dtype is not g.dtype or o.shape != g.shape or o.device != dev or not o.is_contiguous():
                raise MesaError(f"out[{i}] must be as grads[{i}] is")
        to = (ctypes.c_void_p * n)(*map(_data_ptr, out))
    return dev, n, at, to, (ctypes.c_int64 * n)(*sizes), (ctypes.c_int * n)(*codes)


def grad_norm(grads, *, out=None, workspace: Optional[torch.Tensor] = None, stream=None) -> dict:
    """``norm`` [] fp32: the 2-norm of all tensors of the list together (dense fp32 or
    bf16, at any element's address).  ``out`` may pass the tensor for it."""
    dev, n, at, _, sizes, codes = _clip_lists(grads, None, stream)
    norm = _result(out, "norm", (), torch.float32, dev, stream)
    workspace, wbytes = _scratch(workspace, lambda: lib().mesa_grad_clip_workspace_bytes(), dev, stream)
    _launch("mesa_grad_norm", dev, stream, n, at, sizes, codes, _addr(norm), _addr(workspace), wbytes)
    return {"norm": norm}


def grad_clip(grads, max_norm: float, *, eps: float = 1e-6, out=None, workspace: Optional[torch.Tensor] = None,
              stream=None) -> dict:
    """All gradients times min(1, max_norm / (norm + eps)), norm being the 2-norm of all
    of them together: in place, or into the tensors of ``out`` (a list; an entry may be
    its gradient itself).  grads: a list of dense fp32 or bf16 tensors on one device, at
    any element's address.  Returns ``norm`` and ``scale`` ([] fp32) and ``grads``, the
    clipped tensors."""
    dev, n, at, to, sizes, codes = _clip_lists(grads, out, stream)
    both = _new((2,), torch.float32, dev, stream)
    norm, scale = both.unbind()
    workspace, wbytes = _scratch(workspace, lambda: lib().mesa_grad_clip_workspace_bytes(), dev, stream)
    _launch("mesa_grad_clip", dev, stream, n, at, to, sizes, codes, max_norm, eps, _addr(both), both.data_ptr() + 4,
            _addr(workspace), wbytes)
    return {"norm": norm, "scale": scale, "grads": grads if out is None else out}
