"""newton_schulz_gram_amd — batched Newton–Schulz / Gram Newton–Schulz on MI355X.

A thin ctypes binding over libnsg.so (include/nsg.h).  Every step of the
orthogonalization runs in the library's gfx950 HIP kernels; this module only
checks and marshals arguments, takes device memory and the current stream from
PyTorch, and raises if the library is missing or a call fails.  There is no
CPU fallback.

    import torch, newton_schulz_gram_amd as nsg
    O = nsg.orthogonalize(G)            # G: [R, C] or [G, R, C] on the GPU
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
from typing import NamedTuple, Optional, Sequence

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libnsg.so")

NSG_F16, NSG_BF16, NSG_F32, NSG_F8E4M3, NSG_F8E5M2 = 0, 1, 2, 3, 4
NSG_STANDARD, NSG_GRAM = 0, 1
MUON_COEFFS = (3.4445, -4.7750, 2.0315)  # "muon" kernel card, "How it works"

_DT = {torch.float16: NSG_F16, torch.bfloat16: NSG_BF16, torch.float32: NSG_F32}
_DT_NAMES = {"f16": NSG_F16, "fp16": NSG_F16, "float16": NSG_F16,
             "bf16": NSG_BF16, "bfloat16": NSG_BF16,
             "f32": NSG_F32, "fp32": NSG_F32, "float32": NSG_F32}
_F8 = {torch.float8_e4m3fn: NSG_F8E4M3, torch.float8_e5m2: NSG_F8E5M2}
_MODES = {"standard": NSG_STANDARD, "gram": NSG_GRAM}
KIND_NAMES = {0: "norm_reduce", 1: "scale_cast_transpose", 2: "gemm_nt", 3: "gemm_nt_sym"}

STATUS = {0: "ok", 1: "invalid argument", 2: "unsupported dtype", 3: "unsupported shape",
          4: "workspace missing, misaligned or too small", 5: "HIP runtime error",
          6: "bucket needs more than the fixed no-allocation scratch"}
NOALLOC_MAX_BYTES = 128 << 20  # NSG_NOALLOC_MAX_BYTES


class NSGError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {STATUS.get(code, 'status %d' % code)} (nsg status {code})")
        self.code = code


class Params(ctypes.Structure):
    _fields_ = [
        ("steps", ctypes.c_int32),
        ("coeffs", ctypes.POINTER(ctypes.c_double)),
        ("n_coeffs", ctypes.c_int32),
        ("mode", ctypes.c_int32),
        ("restart_after", ctypes.c_int32),
        ("safety", ctypes.c_float),
        ("eps", ctypes.c_float),
        ("compute_dtype", ctypes.c_int32),
        ("sym_updates", ctypes.c_int32),
        ("restart_mask", ctypes.c_uint64),
    ]


class LaunchInfo(ctypes.Structure):
    _fields_ = [
        ("kind", ctypes.c_int32),
        ("step", ctypes.c_int32),
        ("M", ctypes.c_int64),
        ("N", ctypes.c_int64),
        ("K", ctypes.c_int64),
        ("flops", ctypes.c_double),
        ("bytes", ctypes.c_double),
        ("label", ctypes.c_char * 24),
        ("a_kmajor", ctypes.c_int32),
        ("b_kmajor", ctypes.c_int32),
        ("source", ctypes.c_int32),
    ]


# nsg_launch_info_t.source: where a GEMM's operands come from
SOURCE_NAMES = {0: "plain", 1: "A converted from bf16", 2: "B converted from bf16", 3: "raw bf16"}


EXPORTS = ("ns_default_params", "ns_workspace_size", "ns_orthogonalize", "ns_status_string",
           "ns_flops", "ns_plan", "ns_timing_enable", "ns_timing_collect", "nsg_copy",
           "nsg_gemm_nt", "ns_select_workspace_size", "ns_orthogonalize_selected",
           "nsg_l1_workspace_size", "nsg_l1_norms", "nsg_topk", "ns_muon_momentum", "ns_muon_update",
           "ns_muon_workspace_size", "ns_muon_step", "ns_select_count", "ns_orthogonalize_noalloc",
           "nsg_expert_sort_workspace_size", "nsg_expert_sort", "nsg_expert_dispatch", "nsg_expert_combine",
           "nsg_expert_combine_backward", "nsg_quantize_fp8", "nsg_fp8_columns", "nsg_quantize_fp8_columns",
           "nsg_gemm_fp8_nt", "nsg_expert_gemm_fp8", "nsg_expert_wgrad_fp8",
           "nsg_embedding", "nsg_embedding_backward_workspace_size", "nsg_embedding_backward", "nsg_layer_norm",
           "nsg_layer_norm_backward_workspace_size", "nsg_layer_norm_backward", "nsg_expert_route_workspace_size",
           "nsg_expert_route", "nsg_expert_route_backward")
SELECT_ROWS, SELECT_COLS, SELECT_SMALLER = 0, 1, -1

_lib = None


def lib() -> ctypes.CDLL:
    """Load libnsg.so from the package directory (raises if it is not built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"libnsg.so is not built ({LIB_PATH}); run "
                           "`python -m newton_schulz_gram_amd.build` or __graft_entry__.build()")
    L = ctypes.CDLL(LIB_PATH)
    i32, i64, f32, vp, sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t
    P = ctypes.POINTER(Params)
    L.ns_default_params.argtypes = [P]
    L.ns_default_params.restype = None
    L.ns_workspace_size.argtypes = [i64, i64, i64, P, ctypes.POINTER(sz)]
    L.ns_workspace_size.restype = i32
    L.ns_orthogonalize.argtypes = [vp, i32, vp, i32, i64, i64, i64, P, vp, sz, vp, vp]
    L.ns_orthogonalize.restype = i32
    L.ns_orthogonalize_noalloc.argtypes = [vp, i32, vp, i32, i64, i64, i64, P, vp, vp]
    L.ns_orthogonalize_noalloc.restype = i32
    L.ns_status_string.argtypes = [i32]
    L.ns_status_string.restype = ctypes.c_char_p
    L.ns_flops.argtypes = [i64, i64, P, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_double)]
    L.ns_flops.restype = i32
    L.ns_plan.argtypes = [i64, i64, i32, P, ctypes.POINTER(LaunchInfo), i32, ctypes.POINTER(i32)]
    L.ns_plan.restype = i32
    L.ns_timing_enable.argtypes = [i32]
    L.ns_timing_enable.restype = i32
    L.ns_timing_collect.argtypes = [ctypes.POINTER(i32), ctypes.POINTER(f32), i32, ctypes.POINTER(i32)]
    L.ns_timing_collect.restype = i32
    L.nsg_copy.argtypes = [vp, vp, sz, vp]
    L.nsg_copy.restype = i32
    L.nsg_gemm_nt.argtypes = [i32, i32, i64, i64, i64, i64, vp, i64, i32, vp, i64, i32, f32, f32, vp, i64,
                              vp, i64, vp, i64, vp, f32, i32, vp, vp]
    L.nsg_gemm_nt.restype = i32
    L.ns_select_workspace_size.argtypes = [i64, i64, i64, i64, i32, i32, i32, P, ctypes.POINTER(sz)]
    L.ns_select_workspace_size.restype = i32
    L.ns_orthogonalize_selected.argtypes = [vp, i32, vp, i32, i64, i64, i64, i64, i32, P, vp, sz, vp, vp, vp]
    L.ns_orthogonalize_selected.restype = i32
    L.ns_select_count.argtypes = [i64, i64, i32, ctypes.c_double, ctypes.POINTER(i32), ctypes.POINTER(i64)]
    L.ns_select_count.restype = i32
    L.nsg_l1_workspace_size.argtypes = [i64, i64, i64, i32, ctypes.POINTER(sz)]
    L.nsg_l1_workspace_size.restype = i32
    L.nsg_l1_norms.argtypes = [vp, i32, i64, i64, i64, i32, vp, vp, sz, vp]
    L.nsg_l1_norms.restype = i32
    L.nsg_topk.argtypes = [vp, i64, i64, i64, vp, vp, vp]
    L.nsg_topk.restype = i32
    f64, u64 = ctypes.c_double, ctypes.c_uint64
    L.ns_muon_momentum.argtypes = [vp, i32, vp, i32, i64, f32, vp]
    L.ns_muon_momentum.restype = i32
    L.ns_muon_update.argtypes = [vp, i32, vp, i32, i64, f64, f64, f64, i32, u64, u64, vp]
    L.ns_muon_update.restype = i32
    L.ns_muon_workspace_size.argtypes = [i64, i64, i64, P, ctypes.POINTER(sz)]
    L.ns_muon_workspace_size.restype = i32
    L.ns_muon_step.argtypes = [vp, i32, vp, i32, vp, i32, i64, i64, i64, f32, f64, f64, f64, i32, u64, u64, P,
                               vp, sz, vp, vp]
    L.ns_muon_step.restype = i32
    psz = ctypes.POINTER(sz)
    L.nsg_expert_sort_workspace_size.argtypes = [i64, i64, i64, psz]
    L.nsg_expert_sort_workspace_size.restype = i32
    L.nsg_expert_sort.argtypes = [vp, i32, i64, i64, i64, vp, vp, vp, vp, sz, vp]
    L.nsg_expert_sort.restype = i32
    L.nsg_expert_dispatch.argtypes = [vp, i32, i64, i64, i64, vp, i64, vp, i64, vp, vp]
    L.nsg_expert_dispatch.restype = i32
    L.nsg_expert_combine.argtypes = [vp, i32, i64, i64, i64, vp, i64, i64, vp, vp, vp]
    L.nsg_expert_combine.restype = i32
    L.nsg_expert_combine_backward.argtypes = [vp, i64, vp, i64, i32, i64, i64, vp, i64, vp, i64, i64, vp, vp, vp, vp]
    L.nsg_expert_combine_backward.restype = i32
    L.nsg_quantize_fp8.argtypes = [vp, i32, i64, i64, i64, i64, i32, i32, vp, vp, vp, vp, vp]
    L.nsg_quantize_fp8.restype = i32
    L.nsg_fp8_columns.argtypes = [i64, i64, ctypes.POINTER(i64)]
    L.nsg_fp8_columns.restype = i32
    L.nsg_quantize_fp8_columns.argtypes = [vp, i32, i64, i64, i64, vp, i64, vp, i64, i32, vp, vp, vp]
    L.nsg_quantize_fp8_columns.restype = i32
    L.nsg_gemm_fp8_nt.argtypes = [i32, i32, i32, i64, i64, i64, i64, vp, vp, i32, vp, vp, i32, vp, vp]
    L.nsg_gemm_fp8_nt.restype = i32
    L.nsg_expert_gemm_fp8.argtypes = [i32, i32, i32, i64, i64, i64, i64, i64, vp, vp, vp, vp, vp, i32, vp, vp, vp]
    L.nsg_expert_gemm_fp8.restype = i32
    L.nsg_expert_wgrad_fp8.argtypes = [i32, i32, i32, i64, i64, i64, i64, vp, vp, vp, vp, vp, vp, vp]
    L.nsg_expert_wgrad_fp8.restype = i32
    L.nsg_embedding.argtypes = [vp, i32, i64, vp, i32, i64, i64, i64, f32, vp, vp]
    L.nsg_embedding.restype = i32
    L.nsg_embedding_backward_workspace_size.argtypes = [i64, i64, i64, psz]
    L.nsg_embedding_backward_workspace_size.restype = i32
    L.nsg_embedding_backward.argtypes = [vp, i32, i64, i64, i64, vp, i32, i64, f32, vp, i32, i32, vp, sz, vp]
    L.nsg_embedding_backward.restype = i32
    L.nsg_layer_norm.argtypes = [vp, i32, i64, i64, i64, vp, vp, i32, f32, vp, vp, vp]
    L.nsg_layer_norm.restype = i32
    L.nsg_layer_norm_backward_workspace_size.argtypes = [i64, i64, psz]
    L.nsg_layer_norm_backward_workspace_size.restype = i32
    L.nsg_layer_norm_backward.argtypes = [vp, i64, vp, i64, i32, i64, i64, vp, vp, i32, vp, vp, vp, vp, sz, vp]
    L.nsg_layer_norm_backward.restype = i32
    L.nsg_expert_route_workspace_size.argtypes = [i64, i64, psz]
    L.nsg_expert_route_workspace_size.restype = i32
    L.nsg_expert_route.argtypes = [vp, i32, i64, i64, i64, i64, i32, vp, vp, i32, f32, vp, vp, vp, vp, vp, vp, sz, vp]
    L.nsg_expert_route.restype = i32
    L.nsg_expert_route_backward.argtypes = [vp, i32, i64, i64, i64, i64, i32, i32, f32, vp, vp, vp, f32, vp, vp, vp]
    L.nsg_expert_route_backward.restype = i32
    _lib = L
    return L


def _check(code: int, what: str):
    if code != 0:
        raise NSGError(code, what)


def _dtype_code(dt) -> int:
    if isinstance(dt, str):
        return _DT_NAMES[dt]
    if isinstance(dt, torch.dtype):
        if dt not in _DT:
            raise TypeError(f"unsupported dtype {dt}")
        return _DT[dt]
    return int(dt)


def make_params(steps: int = 5, coeffs: Optional[Sequence[float]] = None, mode: str = "gram",
                restart_after: int = 2, safety: float = 1.05, eps: float = 1e-7,
                compute_dtype="f16", sym_updates: bool = True, restarts: Optional[Sequence[int]] = None):
    """Build an nsg_params_t.  Returns (params, keepalive) — keep both alive.

    `restarts` lists the steps t (2..steps) at whose top the Gram iteration
    restarts; it overrides `restart_after` (a single restart)."""
    c = list(MUON_COEFFS if coeffs is None else coeffs)
    arr = (ctypes.c_double * len(c))(*[float(x) for x in c])
    p = Params()
    p.steps = int(steps)
    p.coeffs = ctypes.cast(arr, ctypes.POINTER(ctypes.c_double))
    p.n_coeffs = len(c)
    p.mode = _MODES[mode] if isinstance(mode, str) else int(mode)
    p.restart_after = int(restart_after)
    p.safety = float(safety)
    p.eps = float(eps)
    p.compute_dtype = _dtype_code(compute_dtype)
    p.sym_updates = 1 if sym_updates else 0
    mask = 0
    for t in (restarts or ()):
        t = int(t)
        if not 1 <= t <= 64:
            raise ValueError("restart steps must lie in 2..steps")
        mask |= 1 << (t - 1)
    p.restart_mask = mask
    return p, arr


def workspace_size(G: int, R: int, C: int, **kw) -> int:
    p, _keep = make_params(**kw)
    out = ctypes.c_size_t(0)
    _check(lib().ns_workspace_size(G, R, C, ctypes.byref(p), ctypes.byref(out)), "ns_workspace_size")
    return int(out.value)


def flops(R: int, C: int, **kw):
    """(credited, executed) FLOPs per matrix (the pages' formula; the plan's tiles)."""
    p, _keep = make_params(**kw)
    cr, ex = ctypes.c_double(0), ctypes.c_double(0)
    _check(lib().ns_flops(R, C, ctypes.byref(p), ctypes.byref(cr), ctypes.byref(ex)), "ns_flops")
    return cr.value, ex.value


def plan(R: int, C: int, in_dtype=None, **kw):
    """The launch list of one call on an input of dtype `in_dtype` (default:
    the compute dtype), as a list of dicts (host only)."""
    p, _keep = make_params(**kw)
    idt = p.compute_dtype if in_dtype is None else _dtype_code(in_dtype)
    n = ctypes.c_int32(0)
    _check(lib().ns_plan(R, C, idt, ctypes.byref(p), None, 0, ctypes.byref(n)), "ns_plan")
    arr = (LaunchInfo * max(1, n.value))()
    _check(lib().ns_plan(R, C, idt, ctypes.byref(p), arr, n.value, ctypes.byref(n)), "ns_plan")
    return [dict(kind=e.kind, kernel=KIND_NAMES[e.kind], step=e.step, M=e.M, N=e.N, K=e.K,
                 flops=e.flops, bytes=e.bytes, label=e.label.decode(), a_kmajor=bool(e.a_kmajor),
                 b_kmajor=bool(e.b_kmajor), source=e.source) for e in arr[:n.value]]


def nbytes(t: torch.Tensor) -> int:
    """Bytes of a tensor's storage as the library sees it (numel x element size)."""
    return t.numel() * t.element_size()


def check_out(out: torch.Tensor, nb: int, R: int, C: int, squeeze: bool, device) -> None:
    """A caller-supplied output must hold exactly the bucket: [nb, R, C], or
    [R, C] when the input was one 2-D matrix; contiguous, on the input's device.
    The library writes nb * R * C elements into it."""
    ok_shape = tuple(out.shape) == (nb, R, C) or (squeeze and nb == 1 and tuple(out.shape) == (R, C))
    if not ok_shape:
        raise ValueError(f"out has shape {tuple(out.shape)}; expected {(R, C) if squeeze else (nb, R, C)}")
    if out.dtype not in _DT:
        raise ValueError(f"unsupported out dtype {out.dtype}")
    if not out.is_contiguous() or out.device != device:
        raise ValueError("out must be contiguous on the input's device")


def check_workspace(ws: torch.Tensor, device) -> None:
    if ws.device != device or not ws.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the input's device")


def check_status(status: Optional[torch.Tensor], nb: int, device) -> None:
    """status: None, or int32 with at least nb entries, contiguous, on the input's device."""
    if status is None:
        return
    if status.dtype != torch.int32 or status.numel() < nb or not status.is_contiguous() or status.device != device:
        raise ValueError("status must be a contiguous int32 tensor with G entries on the input's device")


def _stream_handle(device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def orthogonalize(G: torch.Tensor, steps: int = 5, coeffs: Optional[Sequence[float]] = None,
                  mode: str = "gram", restart_after: int = 2, safety: float = 1.05,
                  eps: float = 1e-7, compute_dtype="f16", out_dtype=None,
                  out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                  status: Optional[torch.Tensor] = None, sym_updates: bool = True,
                  restarts: Optional[Sequence[int]] = None) -> torch.Tensor:
    """Orthogonalize one matrix [R, C] or a bucket [G, R, C] on its GPU.

    sym_updates (default) runs Q Z + a Q and R Z + a R on the symmetric kernel
    (Gram mode; half the tiles, exactly symmetric results); False runs them
    as general products.  `restarts` lists several restart steps (see
    make_params).

    Returns `out` (allocated if not given) with dtype out_dtype (default: the
    input's).  `status`, if given, is an int32 CUDA tensor of G entries set to
    1 for matrices whose output has a non-finite value.
    """
    if not G.is_cuda:
        raise ValueError("orthogonalize needs a GPU tensor (no CPU path)")
    squeeze = G.dim() == 2
    Gs = G.unsqueeze(0) if squeeze else G
    if Gs.dim() != 3:
        raise ValueError("expected [R, C] or [G, R, C]")
    if not Gs.is_contiguous():
        raise ValueError("input must be contiguous")
    nb, R, C = Gs.shape
    odt = Gs.dtype if out_dtype is None else out_dtype
    if out is None:
        out = torch.empty((nb, R, C), dtype=odt, device=Gs.device)
    else:
        check_out(out, nb, R, C, squeeze, Gs.device)
        odt = out.dtype
    p, _keep = make_params(steps, coeffs, mode, restart_after, safety, eps, compute_dtype, sym_updates,
                           restarts)
    need = ctypes.c_size_t(0)
    _check(lib().ns_workspace_size(nb, R, C, ctypes.byref(p), ctypes.byref(need)), "ns_workspace_size")
    if workspace is None or nbytes(workspace) < need.value:
        workspace = torch.empty(max(1, need.value), dtype=torch.uint8, device=Gs.device)
    check_workspace(workspace, Gs.device)
    check_status(status, nb, Gs.device)
    with torch.cuda.device(Gs.device):
        code = lib().ns_orthogonalize(
            ctypes.c_void_p(Gs.data_ptr()), _dtype_code(Gs.dtype),
            ctypes.c_void_p(out.data_ptr()), _dtype_code(odt),
            nb, R, C, ctypes.byref(p),
            ctypes.c_void_p(workspace.data_ptr()), nbytes(workspace),
            ctypes.c_void_p(status.data_ptr()) if status is not None else None,
            ctypes.c_void_p(_stream_handle(Gs.device)))
    _check(code, "ns_orthogonalize")
    return out[0] if (squeeze and out.dim() == 3) else out


def orthogonalize_noalloc(G: torch.Tensor, out: torch.Tensor, steps: int = 5,
                          coeffs: Optional[Sequence[float]] = None, mode: str = "gram", restart_after: int = 2,
                          safety: float = 1.05, eps: float = 1e-7, compute_dtype="f16",
                          status: Optional[torch.Tensor] = None, sym_updates: bool = True,
                          restarts: Optional[Sequence[int]] = None) -> torch.Tensor:
    """orthogonalize() through ns_orthogonalize_noalloc: the library's fixed
    scratch array is the workspace, so neither the library nor this wrapper
    allocates device memory (the caller passes `out`).  Buckets whose
    workspace exceeds NOALLOC_MAX_BYTES raise NSGError (status 6).  Calls that
    may overlap on one GPU share that scratch and race."""
    if not G.is_cuda:
        raise ValueError("orthogonalize_noalloc needs a GPU tensor (no CPU path)")
    squeeze = G.dim() == 2
    Gs = G.unsqueeze(0) if squeeze else G
    if Gs.dim() != 3 or not Gs.is_contiguous():
        raise ValueError("expected a contiguous [R, C] or [G, R, C] tensor")
    nb, R, C = Gs.shape
    check_out(out, nb, R, C, squeeze, Gs.device)
    check_status(status, nb, Gs.device)
    p, _keep = make_params(steps, coeffs, mode, restart_after, safety, eps, compute_dtype, sym_updates, restarts)
    with torch.cuda.device(Gs.device):
        code = lib().ns_orthogonalize_noalloc(
            ctypes.c_void_p(Gs.data_ptr()), _dtype_code(Gs.dtype), ctypes.c_void_p(out.data_ptr()),
            _dtype_code(out.dtype), nb, R, C, ctypes.byref(p),
            ctypes.c_void_p(status.data_ptr()) if status is not None else None,
            ctypes.c_void_p(_stream_handle(Gs.device)))
    _check(code, "ns_orthogonalize_noalloc")
    return out


def timing_enable(on: bool = True):
    _check(lib().ns_timing_enable(1 if on else 0), "ns_timing_enable")


def timing_collect(max_entries: int = 1 << 16):
    """[(kernel name, ms), ...] for every launch recorded since the last collect."""
    kinds = (ctypes.c_int32 * max_entries)()
    ms = (ctypes.c_float * max_entries)()
    n = ctypes.c_int32(0)
    _check(lib().ns_timing_collect(kinds, ms, max_entries, ctypes.byref(n)), "ns_timing_collect")
    return [(KIND_NAMES[kinds[i]], float(ms[i])) for i in range(min(n.value, max_entries))]


def copy(src: torch.Tensor, dst: torch.Tensor):
    """Library copy kernel (byte-counter calibration)."""
    nbytes = src.numel() * src.element_size()
    with torch.cuda.device(src.device):
        _check(lib().nsg_copy(ctypes.c_void_p(src.data_ptr()), ctypes.c_void_p(dst.data_ptr()), nbytes,
                              ctypes.c_void_p(_stream_handle(src.device))), "nsg_copy")


def gemm_nt(A: torch.Tensor, B: torch.Tensor, alpha: float = 1.0, beta: float = 0.0,
            Cin: Optional[torch.Tensor] = None, symmetric: bool = False, transposed_out: bool = False,
            diag: Optional[float] = None, tile: int = 0, a_kmajor: bool = False, b_kmajor: bool = False,
            status: Optional[torch.Tensor] = None):
    """Library GEMM building block: V = alpha A B^T + beta Cin over a batch.

    A [b, M, K], B [b, N, K] (M, N, K multiples of 256) in one dtype; tile 128
    or 256 picks the kernel (0: the library's choice).  With a_kmajor
    (b_kmajor) A (B) is passed K-major instead, as [b, K, M] ([b, K, N]).
    Returns (V, V^T or None, V + diag I or None)."""
    b = A.shape[0]
    M, K = (A.shape[2], A.shape[1]) if a_kmajor else (A.shape[1], A.shape[2])
    N = B.shape[2] if b_kmajor else B.shape[1]
    for t in (A, B) + ((Cin,) if Cin is not None else ()):
        if t.stride(2) != 1 or t.stride(0) != t.shape[1] * t.stride(1):
            raise ValueError("gemm_nt operands need unit column stride and packed batches")
    out = torch.empty((b, M, N), dtype=A.dtype, device=A.device)
    out_t = torch.empty((b, N, M), dtype=A.dtype, device=A.device) if transposed_out else None
    out_d = torch.empty((b, M, N), dtype=A.dtype, device=A.device) if diag is not None else None
    ptr = lambda t: ctypes.c_void_p(t.data_ptr()) if t is not None else None
    with torch.cuda.device(A.device):
        code = lib().nsg_gemm_nt(_dtype_code(A.dtype), 1 if symmetric else 0, b, M, N, K,
                                 ptr(A), A.stride(1), 1 if a_kmajor else 0, ptr(B), B.stride(1),
                                 1 if b_kmajor else 0, float(alpha), float(beta), ptr(Cin),
                                 Cin.stride(1) if Cin is not None else N,
                                 ptr(out), N, ptr(out_t), M, ptr(out_d), float(diag or 0.0), int(tile), ptr(status),
                                 ctypes.c_void_p(_stream_handle(A.device)))
    _check(code, "nsg_gemm_nt")
    return out, out_t, out_d


# ---------------------------------------------------------------------------
# Dion3 selection front-end (Dion3 paper, Section 6; Algorithm 4, steps 3-4)
# ---------------------------------------------------------------------------

def select_plan(R: int, C: int, fraction: float, dim: int = SELECT_SMALLER):
    """(resolved dim, k) of the library's selection rule: k = ceil(f n) lines
    of rows (dim 0) or columns (dim 1); -1 picks the smaller dimension."""
    d, k = ctypes.c_int32(0), ctypes.c_int64(0)
    code = lib().ns_select_count(int(R), int(C), int(dim), float(fraction), ctypes.byref(d), ctypes.byref(k))
    if code == 1:
        raise ValueError("fraction must lie in (0, 1] and dim in {-1, 0, 1}")
    _check(code, "ns_select_count")
    return int(d.value), int(k.value)


def select_count(n: int, fraction: float) -> int:
    """k = ceil(f n) lines out of n (at least 1), by the library's rule."""
    return select_plan(n, n, fraction, SELECT_ROWS)[1]


def orthogonalize_selected(M: torch.Tensor, fraction: float = 0.25, k: Optional[int] = None, dim: int = -1,
                           steps: int = 5, coeffs: Optional[Sequence[float]] = None, mode: str = "gram",
                           restart_after: int = 2, safety: float = 1.05, eps: float = 1e-7,
                           compute_dtype="f16", out_dtype=None, out: Optional[torch.Tensor] = None,
                           status: Optional[torch.Tensor] = None, sym_updates: bool = True,
                           restarts: Optional[Sequence[int]] = None):
    """Select the k = ceil(f n) rows (dim 0) or columns (dim 1; -1: the smaller
    dimension) of largest l1 norm of every matrix, orthogonalize them, and
    return (out, idx): out [G, R, C] holds the result in the selected lines and
    zeros elsewhere, idx [G, k] int32 the selected indices (ascending)."""
    if not M.is_cuda:
        raise ValueError("orthogonalize_selected needs a GPU tensor (no CPU path)")
    squeeze = M.dim() == 2
    Ms = M.unsqueeze(0) if squeeze else M
    if Ms.dim() != 3 or not Ms.is_contiguous():
        raise ValueError("expected a contiguous [R, C] or [G, R, C] tensor")
    G, R, C = Ms.shape
    if k is None:
        d, kk = select_plan(R, C, fraction, dim)
    else:
        d, _ = select_plan(R, C, 1.0, dim)
        kk = int(k)
    odt = Ms.dtype if out_dtype is None else out_dtype
    if out is None:
        out = torch.empty((G, R, C), dtype=odt, device=Ms.device)
    else:
        check_out(out, G, R, C, squeeze, Ms.device)
    odt = out.dtype
    check_status(status, G, Ms.device)
    idx = torch.empty((G, kk), dtype=torch.int32, device=Ms.device)
    p, _keep = make_params(steps, coeffs, mode, restart_after, safety, eps, compute_dtype, sym_updates, restarts)
    need = ctypes.c_size_t(0)
    _check(lib().ns_select_workspace_size(G, R, C, kk, d, _dtype_code(Ms.dtype), _dtype_code(odt), ctypes.byref(p),
                                          ctypes.byref(need)), "ns_select_workspace_size")
    ws = torch.empty(max(1, need.value), dtype=torch.uint8, device=Ms.device)
    with torch.cuda.device(Ms.device):
        _check(lib().ns_orthogonalize_selected(
            ctypes.c_void_p(Ms.data_ptr()), _dtype_code(Ms.dtype), ctypes.c_void_p(out.data_ptr()), _dtype_code(odt),
            G, R, C, kk, d, ctypes.byref(p), ctypes.c_void_p(ws.data_ptr()), need.value,
            ctypes.c_void_p(idx.data_ptr()), ctypes.c_void_p(status.data_ptr()) if status is not None else None,
            ctypes.c_void_p(_stream_handle(Ms.device))), "ns_orthogonalize_selected")
    if squeeze:
        return out[0], idx[0]
    return out, idx


def l1_norms(M: torch.Tensor, dim: int = 0) -> torch.Tensor:
    """fp64 l1 norms of the rows (dim 0) or columns (dim 1) of [G, R, C]."""
    Ms = M.unsqueeze(0) if M.dim() == 2 else M
    if not Ms.is_contiguous():
        raise ValueError("input must be contiguous")
    G, R, C = Ms.shape
    n = R if dim == SELECT_ROWS else C
    keys = torch.empty((G, n), dtype=torch.float64, device=Ms.device)
    need = ctypes.c_size_t(0)
    _check(lib().nsg_l1_workspace_size(G, R, C, dim, ctypes.byref(need)), "nsg_l1_workspace_size")
    ws = torch.empty(max(1, need.value), dtype=torch.uint8, device=Ms.device)
    with torch.cuda.device(Ms.device):
        _check(lib().nsg_l1_norms(ctypes.c_void_p(Ms.data_ptr()), _dtype_code(Ms.dtype), G, R, C, dim,
                                  ctypes.c_void_p(keys.data_ptr()), ctypes.c_void_p(ws.data_ptr()), need.value,
                                  ctypes.c_void_p(_stream_handle(Ms.device))), "nsg_l1_norms")
    return keys


def topk(keys: torch.Tensor, k: int):
    """(idx [G, k] ascending, pos [G, n]) of the k largest keys per row of keys."""
    keys = keys.contiguous().to(torch.float64)
    G, n = keys.shape
    idx = torch.empty((G, k), dtype=torch.int32, device=keys.device)
    pos = torch.empty((G, n), dtype=torch.int32, device=keys.device)
    with torch.cuda.device(keys.device):
        _check(lib().nsg_topk(ctypes.c_void_p(keys.data_ptr()), G, n, k, ctypes.c_void_p(idx.data_ptr()),
                              ctypes.c_void_p(pos.data_ptr()), ctypes.c_void_p(_stream_handle(keys.device))),
               "nsg_topk")
    return idx, pos


# ---------------------------------------------------------------------------
# The Muon step (Dion3 paper, Eq. (1); Algorithm 4, steps 8-9; muon card)
# ---------------------------------------------------------------------------

def muon_momentum(M: torch.Tensor, G: torch.Tensor, mu: float):
    """In place: M <- mu M + G (fp32 arithmetic; M is float32 or bfloat16)."""
    if M.numel() != G.numel() or not (M.is_contiguous() and G.is_contiguous()):
        raise ValueError("M and G must be contiguous with the same number of elements")
    with torch.cuda.device(M.device):
        _check(lib().ns_muon_momentum(ctypes.c_void_p(M.data_ptr()), _dtype_code(M.dtype), ctypes.c_void_p(G.data_ptr()),
                                      _dtype_code(G.dtype), M.numel(), float(mu),
                                      ctypes.c_void_p(_stream_handle(M.device))), "ns_muon_momentum")
    return M


def muon_update(W: torch.Tensor, O: torch.Tensor, lr: float, weight_decay: float = 0.0, scale: float = 1.0,
                stochastic: bool = True, seed: int = 0, step: int = 0):
    """In place: W <- (1 - lr wd) W - lr scale O; a bf16 W is written back with
    counter-based stochastic rounding (seed, step, element index)."""
    if W.numel() != O.numel() or not (W.is_contiguous() and O.is_contiguous()):
        raise ValueError("W and O must be contiguous with the same number of elements")
    with torch.cuda.device(W.device):
        _check(lib().ns_muon_update(ctypes.c_void_p(W.data_ptr()), _dtype_code(W.dtype), ctypes.c_void_p(O.data_ptr()),
                                    _dtype_code(O.dtype), W.numel(), float(lr), float(weight_decay), float(scale),
                                    1 if stochastic else 0, int(seed) & (2 ** 64 - 1), int(step) & (2 ** 64 - 1),
                                    ctypes.c_void_p(_stream_handle(W.device))), "ns_muon_update")
    return W


def muon_step(W: torch.Tensor, M: torch.Tensor, G: torch.Tensor, mu: float, lr: float, weight_decay: float = 0.0,
              scale: float = 1.0, stochastic: bool = True, seed: int = 0, step: int = 0,
              status: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, **kw):
    """One Muon step for a bucket [G, R, C] (or one [R, C] matrix), in place on
    W and M; keyword arguments set the Newton-Schulz parameters."""
    Ws, Ms, Gs = (t.unsqueeze(0) if t.dim() == 2 else t for t in (W, M, G))
    if not (Ws.shape == Ms.shape == Gs.shape) or Ws.dim() != 3:
        raise ValueError("W, M and G must share a [G, R, C] or [R, C] shape")
    if not (Ws.is_contiguous() and Ms.is_contiguous() and Gs.is_contiguous()):
        raise ValueError("W, M and G must be contiguous")
    nb, R, C = Ws.shape
    p, _keep = make_params(**kw)
    need = ctypes.c_size_t(0)
    _check(lib().ns_muon_workspace_size(nb, R, C, ctypes.byref(p), ctypes.byref(need)), "ns_muon_workspace_size")
    if workspace is None or nbytes(workspace) < need.value:
        workspace = torch.empty(max(1, need.value), dtype=torch.uint8, device=Ws.device)
    if not (Ms.device == Gs.device == Ws.device):
        raise ValueError("W, M and G must be on one device")
    check_workspace(workspace, Ws.device)
    check_status(status, nb, Ws.device)
    with torch.cuda.device(Ws.device):
        _check(lib().ns_muon_step(
            ctypes.c_void_p(Ws.data_ptr()), _dtype_code(Ws.dtype), ctypes.c_void_p(Ms.data_ptr()), _dtype_code(Ms.dtype),
            ctypes.c_void_p(Gs.data_ptr()), _dtype_code(Gs.dtype), nb, R, C, float(mu), float(lr), float(weight_decay),
            float(scale), 1 if stochastic else 0, int(seed) & (2 ** 64 - 1), int(step) & (2 ** 64 - 1), ctypes.byref(p),
            ctypes.c_void_p(workspace.data_ptr()), nbytes(workspace),
            ctypes.c_void_p(status.data_ptr()) if status is not None else None,
            ctypes.c_void_p(_stream_handle(Ws.device))), "ns_muon_step")
    return W, M


# ---------------------------------------------------------------------------
# The expert layer around the Muon step: tokens sorted by expert and back, 8-bit
# operands with one scale for each block of 128, their products
# ---------------------------------------------------------------------------

class ExpertPlan(NamedTuple):
    """Where expert_sort puts the T x k choices of a router.

    offsets [E + 1] int32: sorted rows offsets[e] .. offsets[e + 1] - 1 are expert
    e's; rows [T, k] int32: the sorted row of each choice, -1 if it was dropped;
    tokens [T k] int32: the token in each sorted row, -1 behind offsets[E]."""
    offsets: torch.Tensor
    rows: torch.Tensor
    tokens: torch.Tensor


def _launch(device, what: str, fn, *args):
    """Call a C entry point on `device`, with its current stream as the last argument.

    Both lookups are torch's raw ones: the public forms (torch.cuda.current_stream,
    torch.cuda.device) cost 2 us of a call of 10."""
    index = device.index
    if index == torch._C._cuda_getDevice():
        code = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(device):
            code = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    if code:
        raise NSGError(code, what)


def _gpu(t: torch.Tensor, what: str):
    if not t.is_cuda:
        raise ValueError(f"{what} needs GPU tensors (no CPU path)")
    return t.device


def _ints(t: torch.Tensor, shape, name: str, device):
    """An int32 plan array of this shape (None: any), contiguous, on the device."""
    if t.dtype != torch.int32 or t.device != device or not t.is_contiguous() or (shape is not None and t.shape != shape):
        raise ValueError(f"{name} must be a contiguous int32 tensor{'' if shape is None else ' of shape %s' % (tuple(shape),)}"
                         " on the input's device")


def _matrix(t: torch.Tensor, name: str, device=None):
    """Rows of a 2-D tensor with unit column stride: their pitch in elements."""
    if t.dim() != 2 or t.dtype not in _DT:
        raise ValueError(f"{name} must be a 2-D float16, bfloat16 or float32 tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on the input's device")
    return _pitch(t, name)


def _pitch(t: torch.Tensor, name: str) -> int:
    """Distance of the rows of t [..., R, C]; its rows must be packed and not overlap."""
    R, C = t.shape[-2:]
    if C > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} needs unit column stride")
    ld = t.stride(-2) if R > 1 else C
    if ld < C:
        raise ValueError(f"{name} has overlapping rows")
    return ld


def _router_weights(weights: Optional[torch.Tensor], rows: torch.Tensor):
    if weights is None:
        return None
    if weights.dtype != torch.float32 or weights.shape != rows.shape or not weights.is_contiguous() or \
            weights.device != rows.device:
        raise ValueError("weights must be a contiguous float32 [T, k] tensor on the input's device")
    return weights.data_ptr()


def _plan_rows(plan: ExpertPlan, device):
    if plan.rows.dim() != 2:
        raise ValueError("plan.rows must be [T, k]")
    _ints(plan.rows, None, "plan.rows", device)
    return plan.rows.shape


def expert_sort(ids: torch.Tensor, num_experts: int, workspace: Optional[torch.Tensor] = None) -> ExpertPlan:
    """Sort the choices ids [T, k] (int32 or int64) of a router by expert, stably.

    An id outside 0 .. num_experts - 1 is dropped.  `workspace`: a uint8 tensor
    of expert_sort_workspace_size(T, k, num_experts) bytes (allocated if not given)."""
    device = _gpu(ids, "expert_sort")
    if ids.dim() != 2 or ids.dtype not in (torch.int32, torch.int64) or not ids.is_contiguous():
        raise ValueError("ids must be a contiguous [T, k] int32 or int64 tensor")
    T, k = ids.shape
    E = int(num_experts)
    need = expert_sort_workspace_size(T, k, E)
    if need and (workspace is None or nbytes(workspace) < need):
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    if workspace is not None:
        check_workspace(workspace, device)
    offsets = torch.empty(E + 1, dtype=torch.int32, device=device)
    rows = torch.empty((T, k), dtype=torch.int32, device=device)
    tokens = torch.empty(T * k, dtype=torch.int32, device=device)
    _launch(device, "nsg_expert_sort", lib().nsg_expert_sort, ids.data_ptr(), 8 * ids.element_size(), T, k, E,
            offsets.data_ptr(), rows.data_ptr(), tokens.data_ptr(),
            workspace.data_ptr() if workspace is not None else None, nbytes(workspace) if workspace is not None else 0)
    return ExpertPlan(offsets, rows, tokens)


def expert_sort_workspace_size(T: int, k: int, num_experts: int) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().nsg_expert_sort_workspace_size(T, k, num_experts, ctypes.byref(out)), "nsg_expert_sort_workspace_size")
    return out.value


def expert_dispatch(x: torch.Tensor, plan: ExpertPlan) -> torch.Tensor:
    """The sorted rows [T k, C] of tokens x [T, C]: x[t] in the rows plan.rows[t],
    zeros behind the last expert's.  Its gradient is expert_combine without weights."""
    device = _gpu(x, "expert_dispatch")
    ld = _matrix(x, "x")
    T, k = _plan_rows(plan, device)
    _ints(plan.offsets, None, "plan.offsets", device)
    C = x.shape[1]
    if x.shape[0] != T:
        raise ValueError(f"x has {x.shape[0]} rows, the plan {T} tokens")
    out = torch.empty((T * k, C), dtype=x.dtype, device=device)
    _launch(device, "nsg_expert_dispatch", lib().nsg_expert_dispatch, x.data_ptr(), _DT[x.dtype], T, C, ld,
            plan.offsets.data_ptr(), plan.offsets.numel() - 1, plan.rows.data_ptr(), k, out.data_ptr())
    return out


def expert_combine(y: torch.Tensor, plan: ExpertPlan, weights: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Bring sorted rows y [T k, C] back: out[t] = sum_j weights[t, j] y[plan.rows[t, j]]
    (fp32 sums, rounded once; dropped choices are left out).  weights: float32
    [T, k], or None for all 1, which is the gradient of expert_dispatch."""
    device = _gpu(y, "expert_combine")
    ld = _matrix(y, "y")
    T, k = _plan_rows(plan, device)
    P, C = y.shape
    if P != T * k:
        raise ValueError(f"y has {P} rows, the plan {T * k}")
    out = torch.empty((T, C), dtype=y.dtype, device=device)
    _launch(device, "nsg_expert_combine", lib().nsg_expert_combine, y.data_ptr(), _DT[y.dtype], P, C, ld,
            plan.rows.data_ptr(), T, k, _router_weights(weights, plan.rows), out.data_ptr())
    return out


def expert_combine_backward(dout: torch.Tensor, y: torch.Tensor, plan: ExpertPlan,
                            weights: Optional[torch.Tensor] = None):
    """The gradient of expert_combine: (dy [T k, C], dw [T, k] float32) for dout [T, C].
    dy is zero in the rows behind the last expert's, dw for a dropped choice."""
    device = _gpu(dout, "expert_combine_backward")
    lddo, ldy = _matrix(dout, "dout"), _matrix(y, "y", device)
    T, k = _plan_rows(plan, device)
    P, C = y.shape
    _ints(plan.offsets, None, "plan.offsets", device)
    if P != T * k or dout.shape != (T, C) or dout.dtype != y.dtype:
        raise ValueError("dout must be [T, C] and y [T k, C] of the plan, of one dtype")
    dy = torch.empty((P, C), dtype=y.dtype, device=device)
    dw = torch.empty((T, k), dtype=torch.float32, device=device)
    _launch(device, "nsg_expert_combine_backward", lib().nsg_expert_combine_backward, dout.data_ptr(), lddo, y.data_ptr(),
            ldy, _DT[y.dtype], P, C, plan.offsets.data_ptr(), plan.offsets.numel() - 1, plan.rows.data_ptr(), T, k,
            _router_weights(weights, plan.rows), dy.data_ptr(), dw.data_ptr())
    return dy, dw


FP8_BLOCK = 128
_BLOCKS = {"row": 0, "tile": 1}


def _up128(n: int) -> int:
    return -(-n // FP8_BLOCK) * FP8_BLOCK


def _f8_code(dtype) -> int:
    if dtype not in _F8:
        raise TypeError(f"unsupported 8-bit dtype {dtype}")
    return _F8[dtype]


def quantize_fp8(x: torch.Tensor, block: str = "row", dtype=torch.float8_e4m3fn, transposed: bool = False):
    """Quantise x [R, C] or [B, R, C] to 8 bits with one fp32 scale for 128 elements
    of a row ("row") or a 128 x 128 tile ("tile").

    Returns (q, scale): q [(B,) R, Cp] with Cp = C rounded up to 128 and zeros
    behind C, scale [(B,) Cp/128, R] or [(B,) Cp/128, ceil(R/128)]; x ~ q * scale
    with scale = max(amax / F, 2^-126).  With `transposed` (tiles) also the
    operand of the transposed matrix, (q, scale, qt, scale_t), with the same
    numbers.  Infinities and NaN do not change their block's scale and become NaN
    (an infinity stays one in float8_e5m2).  At most 2^25 rows of a matrix,
    128 * 65535 with "tile"."""
    device = _gpu(x, "quantize_fp8")
    xs = x.unsqueeze(0) if x.dim() == 2 else x
    if xs.dim() != 3 or x.dtype not in _DT:
        raise ValueError("expected a float16, bfloat16 or float32 tensor [R, C] or [B, R, C]")
    if block not in _BLOCKS:
        raise ValueError("block must be 'row' or 'tile'")
    if transposed and block != "tile":
        raise ValueError("transposed needs block='tile'")
    f8 = _f8_code(dtype)
    ld = _pitch(xs, "x")
    B, R, C = xs.shape
    if B > 1 and xs.stride(0) != R * ld:
        raise ValueError("x needs packed batches")
    Rp, Cp = _up128(R), _up128(C)
    lead = () if x.dim() == 2 else (B,)
    q = torch.empty((*lead, R, Cp), dtype=dtype, device=device)
    s = torch.empty((*lead, Cp // 128, R if block == "row" else Rp // 128), dtype=torch.float32, device=device)
    qt = st = None
    if transposed:
        qt = torch.empty((*lead, C, Rp), dtype=dtype, device=device)
        st = torch.empty((*lead, Rp // 128, Cp // 128), dtype=torch.float32, device=device)
    _launch(device, "nsg_quantize_fp8", lib().nsg_quantize_fp8, xs.data_ptr(), _DT[x.dtype], B, R, C, ld, _BLOCKS[block],
            f8, q.data_ptr(), s.data_ptr(), qt.data_ptr() if transposed else None, st.data_ptr() if transposed else None)
    return (q, s, qt, st) if transposed else (q, s)


def fp8_columns(P: int, num_experts: int) -> int:
    """Columns of the layout of quantize_fp8_columns: 128 (floor(P / 128) + num_experts)."""
    out = ctypes.c_int64(0)
    _check(lib().nsg_fp8_columns(P, num_experts, ctypes.byref(out)), "nsg_fp8_columns")
    return out.value


def quantize_fp8_columns(x: torch.Tensor, offsets: torch.Tensor, rows: Optional[torch.Tensor] = None,
                         dtype=torch.float8_e4m3fn):
    """Quantise sorted rows along the rows, transposed, as expert_wgrad_fp8 takes them.

    offsets [E + 1]: the experts' rows.  Sorted row r is x[r], or x[rows[r]] with
    rows (plan.tokens).  Returns (qt [C, cap], scale [cap/128, C]) with
    cap = fp8_columns(P, E); each expert's rows start at a multiple of 128, the
    columns that are no row hold zeros."""
    device = _gpu(x, "quantize_fp8_columns")
    ld = _matrix(x, "x")
    f8 = _f8_code(dtype)
    _ints(offsets, None, "offsets", device)
    if rows is not None:
        _ints(rows, None, "rows", device)
    R, C = x.shape
    P = R if rows is None else rows.numel()
    E = offsets.numel() - 1
    cap = fp8_columns(P, E)
    qt = torch.empty((C, cap), dtype=dtype, device=device)
    s = torch.empty((cap // 128, C), dtype=torch.float32, device=device)
    _launch(device, "nsg_quantize_fp8_columns", lib().nsg_quantize_fp8_columns, x.data_ptr(), _DT[x.dtype], R, C, ld,
            offsets.data_ptr(), E, rows.data_ptr() if rows is not None else None, P, f8, qt.data_ptr(), s.data_ptr())
    return qt, s


def _operand(q: torch.Tensor, s: torch.Tensor, name: str, dims: int, device, kinds=("row", "tile")) -> int:
    """Check an operand of quantize_fp8's layout; its block code."""
    qs, ss = q.shape, s.shape
    if len(qs) != dims or q.dtype not in _F8 or not q.is_contiguous() or q.device != device:
        raise ValueError(f"{name} must be a contiguous {dims}-D float8_e4m3fn or float8_e5m2 tensor on one device")
    R, K = qs[-2], qs[-1]
    if K % FP8_BLOCK:
        raise ValueError(f"{name} needs rows padded to a multiple of {FP8_BLOCK}")
    if s.dtype is not torch.float32 or not s.is_contiguous() or s.device != device or len(ss) != dims or \
            ss[-2] * FP8_BLOCK != K or (dims == 3 and ss[0] != qs[0]):
        raise ValueError(f"the scales of {name} must be a contiguous float32 tensor [..., K/128, rows or tiles]")
    n = ss[-1]
    if "row" in kinds and n == R:
        return 0
    if "tile" in kinds and n == -(-R // FP8_BLOCK):
        return 1
    raise ValueError(f"the scales of {name} fit neither its rows nor its tiles")


def _product_out(out: Optional[torch.Tensor], shape, out_dtype, device):
    if out is None:
        if out_dtype not in _DT:
            raise TypeError(f"unsupported dtype {out_dtype}")
        return torch.empty(shape, dtype=out_dtype, device=device)
    if out.shape != shape or out.dtype not in _DT or not out.is_contiguous() or out.device != device:
        raise ValueError(f"out must be a contiguous float tensor of shape {tuple(shape)} on the operands' device")
    return out


def gemm_fp8_nt(qa: torch.Tensor, sa: torch.Tensor, qb: torch.Tensor, sb: torch.Tensor, out_dtype=torch.bfloat16,
                out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """A B^T of two 8-bit operands as quantize_fp8 returns them: qa [M, K] and qb
    [N, K], or batches [b, M, K] and [b, N, K]; either may have row or tile
    scales.  fp32 sums, one rounding to out_dtype; zeros for K = 0.

    Products are exact for float32.  For 16-bit outputs each 8 consecutive k add an
    error below 7 * 2^-13 of their largest product (the 8-bit matrix instructions):
    about 1e-5 of the result on normal values, more where large products cancel."""
    device = _gpu(qa, "gemm_fp8_nt")
    ab = _operand(qa, sa, "qa", 2 if qa.dim() == 2 else 3, device)
    bb = _operand(qb, sb, "qb", qa.dim(), device)
    if qa.shape[-1] != qb.shape[-1] or qa.shape[:-2] != qb.shape[:-2]:
        raise ValueError(f"operands {tuple(qa.shape)} and {tuple(qb.shape)} do not fit")
    M, K = qa.shape[-2:]
    N = qb.shape[-2]
    out = _product_out(out, (*qa.shape[:-2], M, N), out_dtype, device)
    if K == 0:  # an empty sum, which the C entry point leaves to its caller
        return out.zero_()
    _launch(device, "nsg_gemm_fp8_nt", lib().nsg_gemm_fp8_nt, _F8[qa.dtype], _F8[qb.dtype], _DT[out.dtype],
            qa.shape[0] if qa.dim() == 3 else 1, M, N, K, qa.data_ptr(), sa.data_ptr(), ab, qb.data_ptr(), sb.data_ptr(),
            bb, out.data_ptr())
    return out


def expert_gemm_fp8(qa: torch.Tensor, sa: torch.Tensor, qb: torch.Tensor, sb: torch.Tensor, offsets: torch.Tensor,
                    rows: Optional[torch.Tensor] = None, out_dtype=torch.bfloat16,
                    out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Each expert's product: out[r] = A[rows[r]] B_e^T for the sorted rows r of
    expert e (A[r] without rows), zeros behind offsets[E], where rows[r] is no row
    of A, and for K = 0.  qa [T, K] with row scales, qb [E, N, K]; offsets and
    rows: a plan's offsets and tokens.  Sums as gemm_fp8_nt's."""
    device = _gpu(qa, "expert_gemm_fp8")
    _operand(qa, sa, "qa", 2, device, ("row",))
    bb = _operand(qb, sb, "qb", 3, device)
    T, K = qa.shape
    E, N, Kb = qb.shape
    _ints(offsets, (E + 1,), "offsets", device)
    if rows is not None:
        _ints(rows, None, "rows", device)
    if K != Kb:
        raise ValueError(f"operands {tuple(qa.shape)} and {tuple(qb.shape)} do not fit")
    P = T if rows is None else rows.numel()
    out = _product_out(out, (P, N), out_dtype, device)
    if K == 0 or T == 0:  # empty sums, which the C entry point leaves to its caller
        return out.zero_()
    _launch(device, "nsg_expert_gemm_fp8", lib().nsg_expert_gemm_fp8, _F8[qa.dtype], _F8[qb.dtype], _DT[out.dtype], T, P,
            E, N, K, qa.data_ptr(), sa.data_ptr(), rows.data_ptr() if rows is not None else None, qb.data_ptr(),
            sb.data_ptr(), bb, offsets.data_ptr(), out.data_ptr())
    return out


def expert_wgrad_fp8(qa: torch.Tensor, sa: torch.Tensor, qb: torch.Tensor, sb: torch.Tensor, offsets: torch.Tensor,
                     out_dtype=torch.bfloat16, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The experts' weight gradients [E, N, K], the bucket muon_step takes: out[e]
    = dy_e^T x_e over expert e's rows, zeros for one without.  (qa [N, cap], sa)
    and (qb [K, cap], sb) are quantize_fp8_columns of dy and x with these offsets.
    Sums as gemm_fp8_nt's."""
    device = _gpu(qa, "expert_wgrad_fp8")
    _operand(qa, sa, "qa", 2, device, ("row",))
    _operand(qb, sb, "qb", 2, device, ("row",))
    _ints(offsets, None, "offsets", device)
    E = offsets.numel() - 1
    (N, cap), K = qa.shape, qb.shape[0]
    P = cap - FP8_BLOCK * E  # P .. P + 127 rows have this layout, at most NSG_MAX_ROWS
    if qb.shape[1] != cap or P < 0:
        raise ValueError(f"operands {tuple(qa.shape)} and {tuple(qb.shape)} do not fit {E} experts")
    out = _product_out(out, (E, N, K), out_dtype, device)
    _launch(device, "nsg_expert_wgrad_fp8", lib().nsg_expert_wgrad_fp8, _F8[qa.dtype], _F8[qb.dtype], _DT[out.dtype],
            max(P, min(P + FP8_BLOCK - 1, 1 << 25)), E, N, K, qa.data_ptr(), sa.data_ptr(), qb.data_ptr(), sb.data_ptr(), offsets.data_ptr(),
            out.data_ptr())
    return out


# ---------------------------------------------------------------------------
# Between token ids and the expert layer: the embedding, layer norm, the router
# with its balance loss, and their gradients
# ---------------------------------------------------------------------------

def _ids(t: torch.Tensor, name: str, device=None):
    if t.dtype not in (torch.int32, torch.int64) or not t.is_contiguous() or (device is not None and t.device != device):
        raise ValueError(f"{name} must be a contiguous int32 or int64 tensor on the input's device")


def _vectors(t: torch.Tensor, name: str, device=None):
    """t [..., C] as rows of C elements: (rows, C, pitch).  Two dimensions may have a pitch,
    more must be contiguous."""
    shape = t.shape
    if len(shape) < 2 or t.dtype not in _DT:
        raise ValueError(f"{name} must be a float16, bfloat16 or float32 tensor of rows")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on the input's device")
    C = shape[-1]
    if t.is_contiguous():
        return t.numel() // C if C else math.prod(shape[:-1]), C, C
    if len(shape) > 2:
        raise ValueError(f"{name} must be contiguous, or a matrix with unit column stride")
    return shape[0], C, _pitch(t, name)


def _like(t: torch.Tensor) -> torch.Tensor:
    """A packed tensor of t's shape and type."""
    return torch.empty_like(t) if t.is_contiguous() else t.new_empty(t.shape)


def _space(workspace: Optional[torch.Tensor], need: int, t: torch.Tensor) -> torch.Tensor:
    """A workspace of `need` bytes on t's device: the caller's where it is large enough."""
    if workspace is not None:
        check_workspace(workspace, t.device)
        if nbytes(workspace) >= need:
            return workspace
    return t.new_empty(need, dtype=torch.uint8)


@functools.lru_cache(maxsize=1024)
def _size_of(what: str, *args) -> int:
    """A workspace's size, which these numbers alone decide (the call is a tenth of a short launch's time)."""
    out = ctypes.c_size_t(0)
    _check(getattr(lib(), what)(*args, ctypes.byref(out)), what)
    return out.value


def embedding(ids: torch.Tensor, weight: torch.Tensor, scale: float = 1.0) -> torch.Tensor:
    """out[t] = scale * weight[ids[t]]: ids of any shape (int32 or int64), weight [V, C],
    out [*ids.shape, C] of weight's dtype (fp32 products, rounded once).  An id outside
    0 .. V - 1, such as -1 for padding, gives zeros.  V <= 2^20."""
    device = _gpu(weight, "embedding")
    if weight.dim() != 2:
        raise ValueError("weight must be [V, C]")
    V, C, ld = _vectors(weight, "weight")
    _ids(ids, "ids", device)
    out = weight.new_empty((*ids.shape, C))
    _launch(device, "nsg_embedding", lib().nsg_embedding, ids.data_ptr(), 8 * ids.element_size(), ids.numel(),
            weight.data_ptr(), _DT[weight.dtype], V, C, ld, float(scale), out.data_ptr())
    return out


def embedding_backward_workspace_size(T: int, V: int, C: int) -> int:
    return _size_of("nsg_embedding_backward_workspace_size", T, V, C)


def embedding_backward(dout: torch.Tensor, ids: torch.Tensor, num_embeddings: int, scale: float = 1.0,
                       out: Optional[torch.Tensor] = None, accumulate: bool = False,
                       workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The gradient of embedding: dW [num_embeddings, C] of dout's dtype (or `out`, of any
    dtype), dW[v] = scale * the sum of dout[t] over the tokens with ids[t] = v; fp32 sums,
    rounded once.  dout [*ids.shape, C].

    With `accumulate` the sums are added to what `out` holds, and rows without tokens are
    left alone.  `workspace`: a uint8 tensor of embedding_backward_workspace_size(T, V, C)
    bytes (allocated if not given)."""
    device = _gpu(dout, "embedding_backward")
    _ids(ids, "ids", device)
    if dout.shape[:-1] != ids.shape:
        raise ValueError(f"dout must have shape [*{tuple(ids.shape)}, C]")
    T = ids.numel()
    C, ld = _vectors(dout if dout.dim() > 1 else dout.unsqueeze(0), "dout")[1:]
    V = int(num_embeddings)
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    if out is None:
        out = dout.new_empty((V, C))
    elif out.shape != (V, C) or out.dtype not in _DT or not out.is_contiguous() or out.device != device:
        raise ValueError(f"out must be a contiguous float tensor of shape {(V, C)} on the input's device")
    ws = _space(workspace, embedding_backward_workspace_size(T, V, C), dout)
    _launch(device, "nsg_embedding_backward", lib().nsg_embedding_backward, dout.data_ptr(), _DT[dout.dtype], T, C, ld,
            ids.data_ptr(), 8 * ids.element_size(), V, float(scale), out.data_ptr(), _DT[out.dtype], 1 if accumulate else 0,
            ws.data_ptr(), nbytes(ws))
    return out


def _norm_weight(t: torch.Tensor, name: str, C: int, device) -> int:
    """The dtype code of layer norm's weight or bias."""
    if t.shape != (C,) or t.dtype not in _DT or not t.is_contiguous() or t.device != device:
        raise ValueError(f"{name} must be a contiguous float tensor of shape {(C,)} on the input's device")
    return _DT[t.dtype]


def layer_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None, eps: float = 1e-5):
    """Layer norm over the last dimension of x [..., C]: (y, stats) with
    y = (x - mean) * rstd * weight + bias of x's dtype and stats [2, R] float32 the R rows'
    means and rstd = 1 / sqrt(var + eps), which layer_norm_backward takes.  weight and
    bias [C]: of one dtype, float32 or another; None for 1 and 0.  fp32 sums: a row's and
    that of its squared differences must not overflow."""
    device = _gpu(x, "layer_norm")
    R, C, ld = _vectors(x, "x")
    code = NSG_F32
    if weight is not None:
        code = _norm_weight(weight, "weight", C, device)
    if bias is not None:
        if weight is not None and bias.dtype != weight.dtype:
            raise ValueError("weight and bias must have one dtype")
        code = _norm_weight(bias, "bias", C, device)
    y = _like(x)
    stats = x.new_empty((2, R), dtype=torch.float32)
    _launch(device, "nsg_layer_norm", lib().nsg_layer_norm, x.data_ptr(), _DT[x.dtype], R, C, ld,
            weight.data_ptr() if weight is not None else None, bias.data_ptr() if bias is not None else None, code, float(eps),
            y.data_ptr(), stats.data_ptr())
    return y, stats


def layer_norm_backward_workspace_size(R: int, C: int) -> int:
    return _size_of("nsg_layer_norm_backward_workspace_size", R, C)


def layer_norm_backward(dy: torch.Tensor, x: torch.Tensor, stats: torch.Tensor, weight: Optional[torch.Tensor] = None,
                        weight_grad: bool = True, bias_grad: bool = True, workspace: Optional[torch.Tensor] = None):
    """The gradient of layer_norm for dy: (dx, dweight, dbias), dx of x's dtype, dweight and
    dbias [C] of weight's (float32 without a weight), None where weight_grad or bias_grad
    is false.  fp32 sums, rounded once.  `workspace`: a uint8 tensor of
    layer_norm_backward_workspace_size(R, C) bytes (allocated if not given)."""
    device = _gpu(x, "layer_norm_backward")
    R, C, ldx = _vectors(x, "x")
    lddy = _vectors(dy, "dy", device)[2]
    if dy.shape != x.shape or dy.dtype != x.dtype:
        raise ValueError("dy must have x's shape and dtype")
    if stats.shape != (2, R) or stats.dtype != torch.float32 or not stats.is_contiguous() or stats.device != device:
        raise ValueError(f"stats must be a contiguous float32 tensor of shape {(2, R)} on the input's device")
    code = NSG_F32 if weight is None else _norm_weight(weight, "weight", C, device)
    row = (lambda: torch.empty_like(weight)) if weight is not None else (lambda: x.new_empty(C, dtype=torch.float32))
    dx = _like(x)
    dweight = row() if weight_grad else None
    dbias = row() if bias_grad else None
    ws = None
    if weight_grad or bias_grad:
        ws = _space(workspace, layer_norm_backward_workspace_size(R, C), x)
    _launch(device, "nsg_layer_norm_backward", lib().nsg_layer_norm_backward, dy.data_ptr(), lddy, x.data_ptr(), ldx, _DT[x.dtype],
            R, C, stats.data_ptr(), weight.data_ptr() if weight is not None else None, code, dx.data_ptr(),
            dweight.data_ptr() if weight_grad else None, dbias.data_ptr() if bias_grad else None,
            ws.data_ptr() if ws is not None else None, nbytes(ws) if ws is not None else 0)
    return dx, dweight, dbias


class Routing(NamedTuple):
    """What expert_route decides.

    ids [T, k] int32, largest first, -1 for none (expert_sort drops it); weights [T, k]
    float32.  With the balance loss: counts [E + 1] int32, the choices of each expert
    and the number of tokens with a choice; probs [E] float32, the mean over these tokens
    of their probabilities; loss, a float32 scalar."""
    ids: torch.Tensor
    weights: torch.Tensor
    counts: Optional[torch.Tensor]
    probs: Optional[torch.Tensor]
    loss: Optional[torch.Tensor]


_SCORES = {"softmax": 0, "sigmoid": 1}


def _score_code(score) -> int:
    if score not in _SCORES:
        raise ValueError("score must be 'softmax' or 'sigmoid'")
    return _SCORES[score]


def expert_route_workspace_size(T: int, num_experts: int) -> int:
    return _size_of("nsg_expert_route_workspace_size", T, num_experts)


def expert_route(logits: torch.Tensor, k: int, score: str = "softmax", bias: Optional[torch.Tensor] = None,
                 mask: Optional[torch.Tensor] = None, normalize: bool = True, scale: float = 1.0, balance: bool = False,
                 workspace: Optional[torch.Tensor] = None) -> Routing:
    """Each token's k experts and their weights, from logits [T, E].

    s = softmax(logits) or sigmoid(logits).  The k largest logits are chosen, with `bias`
    (float32 [E]) the k largest s + bias, compared in 64 bits; equal ones go to the lower
    index.  weights = scale * s, with `normalize` divided by the sum of the token's chosen
    s.  A logit of -inf or NaN is never chosen and a token whose `mask` (bool [T]) is
    False chooses nothing: ids -1, weights 0.

    With `balance` also counts, probs and loss = E / (k N) * sum(counts * probs) over the
    N tokens with a choice (see Routing).  `workspace`, for the loss: a uint8 tensor of
    expert_route_workspace_size(T, E) bytes (allocated if not given).  k <= 64, E <= 1024."""
    device = _gpu(logits, "expert_route")
    if logits.dim() != 2:
        raise ValueError("logits must be [T, E]")
    T, E, ld = _vectors(logits, "logits")
    code = _score_code(score)
    k = int(k)
    if bias is not None and (bias.dtype != torch.float32 or bias.shape != (E,) or not bias.is_contiguous() or bias.device != device):
        raise ValueError("bias must be a contiguous float32 [E] tensor on the input's device")
    if mask is not None and (mask.dtype not in (torch.bool, torch.uint8) or mask.shape != (T,) or not mask.is_contiguous()
                             or mask.device != device):
        raise ValueError("mask must be a contiguous bool [T] tensor on the input's device")
    if not 1 <= k <= min(E, 64):
        raise ValueError("k must lie in 1 .. min(E, 64)")
    ids = logits.new_empty((T, k), dtype=torch.int32)
    weights = logits.new_empty((T, k), dtype=torch.float32)
    counts = probs = loss = ws = None
    if balance:
        counts = logits.new_empty(E + 1, dtype=torch.int32)
        probs = logits.new_empty(E, dtype=torch.float32)
        loss = logits.new_empty((), dtype=torch.float32)
        ws = _space(workspace, expert_route_workspace_size(T, E), logits)
    _launch(device, "nsg_expert_route", lib().nsg_expert_route, logits.data_ptr(), _DT[logits.dtype], T, E, ld, k, code,
            bias.data_ptr() if bias is not None else None, mask.data_ptr() if mask is not None else None,
            1 if normalize else 0, float(scale), ids.data_ptr(), weights.data_ptr(), counts.data_ptr() if balance else None,
            probs.data_ptr() if balance else None, loss.data_ptr() if balance else None, ws.data_ptr() if balance else None,
            nbytes(ws) if balance else 0)
    return Routing(ids, weights, counts, probs, loss)


def expert_route_backward(logits: torch.Tensor, ids: torch.Tensor, dweights: Optional[torch.Tensor] = None,
                          score: str = "softmax", normalize: bool = True, scale: float = 1.0,
                          counts: Optional[torch.Tensor] = None, balance: float = 1.0,
                          dloss: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The gradient of expert_route with respect to the logits, of their dtype [T, E].

    ids as expert_route gave them; dweights [T, k] float32 is the weights' gradient.  With
    counts (of expert_route, or their sum over several processes) the balance loss's is
    added: `balance` times it, times dloss where that (a float32 scalar) is given.
    counts are constants.  A token without a choice gets zeros."""
    device = _gpu(logits, "expert_route_backward")
    if logits.dim() != 2:
        raise ValueError("logits must be [T, E]")
    T, E, ld = _vectors(logits, "logits")
    code = _score_code(score)
    if ids.dim() != 2 or ids.shape[0] != T:
        raise ValueError("ids must be [T, k]")
    _ints(ids, None, "ids", device)
    if dweights is not None and (dweights.dtype != torch.float32 or dweights.shape != ids.shape or not dweights.is_contiguous()
                                 or dweights.device != device):
        raise ValueError("dweights must be a contiguous float32 [T, k] tensor on the input's device")
    if counts is not None:
        _ints(counts, (E + 1,), "counts", device)
    if dloss is not None and (counts is None or dloss.dtype != torch.float32 or dloss.numel() != 1 or dloss.device != device):
        raise ValueError("dloss must be a float32 scalar on the input's device, with counts")
    dlogits = _like(logits)
    _launch(device, "nsg_expert_route_backward", lib().nsg_expert_route_backward, logits.data_ptr(), _DT[logits.dtype], T, E, ld,
            ids.shape[1], code, 1 if normalize else 0, float(scale), ids.data_ptr(),
            dweights.data_ptr() if dweights is not None else None, counts.data_ptr() if counts is not None else None,
            float(balance), dloss.data_ptr() if dloss is not None else None, dlogits.data_ptr())
    return dlogits
