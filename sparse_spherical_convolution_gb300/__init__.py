"""GB300 (sm_103a) DISCO convolution on the sphere: Python binding of the C ABI.

The binding only marshals arguments: every step runs in the CUDA library
``_build/libdisco_gb300_<arch>.so`` (built by ``build.py``).  If the library
is missing, importing the functions raises; there is no fallback.

The functions carry the names of the C ABI (``include/disco.h``) and take
torch tensors for device memory; torch's current CUDA stream is used unless a
stream is given.
"""
from __future__ import annotations

import ctypes
import os
import struct

from . import build as _build_mod

__all__ = [
    "DiscoError", "disco_grid", "disco_basis", "disco_run", "disco_psi", "Psi",
    "disco_version", "disco_build_flags", "DISCO_BUILD_DEBUG_BOUNDS", "DISCO_ERR_DEVICE_BOUNDS",
    "disco_last_error", "disco_psi_workspace_bytes", "disco_psi_plan",
    "disco_build_psi_kpacked", "disco_psi_export_kpacked", "disco_check_wait_timeout", "disco_fwd", "disco_bwd",
    "disco_host_workspace_bytes", "disco_fwd_host", "disco_bwd_host",
    "disco_fused_conv_workspace_bytes",
    "disco_fused_conv", "disco_fused_conv_bwd_input_workspace_bytes", "disco_fused_conv_bwd_input",
    "disco_fused_conv_bwd_input_noalloc", "disco_fused_conv_bwd_weight_workspace_bytes",
    "disco_fused_conv_bwd_weight", "disco_device_status", "disco_check_sched_takeover", "library_path",
    "load_library", "EXPORTED_SYMBOLS", "NOALLOC_SCRATCH_BYTES",
    "DISCO_F32", "DISCO_BF16", "DISCO_F16", "dtype_code", "disco_rms_norm", "disco_rms_norm_bwd_workspace_bytes",
    "disco_rms_norm_bwd", "disco_dequant_e4m3", "disco_grad_tensor", "disco_grads", "disco_grad_plan", "GradPlan",
    "disco_grad_workspace_bytes", "disco_grad_norm", "disco_grad_clip", "disco_grad_norm_clip",
    "DISCO_SILU", "DISCO_GELU",
    "disco_quant_i8", "disco_matmul_i8_workspace_bytes", "disco_matmul_i8",
    "disco_matmul_i8_bwd_input_workspace_bytes", "disco_matmul_i8_bwd_input",
    "disco_matmul_i8_bwd_weight_workspace_bytes", "disco_matmul_i8_bwd_weight", "disco_glu", "disco_glu_bwd",
]

NOALLOC_SCRATCH_BYTES = 64 << 20

DISCO_F32, DISCO_BF16, DISCO_F16 = 0, 1, 2

DISCO_SILU, DISCO_GELU = 0, 1

EXPORTED_SYMBOLS = [
    "disco_version", "disco_last_error", "disco_psi_workspace_bytes", "disco_psi_plan",
    "disco_build_psi_kpacked", "disco_fwd", "disco_bwd", "disco_fused_conv_workspace_bytes",
    "disco_fused_conv", "disco_fused_conv_bwd_input_workspace_bytes", "disco_fused_conv_bwd_input",
    "disco_fused_conv_bwd_input_noalloc", "disco_fused_conv_bwd_weight_workspace_bytes",
    "disco_fused_conv_bwd_weight", "disco_device_status", "disco_psi_export_kpacked",
    "disco_check_wait_timeout", "disco_host_workspace_bytes", "disco_fwd_host", "disco_bwd_host",
    "disco_check_sched_takeover", "disco_build_flags", "disco_rms_norm", "disco_rms_norm_bwd_workspace_bytes",
    "disco_rms_norm_bwd", "disco_dequant_e4m3", "disco_grad_plan", "disco_grad_workspace_bytes", "disco_grad_norm",
    "disco_grad_clip", "disco_grad_norm_clip",
    "disco_quant_i8", "disco_matmul_i8_workspace_bytes", "disco_matmul_i8",
    "disco_matmul_i8_bwd_input_workspace_bytes", "disco_matmul_i8_bwd_input",
    "disco_matmul_i8_bwd_weight_workspace_bytes", "disco_matmul_i8_bwd_weight", "disco_glu", "disco_glu_bwd",
]


class DiscoError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"disco status {status}: {message}")
        self.status = status


class disco_grid(ctypes.Structure):
    _fields_ = [("nlat", ctypes.c_int32), ("nlon", ctypes.c_int32), ("poles", ctypes.c_int32)]


class disco_basis(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("n_radial", ctypes.c_int32), ("cutoff", ctypes.c_double)]


class disco_run(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("ho", "hi", "D", "hoff", "e0", "len", "npair", "anti")]


_PSI_ARRAYS = ["row_ptr", "idx", "val", "csr_row_ptr", "csr_col", "csr_val", "run_ptr", "runs",
               "trun_ptr", "truns", "hval", "row_order", "ftab_off", "ftab", "grp_ptr", "grp", "gtab",
               "ftab_h", "gtab_h"]


class disco_psi(ctypes.Structure):
    _fields_ = [("grid_in", disco_grid), ("grid_out", disco_grid), ("basis", disco_basis),
                ("K", ctypes.c_int32), ("K_pad", ctypes.c_int32), ("s", ctypes.c_int32),
                ("max_row", ctypes.c_int32), ("nnz", ctypes.c_int64), ("nnz_csr", ctypes.c_int64),
                ("nruns", ctypes.c_int64), ("nhval", ctypes.c_int64), ("nftab", ctypes.c_int64),
                ("ngrp", ctypes.c_int32), ("grp_max", ctypes.c_int32), ("ngrp_ent", ctypes.c_int64),
                ("ngtab", ctypes.c_int64), ("bytes", ctypes.c_size_t)] + \
               [(n, ctypes.c_void_p) for n in _PSI_ARRAYS]


class disco_grad_tensor(ctypes.Structure):
    _fields_ = [("grad", ctypes.c_void_p), ("out", ctypes.c_void_p), ("n", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32)]


class disco_grads(ctypes.Structure):
    _fields_ = [("tensors", ctypes.POINTER(disco_grad_tensor)), ("count", ctypes.c_int32),
                ("has_out", ctypes.c_int32), ("numel", ctypes.c_int64), ("device", ctypes.c_int32),
                ("in_place", ctypes.c_int32)]


_lib = None


def library_path() -> str:
    """The product library, or its bounds-checked build when the environment
    sets DISCO_GB300_BOUNDS_CHECKED=1 (a diagnostic build, see build.py)."""
    if os.environ.get("DISCO_GB300_BOUNDS_CHECKED") == "1":
        return _build_mod.LIB_BOUNDS
    return _build_mod.LIB


def load_library():
    """Loads the built library; raises if it is missing (no fallback path)."""
    global _lib
    if _lib is not None:
        return _lib
    path = library_path()
    if not os.path.exists(path):
        raise RuntimeError(f"DISCO CUDA library not built: {path} is missing "
                           "(run `python -m sparse_spherical_convolution_gb300.build`)")
    lib = ctypes.CDLL(path)
    P, I32, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    PG, PB, PP = ctypes.POINTER(disco_grid), ctypes.POINTER(disco_basis), ctypes.POINTER(disco_psi)
    lib.disco_version.restype = I32
    lib.disco_version.argtypes = []
    lib.disco_build_flags.restype = I32
    lib.disco_build_flags.argtypes = []
    lib.disco_last_error.restype = ctypes.c_char_p
    lib.disco_last_error.argtypes = []
    lib.disco_psi_workspace_bytes.restype = ctypes.c_int
    lib.disco_psi_workspace_bytes.argtypes = [PG, PG, PB, ctypes.POINTER(SZ)]
    lib.disco_psi_plan.restype = ctypes.c_int
    lib.disco_psi_plan.argtypes = [PG, PG, PB, P, SZ, P, PP]
    lib.disco_build_psi_kpacked.restype = ctypes.c_int
    lib.disco_build_psi_kpacked.argtypes = [PP, P, SZ, P, SZ, P]
    lib.disco_host_workspace_bytes.restype = SZ
    lib.disco_host_workspace_bytes.argtypes = [PP, I32, I32, I32, ctypes.c_int]
    for nm in ("disco_fwd_host", "disco_bwd_host"):
        getattr(lib, nm).restype = ctypes.c_int
        getattr(lib, nm).argtypes = [PP, P, P, I32, I32, ctypes.c_int, P, SZ, P]
    lib.disco_check_wait_timeout.restype = ctypes.c_int
    lib.disco_check_wait_timeout.argtypes = [ctypes.c_uint32, P]
    lib.disco_check_sched_takeover.restype = ctypes.c_int
    lib.disco_check_sched_takeover.argtypes = []
    lib.disco_psi_export_kpacked.restype = ctypes.c_int
    lib.disco_psi_export_kpacked.argtypes = [PP, P, P, P, I32, P]
    lib.disco_fwd.restype = ctypes.c_int
    lib.disco_fwd.argtypes = [PP, P, P, I32, I32, ctypes.c_int, P]
    lib.disco_bwd.restype = ctypes.c_int
    lib.disco_bwd.argtypes = [PP, P, P, I32, I32, ctypes.c_int, P]
    lib.disco_fused_conv_workspace_bytes.restype = SZ
    lib.disco_fused_conv_workspace_bytes.argtypes = [PP, I32, I32, I32, ctypes.c_int]
    lib.disco_fused_conv.restype = ctypes.c_int
    lib.disco_fused_conv.argtypes = [PP, P, P, P, I32, I32, I32, ctypes.c_int, P, SZ, P]
    lib.disco_fused_conv_bwd_input_workspace_bytes.restype = SZ
    lib.disco_fused_conv_bwd_input_workspace_bytes.argtypes = [PP, I32, I32, ctypes.c_int]
    lib.disco_fused_conv_bwd_input.restype = ctypes.c_int
    lib.disco_fused_conv_bwd_input.argtypes = [PP, P, P, P, I32, I32, I32, ctypes.c_int, P, SZ, P]
    lib.disco_fused_conv_bwd_input_noalloc.restype = ctypes.c_int
    lib.disco_fused_conv_bwd_input_noalloc.argtypes = [PP, P, P, P, I32, I32, I32, ctypes.c_int, P]
    lib.disco_fused_conv_bwd_weight_workspace_bytes.restype = SZ
    lib.disco_fused_conv_bwd_weight_workspace_bytes.argtypes = [PP, I32, I32, I32, ctypes.c_int]
    lib.disco_fused_conv_bwd_weight.restype = ctypes.c_int
    lib.disco_fused_conv_bwd_weight.argtypes = [PP, P, P, P, I32, I32, I32, ctypes.c_int, P, SZ, P]
    I64, F32 = ctypes.c_int64, ctypes.c_float
    PGR = ctypes.POINTER(disco_grads)
    lib.disco_rms_norm.restype = ctypes.c_int
    lib.disco_rms_norm.argtypes = [P, P, P, F32, P, P, P, P, I32, I32, I32, I64, ctypes.c_int, P]
    lib.disco_rms_norm_bwd_workspace_bytes.restype = SZ
    lib.disco_rms_norm_bwd_workspace_bytes.argtypes = [I32, I32, I64, ctypes.c_int]
    lib.disco_rms_norm_bwd.restype = ctypes.c_int
    lib.disco_rms_norm_bwd.argtypes = [P, P, P, P, F32, P, P, I32, I32, I64, ctypes.c_int, P, SZ, P]
    lib.disco_dequant_e4m3.restype = ctypes.c_int
    lib.disco_dequant_e4m3.argtypes = [P, P, P, I32, I32, I32, I64, ctypes.c_int, P]
    lib.disco_grad_plan.restype = ctypes.c_int
    lib.disco_grad_plan.argtypes = [ctypes.POINTER(disco_grad_tensor), I32, PGR]
    lib.disco_grad_workspace_bytes.restype = SZ
    lib.disco_grad_workspace_bytes.argtypes = [PGR]
    lib.disco_grad_norm.restype = ctypes.c_int
    lib.disco_grad_norm.argtypes = [PGR, F32, P, P, SZ, P]
    lib.disco_grad_clip.restype = ctypes.c_int
    lib.disco_grad_clip.argtypes = [PGR, F32, F32, P, P]
    lib.disco_grad_norm_clip.restype = ctypes.c_int
    lib.disco_grad_norm_clip.argtypes = [PGR, F32, F32, P, P, SZ, P]
    lib.disco_quant_i8.restype = ctypes.c_int
    lib.disco_quant_i8.argtypes = [P, P, P, I32, I32, I64, ctypes.c_int, P]
    for nm, ptrs in (("disco_matmul_i8", 5), ("disco_matmul_i8_bwd_input", 4), ("disco_matmul_i8_bwd_weight", 4)):
        getattr(lib, nm + "_workspace_bytes").restype = SZ
        getattr(lib, nm + "_workspace_bytes").argtypes = [I32, I32, I32, I64, ctypes.c_int]
        getattr(lib, nm).restype = ctypes.c_int
        getattr(lib, nm).argtypes = [P] * ptrs + [I32, I32, I32, I64, ctypes.c_int, P, SZ, P]
    lib.disco_glu.restype = ctypes.c_int
    lib.disco_glu.argtypes = [P, P, P, P, P, P, ctypes.c_int, I32, I32, I64, ctypes.c_int, P]
    lib.disco_glu_bwd.restype = ctypes.c_int
    lib.disco_glu_bwd.argtypes = [P, P, P, P, ctypes.c_int, I32, I32, I64, ctypes.c_int, P]
    lib.disco_device_status.restype = ctypes.c_int
    lib.disco_device_status.argtypes = [ctypes.POINTER(I32), I32]
    _lib = lib
    return lib


def _check(status: int):
    if status != 0:
        raise DiscoError(status, load_library().disco_last_error().decode())


_torch = None          # torch, its current-device and raw-stream calls and the type codes, from the first use on
_device = _raw_stream = None
_CODES = {}


def _runtime():
    """Imports torch (the module itself loads without it)."""
    global _torch, _device, _raw_stream
    import torch
    _CODES.update({torch.float32: DISCO_F32, torch.bfloat16: DISCO_BF16, torch.float16: DISCO_F16})
    _device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    _raw_stream = (getattr(torch._C, "_cuda_getCurrentRawStream", None) or
                   (lambda device: torch.cuda.current_stream(device).cuda_stream))
    _torch = torch
    return torch


def _stream(stream):
    if stream is None:
        if _torch is None:
            _runtime()
        return _raw_stream(_torch.cuda.current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def dtype_code(dtype) -> int:
    """The library's code (DISCO_F32, DISCO_BF16, DISCO_F16) of a torch dtype."""
    if _torch is None:
        _runtime()
    code = _CODES.get(dtype)
    if code is None:
        raise DiscoError(-2, f"unsupported dtype {dtype}")
    return code


def _dtype(t) -> int:
    return dtype_code(t.dtype)


def _ptr(t):
    if t is None:
        return None
    if not t.is_contiguous():
        raise DiscoError(-1, "tensors must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _dev(t, name: str, numel: int, dtype=None):
    """Pointer of a device tensor after checking it: on the current CUDA
    device, contiguous, `numel` elements, and of `dtype` when given.  A
    mismatch raises DiscoError(-1) before any call into the library."""
    import torch
    if t is None:
        raise DiscoError(-1, f"{name} is None")
    if not t.is_cuda or t.device.index != torch.cuda.current_device():
        raise DiscoError(-1, f"{name} must be a tensor on the current CUDA device, got {t.device}")
    if dtype is not None and t.dtype != dtype:
        raise DiscoError(-1, f"{name} has dtype {t.dtype}, the call's dtype is {dtype}")
    if t.numel() != int(numel):
        raise DiscoError(-1, f"{name} has {t.numel()} elements, the call needs {int(numel)}")
    return _ptr(t)


def _host(t, name: str, numel: int, dtype=None):
    """Pointer of a host (CPU) tensor after the same checks as _dev."""
    if t is None or t.is_cuda:
        raise DiscoError(-1, f"{name} must be a CPU tensor")
    if dtype is not None and t.dtype != dtype:
        raise DiscoError(-1, f"{name} has dtype {t.dtype}, the call's dtype is {dtype}")
    if t.numel() != int(numel):
        raise DiscoError(-1, f"{name} has {t.numel()} elements, the call needs {int(numel)}")
    return _ptr(t)


def _ws(t, name: str = "workspace"):
    """(pointer, bytes) of an optional device workspace."""
    import torch
    if t is None:
        return None, 0
    if not t.is_cuda or t.get_device() != torch.cuda.current_device():
        raise DiscoError(-1, f"{name} must be a tensor on the current CUDA device")
    return _ptr(t), t.nbytes


def _sizes(psi):
    """(H_in*W_in, K*H_out*W_out, H_out*W_out, K) of a built psi."""
    pin = psi.grid_in.nlat * psi.grid_in.nlon
    pout = psi.grid_out.nlat * psi.grid_out.nlon
    return pin, psi.K * pout, pout, psi.K


# ------------------------------------------------------------------ ABI calls

def disco_version() -> int:
    return load_library().disco_version()


DISCO_BUILD_DEBUG_BOUNDS = 1
DISCO_ERR_DEVICE_BOUNDS = -8


def disco_build_flags() -> int:
    """DISCO_BUILD_DEBUG_BOUNDS when the loaded library is the bounds-checked build."""
    return load_library().disco_build_flags()


def disco_last_error() -> str:
    return load_library().disco_last_error().decode()


def _grid(g) -> disco_grid:
    return g if isinstance(g, disco_grid) else disco_grid(*[int(v) for v in g])


def _basis(kind, n_radial=None, cutoff=None) -> disco_basis:
    if isinstance(kind, disco_basis):
        return kind
    return disco_basis(int(kind), int(n_radial), float(cutoff))


def disco_psi_workspace_bytes(grid_in, grid_out, basis) -> int:
    n = ctypes.c_size_t()
    _check(load_library().disco_psi_workspace_bytes(
        ctypes.byref(_grid(grid_in)), ctypes.byref(_grid(grid_out)), ctypes.byref(basis),
        ctypes.byref(n)))
    return n.value


def disco_psi_plan(grid_in, grid_out, basis, workspace, stream=None) -> disco_psi:
    psi = disco_psi()
    _check(load_library().disco_psi_plan(
        ctypes.byref(_grid(grid_in)), ctypes.byref(_grid(grid_out)), ctypes.byref(basis),
        *_ws(workspace), _stream(stream), ctypes.byref(psi)))
    return psi


def disco_build_psi_kpacked(psi: disco_psi, buffer, workspace, stream=None) -> None:
    _check(load_library().disco_build_psi_kpacked(
        ctypes.byref(psi), *_ws(buffer, "buffer"), *_ws(workspace), _stream(stream)))


def disco_host_workspace_bytes(psi: disco_psi, B: int, C: int, forward: bool, dtype=DISCO_BF16) -> int:
    return load_library().disco_host_workspace_bytes(ctypes.byref(psi), B, C, 1 if forward else 0, dtype)


def disco_fwd_host(psi: disco_psi, x_host, X_host, B: int, C: int, workspace, stream=None) -> None:
    """x_host, X_host: CPU tensors (pinned for overlap); workspace: device."""
    pin, pX, _, _ = _sizes(psi)
    dt = x_host.dtype
    xp = _host(x_host, "x_host", B * C * pin, dt)
    Xp = _host(X_host, "X_host", B * C * pX, dt)
    wp, wn = _ws(workspace)
    _check(load_library().disco_fwd_host(ctypes.byref(psi), xp, Xp, B, C, _dtype(x_host), wp, wn,
                                         _stream(stream)))


def disco_bwd_host(psi: disco_psi, G_host, gx_host, B: int, C: int, workspace, stream=None) -> None:
    """G_host, gx_host: CPU tensors (pinned for overlap); workspace: device."""
    pin, pX, _, _ = _sizes(psi)
    dt = G_host.dtype
    Gp = _host(G_host, "G_host", B * C * pX, dt)
    gp = _host(gx_host, "gx_host", B * C * pin, dt)
    wp, wn = _ws(workspace)
    _check(load_library().disco_bwd_host(ctypes.byref(psi), Gp, gp, B, C, _dtype(G_host), wp, wn,
                                         _stream(stream)))


def disco_check_wait_timeout(limit: int, stream=None) -> None:
    _check(load_library().disco_check_wait_timeout(limit, _stream(stream)))


def disco_check_sched_takeover() -> None:
    """Walks the scheduler protocol, then leaves a foreign tag in the next launch's words (diagnostic)."""
    _check(load_library().disco_check_sched_takeover())


def disco_psi_export_kpacked(psi: disco_psi, pack_idx, pack_val, pack_count, nbr_pad: int,
                             stream=None) -> None:
    import torch
    H = psi.grid_out.nlat
    ip = _dev(pack_idx, "pack_idx", H * nbr_pad * 2, torch.int64)
    vp = _dev(pack_val, "pack_val", H * nbr_pad * psi.K_pad, torch.float32)
    cp = _dev(pack_count, "pack_count", H, torch.int64)
    _check(load_library().disco_psi_export_kpacked(ctypes.byref(psi), ip, vp, cp, nbr_pad, _stream(stream)))


def disco_fwd(psi: disco_psi, x, X, B: int, C: int, stream=None) -> None:
    pin, pX, _, _ = _sizes(psi)
    xp = _dev(x, "x", B * C * pin)
    Xp = _dev(X, "X", B * C * pX, x.dtype)
    _check(load_library().disco_fwd(ctypes.byref(psi), xp, Xp, B, C, _dtype(x), _stream(stream)))


def disco_bwd(psi: disco_psi, G, gx, B: int, C: int, stream=None) -> None:
    pin, pX, _, _ = _sizes(psi)
    Gp = _dev(G, "G", B * C * pX)
    gp = _dev(gx, "gx", B * C * pin, G.dtype)
    _check(load_library().disco_bwd(ctypes.byref(psi), Gp, gp, B, C, _dtype(G), _stream(stream)))


def disco_fused_conv_workspace_bytes(psi: disco_psi, B: int, Cin: int, Cout: int, dtype=DISCO_BF16) -> int:
    return load_library().disco_fused_conv_workspace_bytes(ctypes.byref(psi), B, Cin, Cout, dtype)


def disco_fused_conv(psi: disco_psi, x, W, y, B: int, Cin: int, Cout: int, workspace=None,
                     stream=None) -> None:
    pin, _, pout, K = _sizes(psi)
    xp = _dev(x, "x", B * Cin * pin)
    Wp = _dev(W, "W", Cout * Cin * K, x.dtype)
    yp = _dev(y, "y", B * Cout * pout, x.dtype)
    wp, wn = _ws(workspace)
    _check(load_library().disco_fused_conv(ctypes.byref(psi), xp, Wp, yp, B, Cin, Cout, _dtype(x), wp, wn,
                                           _stream(stream)))


def disco_fused_conv_bwd_input_workspace_bytes(psi: disco_psi, B: int, Cin: int, dtype=DISCO_BF16) -> int:
    return load_library().disco_fused_conv_bwd_input_workspace_bytes(ctypes.byref(psi), B, Cin, dtype)


def disco_fused_conv_bwd_input(psi: disco_psi, dy, W, gx, B: int, Cin: int, Cout: int,
                               workspace, stream=None) -> None:
    pin, _, pout, K = _sizes(psi)
    dp = _dev(dy, "dy", B * Cout * pout)
    Wp = _dev(W, "W", Cout * Cin * K, dy.dtype)
    gp = _dev(gx, "gx", B * Cin * pin, dy.dtype)
    wp, wn = _ws(workspace)
    _check(load_library().disco_fused_conv_bwd_input(ctypes.byref(psi), dp, Wp, gp, B, Cin, Cout, _dtype(dy),
                                                     wp, wn, _stream(stream)))


def disco_fused_conv_bwd_weight_workspace_bytes(psi: disco_psi, B: int, Cin: int, Cout: int,
                                                 dtype=DISCO_BF16) -> int:
    return load_library().disco_fused_conv_bwd_weight_workspace_bytes(ctypes.byref(psi), B, Cin, Cout, dtype)


def disco_fused_conv_bwd_weight(psi: disco_psi, x, dy, dW, B: int, Cin: int, Cout: int,
                                workspace, stream=None) -> None:
    pin, _, pout, K = _sizes(psi)
    xp = _dev(x, "x", B * Cin * pin)
    dp = _dev(dy, "dy", B * Cout * pout, x.dtype)
    Wp = _dev(dW, "dW", Cout * Cin * K, x.dtype)
    wp, wn = _ws(workspace)
    _check(load_library().disco_fused_conv_bwd_weight(ctypes.byref(psi), xp, dp, Wp, B, Cin, Cout, _dtype(x),
                                                      wp, wn, _stream(stream)))


def disco_fused_conv_bwd_input_noalloc(psi: disco_psi, dy, W, gx, B: int, Cin: int, Cout: int,
                                       stream=None) -> None:
    """disco_fused_conv_bwd_input without a workspace argument: the library's
    fixed device scratch holds dX (see include/disco.h for limits and rules)."""
    pin, _, pout, K = _sizes(psi)
    dp = _dev(dy, "dy", B * Cout * pout)
    Wp = _dev(W, "W", Cout * Cin * K, dy.dtype)
    gp = _dev(gx, "gx", B * Cin * pin, dy.dtype)
    _check(load_library().disco_fused_conv_bwd_input_noalloc(
        ctypes.byref(psi), dp, Wp, gp, B, Cin, Cout, _dtype(dy), _stream(stream)))


def _groups(C: int, group: int) -> int:
    return -(-C // group) if 0 < group < C else 1


def _on(t, name: str) -> int:
    """The current CUDA device, which ``t`` has to be on."""
    if t is None or not t.is_cuda:
        _dev(t, name, 0)
    if _torch is None:
        _runtime()
    return _device()


def _in(t, name: str, numel: int, dtype, device: int):
    """Address of a device tensor after _dev's checks, None for None."""
    if t is None:
        return None
    if t.get_device() != device or t.dtype is not dtype or t.numel() != numel or not t.is_contiguous():
        return _dev(t, name, numel, dtype)
    return t.data_ptr()


def _q8(t, numel: int, device: int):
    """Address of an 8-bit tensor: float8_e4m3fn, or its bytes as uint8."""
    if t is None:
        return None
    if t.dtype not in (_torch.float8_e4m3fn, _torch.uint8):
        raise DiscoError(-1, f"q has dtype {t.dtype}, the call needs float8_e4m3fn or uint8")
    return _in(t, "q", numel, t.dtype, device)


def _bytes(t, name: str, device: int):
    """(address, bytes) of an optional device workspace."""
    if t is None:
        return None, 0
    if t.get_device() != device or not t.is_contiguous():
        return _ws(t, name)
    return t.data_ptr(), t.nbytes


def disco_rms_norm(x, residual, weight, eps: float, h, y, B: int, C: int, P: int, q=None, scale=None,
                   group: int = 0, stream=None) -> None:
    """h = x + residual, its root-mean-square norm over the C channels times
    weight in y, and y in 8 bits with scales in q and scale; see
    include/disco.h.  residual, weight, h, y, and q with scale may be None."""
    n, dev = B * C * P, _on(x, "x")
    dt = x.dtype
    _check((_lib or load_library()).disco_rms_norm(
        _in(x, "x", n, dt, dev), _in(residual, "residual", n, dt, dev), _in(weight, "weight", C, dt, dev), eps,
        _in(h, "h", n, dt, dev), _in(y, "y", n, dt, dev), _q8(q, n, dev),
        None if scale is None else _in(scale, "scale", B * _groups(C, group) * P, _torch.float32, dev), group, B, C, P,
        dtype_code(dt), _raw_stream(dev) if stream is None else _stream(stream)))


def disco_rms_norm_bwd_workspace_bytes(B: int, C: int, P: int, dtype=DISCO_BF16) -> int:
    return load_library().disco_rms_norm_bwd_workspace_bytes(B, C, P, dtype)


def disco_rms_norm_bwd(dy, h, weight, dh, eps: float, dx, dweight, B: int, C: int, P: int, workspace=None,
                       stream=None) -> None:
    """dx and dweight of disco_rms_norm from the stored h; weight, dh and
    dweight (with its workspace) may be None."""
    n, dev = B * C * P, _on(dy, "dy")
    dt = dy.dtype
    code = dtype_code(dt)
    wp, wn = _bytes(workspace, "workspace", dev)
    _check((_lib or load_library()).disco_rms_norm_bwd(
        _in(dy, "dy", n, dt, dev), _in(h, "h", n, dt, dev), _in(weight, "weight", C, dt, dev), _in(dh, "dh", n, dt, dev),
        eps, _in(dx, "dx", n, dt, dev), _in(dweight, "dweight", C, dt, dev), B, C, P, code, wp, wn,
        _raw_stream(dev) if stream is None else _stream(stream)))


def disco_dequant_e4m3(q, scale, x, B: int, C: int, P: int, group: int = 0, stream=None) -> None:
    """x = q * scale, the activation that disco_rms_norm's q and scale stand for."""
    n, dev = B * C * P, _on(q, "q")
    _check((_lib or load_library()).disco_dequant_e4m3(
        _q8(q, n, dev), _in(scale, "scale", B * _groups(C, group) * P, _torch.float32, dev),
        None if x is None else _in(x, "x", n, x.dtype, dev), group, B, C, P, -1 if x is None else dtype_code(x.dtype),
        _raw_stream(dev) if stream is None else _stream(stream)))


def disco_grad_plan(grads, outs=None):
    """(disco_grads, host array) of a list of gradients and the tensors their
    clipped values go to (None: the norm alone; the same tensors: in place).
    The struct keeps the array it points to, and the tensors, alive."""
    grads = list(grads)
    outs = [None] * len(grads) if outs is None else list(outs)
    if len(outs) != len(grads):
        raise DiscoError(-1, f"{len(grads)} gradients and {len(outs)} outs")
    fields, dev = [], None
    for i, (g, o) in enumerate(zip(grads, outs)):
        if g is None:
            raise DiscoError(-1, f"gradient {i} is None")
        n, gp, op = g.numel(), None, None
        if n:  # a tensor without elements has no memory to check
            if dev is None:
                dev = _on(g, f"gradient {i}")
            gp = _in(g, "a gradient", n, g.dtype, dev)
            if o is not None:
                op = _in(o, "an out", n, o.dtype, dev)
        elif o is not None and o.numel():
            raise DiscoError(-1, f"out of gradient {i} has {o.numel()} elements, the gradient 0")
        fields += (gp or 0, op or 0, n, dtype_code(g.dtype), 0 if o is None else dtype_code(o.dtype))
    arr = (disco_grad_tensor * len(grads)).from_buffer_copy(struct.pack("QQqii" * len(grads), *fields))
    grads_c = disco_grads()
    _check(load_library().disco_grad_plan(arr, len(grads), ctypes.byref(grads_c)))
    grads_c.keep = (arr, grads, outs)
    return grads_c, arr


def disco_grad_workspace_bytes(grads: disco_grads) -> int:
    return load_library().disco_grad_workspace_bytes(ctypes.byref(grads))


def disco_grad_norm(grads: disco_grads, norm, workspace, grad_scale: float = 1.0, stream=None) -> None:
    """The Euclidean norm over all gradients, times grad_scale, to ``norm`` (one fp32)."""
    dev = _on(norm, "norm")
    np_ = _in(norm, "norm", 1, _torch.float32, dev)
    wp, wn = _bytes(workspace, "workspace", dev)
    _check((_lib or load_library()).disco_grad_norm(grads, grad_scale, np_, wp, wn,
                                                    _raw_stream(dev) if stream is None else _stream(stream)))


def disco_grad_clip(grads: disco_grads, max_norm: float, norm, grad_scale: float = 1.0, stream=None) -> None:
    """Every gradient scaled by grad_scale and down to ``max_norm`` given ``norm``, to its out."""
    dev = _on(norm, "norm")
    np_ = _in(norm, "norm", 1, _torch.float32, dev)
    _check((_lib or load_library()).disco_grad_clip(grads, grad_scale, max_norm, np_,
                                                    _raw_stream(dev) if stream is None else _stream(stream)))


def disco_grad_norm_clip(grads: disco_grads, max_norm: float, norm, workspace, grad_scale: float = 1.0,
                         stream=None) -> None:
    """disco_grad_norm and disco_grad_clip in one call."""
    dev = _on(norm, "norm")
    np_ = _in(norm, "norm", 1, _torch.float32, dev)
    wp, wn = _bytes(workspace, "workspace", dev)
    _check((_lib or load_library()).disco_grad_norm_clip(grads, grad_scale, max_norm, np_, wp, wn,
                                                         _raw_stream(dev) if stream is None else _stream(stream)))


def disco_quant_i8(x, q, scale, B: int, C: int, P: int, stream=None) -> None:
    """The tokens of x in 8-bit integers q with a scale for each; see include/disco.h."""
    n, dev = B * C * P, _on(x, "x")
    _check((_lib or load_library()).disco_quant_i8(
        _in(x, "x", n, x.dtype, dev), _in(q, "q", n, _torch.int8, dev), _in(scale, "scale", B * P, _torch.float32, dev),
        B, C, P, dtype_code(x.dtype), _raw_stream(dev) if stream is None else _stream(stream)))


def disco_matmul_i8_workspace_bytes(B: int, Cin: int, Cout: int, P: int, dtype=DISCO_BF16) -> int:
    return load_library().disco_matmul_i8_workspace_bytes(B, Cin, Cout, P, dtype)


def disco_matmul_i8(q, scale, W, wscale, y, B: int, Cin: int, Cout: int, P: int, workspace=None, stream=None) -> None:
    """y = scale wscale (W q), products of 8-bit integers over the channels of each token."""
    T, dev = B * P, _on(y, "y")
    f32, i8 = _torch.float32, _torch.int8
    wp, wn = _bytes(workspace, "workspace", dev)
    _check((_lib or load_library()).disco_matmul_i8(
        _in(q, "q", T * Cin, i8, dev), _in(scale, "scale", T, f32, dev), _in(W, "W", Cout * Cin, i8, dev),
        _in(wscale, "wscale", Cout, f32, dev), _in(y, "y", T * Cout, y.dtype, dev), B, Cin, Cout, P, dtype_code(y.dtype),
        wp, wn, _raw_stream(dev) if stream is None else _stream(stream)))


def disco_matmul_i8_bwd_input_workspace_bytes(B: int, Cin: int, Cout: int, P: int, dtype=DISCO_BF16) -> int:
    return load_library().disco_matmul_i8_bwd_input_workspace_bytes(B, Cin, Cout, P, dtype)


def disco_matmul_i8_bwd_input(dy, W, wscale, dx, B: int, Cin: int, Cout: int, P: int, workspace=None,
                              stream=None) -> None:
    """dx = (wscale W)^T dy, the gradient of disco_matmul_i8's activation."""
    T, dev = B * P, _on(dy, "dy")
    dt = dy.dtype
    wp, wn = _bytes(workspace, "workspace", dev)
    _check((_lib or load_library()).disco_matmul_i8_bwd_input(
        _in(dy, "dy", T * Cout, dt, dev), _in(W, "W", Cout * Cin, _torch.int8, dev),
        _in(wscale, "wscale", Cout, _torch.float32, dev), _in(dx, "dx", T * Cin, dt, dev), B, Cin, Cout, P, dtype_code(dt),
        wp, wn, _raw_stream(dev) if stream is None else _stream(stream)))


def disco_matmul_i8_bwd_weight_workspace_bytes(B: int, Cin: int, Cout: int, P: int, dtype=DISCO_BF16) -> int:
    return load_library().disco_matmul_i8_bwd_weight_workspace_bytes(B, Cin, Cout, P, dtype)


def disco_matmul_i8_bwd_weight(dy, q, scale, dW, B: int, Cin: int, Cout: int, P: int, workspace=None,
                               stream=None) -> None:
    """dW = dy (scale q)^T summed over tokens, from the kept 8-bit activation."""
    T, dev = B * P, _on(dy, "dy")
    dt = dy.dtype
    wp, wn = _bytes(workspace, "workspace", dev)
    _check((_lib or load_library()).disco_matmul_i8_bwd_weight(
        _in(dy, "dy", T * Cout, dt, dev), _in(q, "q", T * Cin, _torch.int8, dev),
        _in(scale, "scale", T, _torch.float32, dev), _in(dW, "dW", Cout * Cin, dt, dev), B, Cin, Cout, P, dtype_code(dt),
        wp, wn, _raw_stream(dev) if stream is None else _stream(stream)))


def disco_glu(x, y, act: int, B: int, C: int, P: int, q=None, scale=None, xq=None, xscale=None, stream=None) -> None:
    """y = act(x[:, :C]) x[:, C:] for x [B, 2 C, P], y in 8 bits (q, scale) and x
    in 8 bits (xq, xscale, what disco_glu_bwd needs); y, or either pair, may be None."""
    n, T, dev = B * C * P, B * P, _on(x, "x")
    dt = x.dtype
    f32, i8 = _torch.float32, _torch.int8
    _check((_lib or load_library()).disco_glu(
        _in(x, "x", 2 * n, dt, dev), _in(y, "y", n, dt, dev), _in(q, "q", n, i8, dev), _in(scale, "scale", T, f32, dev),
        _in(xq, "xq", 2 * n, i8, dev), _in(xscale, "xscale", T, f32, dev), act, B, C, P, dtype_code(dt),
        _raw_stream(dev) if stream is None else _stream(stream)))


def disco_glu_bwd(dy, xq, xscale, dx, act: int, B: int, C: int, P: int, stream=None) -> None:
    """dx of disco_glu for the gradient dy of y, from the kept 8-bit input."""
    n, dev = B * C * P, _on(dy, "dy")
    dt = dy.dtype
    _check((_lib or load_library()).disco_glu_bwd(
        _in(dy, "dy", n, dt, dev), _in(xq, "xq", 2 * n, _torch.int8, dev), _in(xscale, "xscale", B * P, _torch.float32, dev),
        _in(dx, "dx", 2 * n, dt, dev), act, B, C, P, dtype_code(dt), _raw_stream(dev) if stream is None else _stream(stream)))


def disco_device_status(clear: bool = True) -> int:
    """Device status word (0 = no bounded wait timed out); synchronises the device.
    Raises DiscoError with status DISCO_ERR_DEVICE_BOUNDS when a range check
    of the bounds-checked build failed."""
    v = ctypes.c_int32()
    _check(load_library().disco_device_status(ctypes.byref(v), 1 if clear else 0))
    return v.value


# ------------------------------------------------------------ convenience

class Psi:
    """psi built on the device, with the torch buffers that own its memory
    (``.c``, the struct that the calls take, keeps its buffer alive).

    ``Psi(grid_in, grid_out, kind, n_radial, cutoff)`` runs disco_psi_plan and
    disco_build_psi_kpacked on the current CUDA device and stream."""

    _DT = {"row_ptr": "int32", "idx": "int32", "val": "float32", "csr_row_ptr": "int32",
           "csr_col": "int32", "csr_val": "float32", "run_ptr": "int32", "runs": "int32",
           "trun_ptr": "int32", "truns": "int32", "hval": "float32", "row_order": "int32",
           "ftab_off": "int32", "ftab": "int16", "grp_ptr": "int32", "grp": "int32", "gtab": "int16",
           "ftab_h": "int16", "gtab_h": "int16"}

    def __init__(self, grid_in, grid_out, kind: int, n_radial: int, cutoff: float, stream=None):
        import torch
        self.basis = _basis(kind, n_radial, cutoff)
        gi, go = _grid(grid_in), _grid(grid_out)
        wsb = disco_psi_workspace_bytes(gi, go, self.basis)
        self.workspace = torch.empty(max(wsb, 256), dtype=torch.uint8, device="cuda")
        self.c = disco_psi_plan(gi, go, self.basis, self.workspace, stream)
        self.buffer = torch.empty(max(self.c.bytes, 256), dtype=torch.uint8, device="cuda")
        self.c.keep = self.buffer  # the struct points into it
        disco_build_psi_kpacked(self.c, self.buffer, self.workspace, stream)

    def _sizes(self):
        c = self.c
        Hin, Hout = c.grid_in.nlat, c.grid_out.nlat
        return {"row_ptr": (Hout + 1,), "idx": (c.nnz, 2), "val": (c.nnz, c.K_pad),
                "csr_row_ptr": (c.K * Hout + 1,), "csr_col": (c.nnz_csr,),
                "csr_val": (c.nnz_csr,), "run_ptr": (Hout + 1,), "runs": (c.nruns, 8),
                "trun_ptr": (Hin + 1,), "truns": (c.nruns,), "hval": (c.nhval, c.K_pad),
                "row_order": (Hout,), "ftab_off": (c.nruns + 1,), "ftab": (c.nftab,),
                "grp_ptr": (c.ngrp + 1,), "grp": (c.ngrp_ent, 4), "gtab": (c.ngtab,),
                "ftab_h": (c.nftab,), "gtab_h": (c.ngtab,)}

    def tensor(self, name: str):
        """Device view of one psi array (for inspection and tests)."""
        import torch
        ptr = getattr(self.c, name)
        off = ptr - self.buffer.data_ptr()
        shape = self._sizes()[name]
        n = 1
        for v in shape:
            n *= int(v)
        dt = getattr(torch, self._DT[name])
        esz = torch.tensor([], dtype=dt).element_size()
        return self.buffer[off:off + n * esz].view(dt).view(*[int(v) for v in shape])


class GradPlan:
    """A list of gradients checked once (disco_grad_plan), with the tensors it
    refers to.  ``GradPlan(grads, outs)``; pass ``.c`` (which keeps the tensors
    too) to disco_grad_norm, disco_grad_clip and disco_grad_norm_clip.
    Gradients allocated anew need a new plan."""

    def __init__(self, grads, outs=None):
        self.grads = list(grads)
        self.outs = None if outs is None else list(outs)
        self.c, self._array = disco_grad_plan(self.grads, self.outs)
