"""Python binding of libzs (include/zs.h): argument marshalling only.

Every entry point has the name of the C function it calls.  Tensors must be
CUDA tensors of the documented dtype and shape; outputs and workspaces are
allocated with torch when not given.  A call runs on the current stream, or on
``stream`` (an object or a handle) as if that one were current: it has to be
ordered after the work that makes the operands.  All compute runs in libzs's
kernels; there is no fallback, and a missing or unbuildable library raises.
"""
from __future__ import annotations

import ctypes
import importlib.util
import operator
import os
import re
import threading
import warnings

import torch

from . import build as _build

_lock = threading.Lock()
_lib = None

ZS_OK = 0
STATUS_NAMES = {0: "ZS_OK", 1: "ZS_ERR_INVALID_ARG", 2: "ZS_ERR_UNSUPPORTED", 3: "ZS_ERR_CUDA", 4: "ZS_ERR_TIMEOUT"}


class ZsError(RuntimeError):
    def __init__(self, fn: str, status: int, msg: str):
        super().__init__(f"{fn} -> {STATUS_NAMES.get(status, status)}: {msg}")
        self.status = status


def library_path() -> str:
    return _build.LIB


def load(build_if_missing: bool = True):
    """Load libzs.so (building it with nvcc first if it is missing or stale)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if build_if_missing:
            _build.build()
        if not os.path.exists(_build.LIB):
            raise RuntimeError(f"libzs.so not found at {_build.LIB}; run equivariant_interatomic_potential_gb300.build")
        lib = ctypes.CDLL(_build.LIB)
        P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        lib.zs_status_string.restype = ctypes.c_char_p
        lib.zs_status_string.argtypes = [ctypes.c_int]
        lib.zs_last_error.restype = ctypes.c_char_p
        lib.zs_last_error.argtypes = []
        lib.zs_version.restype = ctypes.c_int
        lib.zs_version.argtypes = []
        lib.zs_build_csr_workspace_bytes.restype = SZ
        lib.zs_build_csr_workspace_bytes.argtypes = [I64, I32]
        lib.zs_build_csr.restype = ctypes.c_int
        lib.zs_build_csr.argtypes = [P, I64, I32, P, P, P, P, SZ, P]
        lib.zs_forward_workspace_bytes.restype = SZ
        lib.zs_forward_workspace_bytes.argtypes = [I64, I32, I32]
        lib.zs_forward_workspace_bytes_lmax.restype = SZ
        lib.zs_forward_workspace_bytes_lmax.argtypes = [I64, I32, I32, I32]
        lib.zs_forward.restype = ctypes.c_int
        lib.zs_forward.argtypes = [P, P, P, P, I64, I32, I32, I32, P, P, SZ, P]
        lib.zs_backward.restype = ctypes.c_int
        lib.zs_backward.argtypes = [P, P, P, P, I64, I32, I32, I32, P, P, P]
        lib.zs_forward_ld.restype = ctypes.c_int
        lib.zs_forward_ld.argtypes = [P, I64, P, P, P, I64, I32, I32, I32, P, P, SZ, P]
        lib.zs_backward_ld.restype = ctypes.c_int
        lib.zs_backward_ld.argtypes = [P, P, I64, P, P, I64, I32, I32, I32, P, I64, P, P]
        lib.zs_forward_scaled.restype = ctypes.c_int
        lib.zs_forward_scaled.argtypes = [P, P, P, P, P, I64, I32, I32, I32, P, P, P, SZ, P]
        lib.zs_backward_scaled.restype = ctypes.c_int
        lib.zs_backward_scaled.argtypes = [P, P, P, P, P, P, I64, I32, I32, I32, P, P, P, P]
        lib.zs_backward_csr.restype = ctypes.c_int
        lib.zs_backward_csr.argtypes = [P, P, P, P, P, I64, I32, I32, I32, P, P, P]
        lib.zs_forward_noalloc.restype = ctypes.c_int
        lib.zs_forward_noalloc.argtypes = [P, P, P, P, I64, I32, I32, I32, P, P]
        lib.zs_selftest_bounded_wait.restype = ctypes.c_int
        lib.zs_selftest_bounded_wait.argtypes = [ctypes.c_uint32, P]
        lib.zs_check_timeouts.restype = ctypes.c_int
        lib.zs_check_timeouts.argtypes = []
        lib.zs_set_timeout_flag.restype = ctypes.c_int
        lib.zs_set_timeout_flag.argtypes = [P]
        F32 = ctypes.c_float
        lib.zs_grouped_matmul.restype = ctypes.c_int
        lib.zs_grouped_matmul.argtypes = [I32, P, I64, P, P, P, I64, I32, I32, I32, P, I64, P]
        lib.zs_grouped_matmul_dx.restype = ctypes.c_int
        lib.zs_grouped_matmul_dx.argtypes = [I32, P, I64, P, P, P, I64, I32, I32, I32, P, I64, P]
        lib.zs_grouped_matmul_workspace_bytes.restype = SZ
        lib.zs_grouped_matmul_workspace_bytes.argtypes = [I32, I64, I32, I32, I32]
        for fn in (lib.zs_grouped_matmul_ws, lib.zs_grouped_matmul_dx_ws):
            fn.restype = ctypes.c_int
            fn.argtypes = [I32, P, I64, P, P, P, I64, I32, I32, I32, P, I64, P, SZ, P]
        lib.zs_grouped_matmul_dw_workspace_bytes.restype = SZ
        lib.zs_grouped_matmul_dw_workspace_bytes.argtypes = [I32, I64, I32, I32, I32]
        lib.zs_grouped_matmul_dw_copy_bytes.restype = SZ
        lib.zs_grouped_matmul_dw_copy_bytes.argtypes = [I32, I64, I32, I32, I32]
        lib.zs_grouped_matmul_dw.restype = ctypes.c_int
        lib.zs_grouped_matmul_dw.argtypes = [I32, P, I64, P, I64, P, P, I64, I32, I32, I32, P, P, SZ, P]
        lib.zs_norm_gate_residual.restype = ctypes.c_int
        lib.zs_norm_gate_residual.argtypes = [I32, I32, P, I64, P, I64, P, I64, I32, P, P, P, F32, I64, I32, P, P, P, P]
        lib.zs_norm_gate_residual_backward_workspace_bytes.restype = SZ
        lib.zs_norm_gate_residual_backward_workspace_bytes.argtypes = [I64, I32]
        lib.zs_norm_gate_residual_backward.restype = ctypes.c_int
        lib.zs_norm_gate_residual_backward.argtypes = [I32, I32, P, I64, P, I64, P, I64, P, I64, P, I64, I32, P, P, P, P,
                                                       I64, I32, P, P, P, P, P, P, P, SZ, P]
        lib.zs_adamw_step.restype = ctypes.c_int
        lib.zs_adamw_step.argtypes = [P, I32, I32, I32, P, P, P]
        lib.zs_adamw_step_seeded.restype = ctypes.c_int
        lib.zs_adamw_step_seeded.argtypes = [P, I32, I32, I32, P, ctypes.c_uint64, P, P]
        U32, U64 = ctypes.c_uint32, ctypes.c_uint64
        lib.zs_embedding.restype = ctypes.c_int
        lib.zs_embedding.argtypes = [I32, P, I64, P, I64, I32, I32, F32, P, I64, P]
        lib.zs_embedding_backward_workspace_bytes.restype = SZ
        lib.zs_embedding_backward_workspace_bytes.argtypes = [I32, I64, I32, I32]
        lib.zs_embedding_backward.restype = ctypes.c_int
        lib.zs_embedding_backward.argtypes = [I32, P, I64, P, P, I64, I32, I32, F32, P, P, SZ, P]
        lib.zs_route.restype = ctypes.c_int
        lib.zs_route.argtypes = [I32, I32, P, I64, P, I64, I32, I32, I32, I32, I32, I32, F32, P, P, P]
        lib.zs_route_backward.restype = ctypes.c_int
        lib.zs_route_backward.argtypes = [I32, I32, P, P, I64, P, I64, I32, I32, I32, F32, P, P]
        lib.zs_dispatch.restype = ctypes.c_int
        lib.zs_dispatch.argtypes = [I32, P, I64, P, P, I64, I32, I32, I32, P, P, P]
        lib.zs_combine.restype = ctypes.c_int
        lib.zs_combine.argtypes = [I32, P, I64, P, P, I64, I32, I64, I32, P, I64, P]
        lib.zs_combine_backward.restype = ctypes.c_int
        lib.zs_combine_backward.argtypes = [I32, P, I64, P, I64, P, P, P, I64, I32, I32, I32, P, P, P]
        lib.zs_dropout.restype = ctypes.c_int
        lib.zs_dropout.argtypes = [I32, P, I64, P, I64, I64, I32, ctypes.c_double, U64, U32, I64, P, P, I64, P]
        _lib = lib
        return lib


class _Fast:
    """zs_torch, the short way for ordinary operands; built if need be and loaded on first
    use.  Where that fails, every call is left to the binding."""

    NAMES = ("matmul", "dw", "norm", "norm_backward", "csr", "embedding", "embedding_backward", "route", "route_backward", "dispatch",
             "combine", "combine_backward", "dropout")
    LIBRARY = ("zs_build_csr", "zs_grouped", "zs_norm", "zs_embedding", "zs_route", "zs_dispatch", "zs_combine", "zs_dropout")

    def __getattr__(self, name):
        if name not in self.NAMES:
            raise AttributeError(name)
        lib = load()
        try:
            spec = importlib.util.spec_from_file_location("zs_torch", _build.build_ext())
            ext = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(ext)
            names = [n for n in declared_functions() if n.startswith(self.LIBRARY)]
            ext.bind({n: ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in names}, _check)
            calls = {n: getattr(ext, n) for n in self.NAMES}
        except Exception as e:
            warnings.warn(f"zs_torch cannot be used, calls of the training operators take longer on the host: {e}")
            calls = dict.fromkeys(self.NAMES, lambda *operands: NotImplemented)
        for n, call in calls.items():
            setattr(self, n, call)
        return getattr(self, name)


_fast = _Fast()


def declared_functions(header: str | None = None) -> list[str]:
    """Names of the functions include/zs.h declares (ZS_API prototypes)."""
    header = header or os.path.join(_build.INCLUDE, "zs.h")
    with open(header) as f:
        text = f.read()
    return re.findall(r"ZS_API\s+[\w\s\*]*?\b(zs_\w+)\s*\(", text)


def _check(fn: str, status: int):
    if status != ZS_OK:
        raise ZsError(fn, status, load().zs_last_error().decode())


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr() if t.numel() > 0 else None


# The current stream's handle without building a Stream object for it (0.2
# against 2.9 us a call on the host of a GB300).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_raw_device = getattr(torch._C, "_cuda_getDevice", None)


def _stream(stream) -> int | None:
    if stream is None:
        if _raw_stream is None or _raw_device is None:
            return torch.cuda.current_stream().cuda_stream
        return _raw_stream(_raw_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _current_device() -> int:
    return torch.cuda.current_device() if _raw_device is None else _raw_device()


def _one_device(operands, device=None) -> int:
    """The index of the device that every CUDA tensor among the operands is on, which is
    that of ``device`` (a stream's) where it is given."""
    on = {t.get_device() for t in operands if isinstance(t, torch.Tensor) and t.is_cuda}
    if device is not None:
        on.add(device.index)
    if len(on) > 1:
        names = " and ".join(f"cuda:{i}" for i in sorted(on))
        raise ValueError(f"the operands{'' if device is None else ' and the stream'} must be on one device, got {names}")
    return on.pop() if on else -1


def _elsewhere(*operands):
    """The device of the operands where it is not the current one, which a call then enters."""
    device = _one_device(operands)
    return device if device >= 0 and device != _current_device() else None


def _on(stream, call, *args, **kw):
    """call(...) with ``stream`` (a stream object or a handle) current, so that what the call
    allocates is that stream's: no other stream is handed its workspace while the kernels
    run.  The results may be used and dropped on the caller's stream too (once it has waited
    for ``stream``)."""
    handle = _stream(stream)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(handle) if handle else torch.cuda.default_stream()
    _one_device((*args, *kw.values()), stream.device)
    caller = torch.cuda.current_stream()
    with torch.cuda.stream(stream):
        result = call(*args, **kw)
    if caller.cuda_stream != handle:
        for t in result if isinstance(result, tuple) else (result,):
            if t is not None:
                t.record_stream(caller)
    return result


def _need(t: torch.Tensor, name: str, dtype: torch.dtype, shape: tuple):
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _need_rows(t: torch.Tensor, name: str, shape: tuple) -> int:
    """A float32 CUDA matrix whose rows are contiguous and evenly spaced (a
    view into a wider array allowed): returns the row stride in elements."""
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != torch.float32:
        raise ValueError(f"{name} must be torch.float32, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.numel() and (t.stride(1) != 1 or (t.shape[0] > 1 and t.stride(0) < t.shape[1])):
        raise ValueError(f"{name} must have contiguous rows (stride (ld, 1) with ld >= {t.shape[1]})")
    return max(int(t.stride(0)), int(t.shape[1])) if t.shape[0] > 1 else int(t.shape[1])


def _workspace(nbytes: int, device) -> torch.Tensor | None:
    if nbytes == 0:
        return None
    # torch's caching allocator returns blocks aligned to at least 512 bytes
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def zs_build_csr_workspace_bytes(E: int, N: int) -> int:
    return int(load().zs_build_csr_workspace_bytes(E, N))


def zs_forward_workspace_bytes(E: int, N: int, C: int, lmax: int = 3) -> int:
    return int(load().zs_forward_workspace_bytes_lmax(E, N, C, lmax))


def ladder(lmax: int) -> tuple[int, int]:
    """(D, R): node rows (lmax+1)^2 and zonal rows D - 1 of the degree-lmax ladder."""
    D = (lmax + 1) ** 2
    return D, D - 1


def _lmax(rad: torch.Tensor, lmax: int | None) -> int:
    """The ladder degree: given, else the radial operand's slot count (E, lmax, C)."""
    return int(rad.shape[1]) if lmax is None else int(lmax)


def zs_build_csr(dst: torch.Tensor, N: int, row_ptr=None, perm=None, bad_dst_count=None,
                 workspace=None, stream=None):
    """Stable destination CSR.  Returns (row_ptr (N+1,), perm (E,), bad_dst_count (1,)) int32."""
    if stream is not None:
        return _on(stream, zs_build_csr, dst, N, row_ptr, perm, bad_dst_count, workspace)
    if row_ptr is None and perm is None and bad_dst_count is None and workspace is None:
        r = _fast.csr(dst, N)
        if r is not NotImplemented:
            return r
    E = dst.shape[0]
    dev = dst.device
    _need(dst, "dst", torch.int32, (E,))
    row_ptr = torch.empty(N + 1, dtype=torch.int32, device=dev) if row_ptr is None else row_ptr
    perm = torch.empty(E, dtype=torch.int32, device=dev) if perm is None else perm
    bad_dst_count = torch.empty(1, dtype=torch.int32, device=dev) if bad_dst_count is None else bad_dst_count
    _need(row_ptr, "row_ptr", torch.int32, (N + 1,))
    _need(perm, "perm", torch.int32, (E,))
    need = zs_build_csr_workspace_bytes(E, N)
    if workspace is None:
        workspace = _workspace(need, dev)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("zs_build_csr", load().zs_build_csr(_ptr(dst), E, N, _ptr(row_ptr), _ptr(perm), _ptr(bad_dst_count),
                                               _ptr(workspace), wbytes, _stream(None)))
    return row_ptr, perm, bad_dst_count


def zs_forward(coup: torch.Tensor, rad: torch.Tensor, row_ptr: torch.Tensor, perm: torch.Tensor, N: int,
               out=None, workspace=None, stream=None, lmax: int | None = None):
    """Forward zonal scatter.  Returns out (N, D, C) fp32; lmax defaults to rad.shape[1]."""
    if stream is not None:
        return _on(stream, zs_forward, coup, rad, row_ptr, perm, N, out, workspace, lmax=lmax)
    lmax = _lmax(rad, lmax)
    D, R = ladder(lmax)
    E = coup.shape[0]
    C = rad.shape[2]
    dev = coup.device
    _need(coup, "coup", torch.float32, (E, R))
    _need(rad, "rad", torch.float32, (E, lmax, C))
    _need(row_ptr, "row_ptr", torch.int32, (N + 1,))
    _need(perm, "perm", torch.int32, (E,))
    out = torch.empty((N, D, C), dtype=torch.float32, device=dev) if out is None else out
    _need(out, "out", torch.float32, (N, D, C))
    if workspace is None:
        workspace = _workspace(zs_forward_workspace_bytes(E, N, C, lmax), dev)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("zs_forward", load().zs_forward(_ptr(coup), _ptr(rad), _ptr(row_ptr), _ptr(perm), E, N, C, lmax,
                                           _ptr(out), _ptr(workspace), wbytes, _stream(None)))
    return out


def zs_forward_ld(coup: torch.Tensor, rad: torch.Tensor, row_ptr: torch.Tensor, perm: torch.Tensor, N: int,
                  out=None, workspace=None, stream=None, lmax: int | None = None):
    """zs_forward with coup a row-strided view (for example the m = 0 segment of a
    packed (E, 3D-2) Wigner band): coup[e] = coup.data_ptr() + e * coup.stride(0)."""
    if stream is not None:
        return _on(stream, zs_forward_ld, coup, rad, row_ptr, perm, N, out, workspace, lmax=lmax)
    lmax = _lmax(rad, lmax)
    D, R = ladder(lmax)
    E = coup.shape[0]
    C = rad.shape[2]
    dev = coup.device
    ld = _need_rows(coup, "coup", (E, R))
    _need(rad, "rad", torch.float32, (E, lmax, C))
    _need(row_ptr, "row_ptr", torch.int32, (N + 1,))
    _need(perm, "perm", torch.int32, (E,))
    out = torch.empty((N, D, C), dtype=torch.float32, device=dev) if out is None else out
    _need(out, "out", torch.float32, (N, D, C))
    if workspace is None:
        workspace = _workspace(zs_forward_workspace_bytes(E, N, C, lmax), dev)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("zs_forward_ld", load().zs_forward_ld(_ptr(coup), ld, _ptr(rad), _ptr(row_ptr), _ptr(perm), E, N, C, lmax,
                                                 _ptr(out), _ptr(workspace), wbytes, _stream(None)))
    return out


def zs_backward_ld(g: torch.Tensor, coup: torch.Tensor, rad: torch.Tensor, dst: torch.Tensor, N: int,
                   d_coup: torch.Tensor, d_rad=None, stream=None, lmax: int | None = None):
    """zs_backward with coup and d_coup row-strided views (d_coup must be given)."""
    if stream is not None:
        return _on(stream, zs_backward_ld, g, coup, rad, dst, N, d_coup, d_rad, lmax=lmax)
    lmax = _lmax(rad, lmax)
    D, R = ladder(lmax)
    E = coup.shape[0]
    C = rad.shape[2]
    dev = coup.device
    _need(g, "g", torch.float32, (N, D, C))
    ld = _need_rows(coup, "coup", (E, R))
    dld = _need_rows(d_coup, "d_coup", (E, R))
    _need(rad, "rad", torch.float32, (E, lmax, C))
    _need(dst, "dst", torch.int32, (E,))
    d_rad = torch.empty((E, lmax, C), dtype=torch.float32, device=dev) if d_rad is None else d_rad
    _need(d_rad, "d_rad", torch.float32, (E, lmax, C))
    _check("zs_backward_ld", load().zs_backward_ld(_ptr(g), _ptr(coup), ld, _ptr(rad), _ptr(dst), E, N, C, lmax,
                                                   _ptr(d_coup), dld, _ptr(d_rad), _stream(None)))
    return d_coup, d_rad


def zs_forward_scaled(coup: torch.Tensor, rad: torch.Tensor, row_ptr: torch.Tensor, perm: torch.Tensor,
                      node_scale: torch.Tensor, N: int, out=None, out_raw=None, want_raw: bool = True,
                      workspace=None, stream=None, lmax: int | None = None):
    """Forward with the per-node factor fused in.  Returns (out, out_raw); out_raw is
    None when want_raw is False and none is given."""
    if stream is not None:
        return _on(stream, zs_forward_scaled, coup, rad, row_ptr, perm, node_scale, N, out, out_raw, want_raw,
                   workspace, lmax=lmax)
    lmax = _lmax(rad, lmax)
    D, R = ladder(lmax)
    E = coup.shape[0]
    C = rad.shape[2]
    dev = coup.device
    _need(coup, "coup", torch.float32, (E, R))
    _need(rad, "rad", torch.float32, (E, lmax, C))
    _need(row_ptr, "row_ptr", torch.int32, (N + 1,))
    _need(perm, "perm", torch.int32, (E,))
    _need(node_scale, "node_scale", torch.float32, (N,))
    out = torch.empty((N, D, C), dtype=torch.float32, device=dev) if out is None else out
    _need(out, "out", torch.float32, (N, D, C))
    if out_raw is None and want_raw:
        out_raw = torch.empty((N, D, C), dtype=torch.float32, device=dev)
    if out_raw is not None:
        _need(out_raw, "out_raw", torch.float32, (N, D, C))
    if workspace is None:
        workspace = _workspace(zs_forward_workspace_bytes(E, N, C, lmax), dev)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("zs_forward_scaled", load().zs_forward_scaled(_ptr(coup), _ptr(rad), _ptr(row_ptr), _ptr(perm),
                                                         _ptr(node_scale), E, N, C, lmax, _ptr(out), _ptr(out_raw),
                                                         _ptr(workspace), wbytes, _stream(None)))
    return out, out_raw


def zs_backward_scaled(g: torch.Tensor, coup: torch.Tensor, rad: torch.Tensor, dst: torch.Tensor,
                       node_scale: torch.Tensor, N: int, out_raw=None, d_coup=None, d_rad=None, d_scale=None,
                       want_scale_grad: bool = True, stream=None, lmax: int | None = None):
    """Backward of zs_forward_scaled.  Returns (d_coup, d_rad, d_scale); d_scale is
    None unless out_raw is given (and want_scale_grad)."""
    if stream is not None:
        return _on(stream, zs_backward_scaled, g, coup, rad, dst, node_scale, N, out_raw, d_coup, d_rad, d_scale,
                   want_scale_grad, lmax=lmax)
    lmax = _lmax(rad, lmax)
    D, R = ladder(lmax)
    E = coup.shape[0]
    C = rad.shape[2]
    dev = coup.device
    _need(g, "g", torch.float32, (N, D, C))
    _need(coup, "coup", torch.float32, (E, R))
    _need(rad, "rad", torch.float32, (E, lmax, C))
    _need(dst, "dst", torch.int32, (E,))
    _need(node_scale, "node_scale", torch.float32, (N,))
    d_coup = torch.empty((E, R), dtype=torch.float32, device=dev) if d_coup is None else d_coup
    d_rad = torch.empty((E, lmax, C), dtype=torch.float32, device=dev) if d_rad is None else d_rad
    _need(d_coup, "d_coup", torch.float32, (E, R))
    _need(d_rad, "d_rad", torch.float32, (E, lmax, C))
    if out_raw is not None:
        _need(out_raw, "out_raw", torch.float32, (N, D, C))
        if d_scale is None and want_scale_grad:
            d_scale = torch.empty(N, dtype=torch.float32, device=dev)
    if d_scale is not None:
        _need(d_scale, "d_scale", torch.float32, (N,))
    _check("zs_backward_scaled", load().zs_backward_scaled(_ptr(g), _ptr(coup), _ptr(rad), _ptr(dst),
                                                           _ptr(node_scale), _ptr(out_raw), E, N, C, lmax,
                                                           _ptr(d_coup), _ptr(d_rad), _ptr(d_scale),
                                                           _stream(None)))
    return d_coup, d_rad, d_scale


def zs_backward(g: torch.Tensor, coup: torch.Tensor, rad: torch.Tensor, dst: torch.Tensor, N: int,
                d_coup=None, d_rad=None, stream=None, lmax: int | None = None):
    """Backward.  Returns (d_coup (E, R), d_rad (E, lmax, C)) fp32; lmax defaults to rad.shape[1]."""
    if stream is not None:
        return _on(stream, zs_backward, g, coup, rad, dst, N, d_coup, d_rad, lmax=lmax)
    lmax = _lmax(rad, lmax)
    D, R = ladder(lmax)
    E = coup.shape[0]
    C = rad.shape[2]
    dev = coup.device
    _need(g, "g", torch.float32, (N, D, C))
    _need(coup, "coup", torch.float32, (E, R))
    _need(rad, "rad", torch.float32, (E, lmax, C))
    _need(dst, "dst", torch.int32, (E,))
    d_coup = torch.empty((E, R), dtype=torch.float32, device=dev) if d_coup is None else d_coup
    d_rad = torch.empty((E, lmax, C), dtype=torch.float32, device=dev) if d_rad is None else d_rad
    _need(d_coup, "d_coup", torch.float32, (E, R))
    _need(d_rad, "d_rad", torch.float32, (E, lmax, C))
    _check("zs_backward", load().zs_backward(_ptr(g), _ptr(coup), _ptr(rad), _ptr(dst), E, N, C, lmax,
                                             _ptr(d_coup), _ptr(d_rad), _stream(None)))
    return d_coup, d_rad


def zs_backward_csr(g: torch.Tensor, coup: torch.Tensor, rad: torch.Tensor, row_ptr: torch.Tensor,
                    perm: torch.Tensor, N: int, d_coup=None, d_rad=None, stream=None, lmax: int | None = None):
    """Backward with edges visited in CSR order.  Returns (d_coup (E, R), d_rad (E, lmax, C)) fp32."""
    if stream is not None:
        return _on(stream, zs_backward_csr, g, coup, rad, row_ptr, perm, N, d_coup, d_rad, lmax=lmax)
    lmax = _lmax(rad, lmax)
    D, R = ladder(lmax)
    E = coup.shape[0]
    C = rad.shape[2]
    dev = coup.device
    _need(g, "g", torch.float32, (N, D, C))
    _need(coup, "coup", torch.float32, (E, R))
    _need(rad, "rad", torch.float32, (E, lmax, C))
    _need(row_ptr, "row_ptr", torch.int32, (N + 1,))
    _need(perm, "perm", torch.int32, (E,))
    d_coup = torch.empty((E, R), dtype=torch.float32, device=dev) if d_coup is None else d_coup
    d_rad = torch.empty((E, lmax, C), dtype=torch.float32, device=dev) if d_rad is None else d_rad
    _need(d_coup, "d_coup", torch.float32, (E, R))
    _need(d_rad, "d_rad", torch.float32, (E, lmax, C))
    _check("zs_backward_csr", load().zs_backward_csr(_ptr(g), _ptr(coup), _ptr(rad), _ptr(row_ptr), _ptr(perm),
                                                     E, N, C, lmax, _ptr(d_coup), _ptr(d_rad), _stream(None)))
    return d_coup, d_rad


def zs_check_timeouts() -> None:
    """Raise ZsError if a bounded device wait ran out since the last check
    (synchronises).  Also clears the current device's page-locked timeout
    flag (``timeout_flag``), if registered: the timeout has been reported."""
    st = load().zs_check_timeouts()
    f = _flags.get(torch.cuda.current_device()) if torch.cuda.is_available() else None
    if f is not None:
        f[0] = 0
    _check("zs_check_timeouts", st)


def zs_set_timeout_flag(flag: torch.Tensor | None) -> None:
    """Register (or, with None, unregister) the current device's timeout flag
    word: an int32 tensor of one element, on the device or in page-locked
    host memory, that the kernels set to 1 when a bounded wait runs out."""
    if flag is not None:
        if flag.dtype != torch.int32 or flag.numel() != 1:
            raise ValueError("the timeout flag is a one-element int32 tensor")
        if flag.device.type == "cpu" and not flag.is_pinned():
            raise ValueError("a host timeout flag must be in page-locked (pinned) memory")
    _check("zs_set_timeout_flag", load().zs_set_timeout_flag(_ptr(flag)))


_flags: dict[int, torch.Tensor] = {}
_flags_lock = threading.Lock()


def _device_index(device) -> int:
    idx = None if device is None else torch.device(device).index
    return torch.cuda.current_device() if idx is None else idx


def timeout_flag(device=None) -> torch.Tensor:
    """The page-locked host word registered for ``device`` (the current CUDA
    device by default), registering it on first use (not during stream
    capture: the registration is a synchronous copy).  It reads 1 once a
    bounded wait of a kernel launched after the registration has run out;
    reading it does not synchronise anything."""
    idx = _device_index(device)
    with _flags_lock:
        f = _flags.get(idx)
        if f is None:
            f = torch.zeros(1, dtype=torch.int32, pin_memory=True)
            with torch.cuda.device(idx):
                zs_set_timeout_flag(f)
            _flags[idx] = f
        return f


def raise_on_timeout_flag(device=None) -> None:
    """Raise ZsError (ZS_ERR_TIMEOUT) if the device's timeout flag is set, and
    clear it.  A host read only: a timeout inside a kernel that has not
    finished yet shows up at a later check.  Registers the flag on first use,
    except while the current stream is being captured."""
    idx = _device_index(device)
    f = _flags.get(idx)
    if f is None:
        if torch.cuda.is_current_stream_capturing():
            return
        f = timeout_flag(idx)
    if int(f[0]) != 0:
        f[0] = 0
        raise ZsError("timeout flag", 4, "a bounded device wait ran out in an earlier launch; its outputs are undefined")


def zs_forward_noalloc(coup: torch.Tensor, rad: torch.Tensor, row_ptr: torch.Tensor, perm: torch.Tensor, N: int,
                       out: torch.Tensor, stream=None, lmax: int | None = None):
    """zs_forward with the library's static device scratch instead of a workspace.

    For callers that cannot allocate device memory: ``out`` must be given,
    nothing is allocated.  See include/zs.h for the size limit and the rule
    that overlapping calls race.
    """
    lmax = _lmax(rad, lmax)
    D, R = ladder(lmax)
    E = coup.shape[0]
    C = rad.shape[2]
    _need(coup, "coup", torch.float32, (E, R))
    _need(rad, "rad", torch.float32, (E, lmax, C))
    _need(row_ptr, "row_ptr", torch.int32, (N + 1,))
    _need(perm, "perm", torch.int32, (E,))
    _need(out, "out", torch.float32, (N, D, C))
    _check("zs_forward_noalloc", load().zs_forward_noalloc(_ptr(coup), _ptr(rad), _ptr(row_ptr), _ptr(perm),
                                                           E, N, C, lmax, _ptr(out), _stream(stream)))
    return out


# ---------------------------------------------------------------------------
# Training operators: products grouped by a CSR, residual norms with a gate,
# the AdamW step.  Small calls last as long as their host side, so the checks
# have a short way for operands that are as they should be.

DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
NORM_KINDS = {"rms": 0, "layer": 1}
ADAMW_BLOCK = 256          # elements that share a scale of an 8-bit state


def _dtype(t: torch.Tensor, name: str) -> int:
    d = DTYPES.get(t.dtype)
    if d is None:
        raise ValueError(f"{name} must be float32, bfloat16 or float16, got {t.dtype}")
    return d


def _array(t: torch.Tensor, name: str, dtype: torch.dtype, shape: tuple) -> int:
    """Checks a contiguous CUDA tensor and returns its address."""
    if not (t.is_cuda and t.dtype is dtype and t.shape == shape and t.is_contiguous()):
        _need(t, name, dtype, shape)
    return t.data_ptr()


def _matrix(t: torch.Tensor, name: str, dtype: torch.dtype, rows: int, cols: int) -> int:
    """Checks a CUDA matrix whose rows are contiguous (a row-strided view
    allowed) and returns its row stride in elements."""
    if t.is_cuda and t.dtype is dtype and t.shape == (rows, cols) and t.is_contiguous():
        return cols
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != (rows, cols):
        raise ValueError(f"{name} must have shape {(rows, cols)}, got {tuple(t.shape)}")
    ld, step = t.stride()
    if t.numel() and (rows > 1 and ld < cols or cols > 1 and step != 1):
        raise ValueError(f"{name} must have contiguous rows (stride (ld, 1) with ld >= {cols})")
    return ld if rows > 1 and ld >= cols else cols


def _rows(t: torch.Tensor, name: str) -> tuple[int, int]:
    if t.dim() != 2:
        raise ValueError(f"{name} must be a matrix, got shape {tuple(t.shape)}")
    return t.shape


def _groups(w: torch.Tensor, row_ptr: torch.Tensor, perm: torch.Tensor | None, M: int):
    """Checks the weights and the CSR; returns (dtype, G, N, K, their addresses)."""
    d = _dtype(w, "w")
    if w.dim() != 3:
        raise ValueError(f"w must have shape (G, N, K), got {tuple(w.shape)}")
    G, N, K = w.shape
    return (d, G, N, K, _array(w, "w", w.dtype, (G, N, K)), _array(row_ptr, "row_ptr", torch.int32, (G + 1,)),
            None if perm is None else _array(perm, "perm", torch.int32, (M,)))


def _copies(w, perm):
    """Whether grouped products may lay out operands of weights like w anew."""
    return perm is not None or ((w.shape[1] | w.shape[2]) * w.element_size()) % 16 != 0


def zs_grouped_matmul(x: torch.Tensor, w: torch.Tensor, row_ptr: torch.Tensor, perm: torch.Tensor | None = None,
                      out=None, stream=None) -> torch.Tensor:
    """y[i] = w[g(i)] x[i] for rows grouped by the CSR (row_ptr, perm); perm None: rows
    are in group order already.  x (M, K) and w (G, N, K) float32, bfloat16 or
    float16; returns y (M, N).  x and out may be row-strided views."""
    if stream is not None:
        return _on(stream, zs_grouped_matmul, x, w, row_ptr, perm, out)
    if out is None:
        y = _fast.matmul(x, w, row_ptr, perm, False)
        if y is not NotImplemented:
            return y
    device = _elsewhere(x, w, row_ptr, perm, out)
    if device is not None:
        with torch.cuda.device(device):
            return zs_grouped_matmul(x, w, row_ptr, perm, out)
    M, _ = _rows(x, "x")
    d, G, N, K, wp, rp, pp = _groups(w, row_ptr, perm, M)
    dt = w.dtype
    x_ld = _matrix(x, "x", dt, M, K)
    out_ld = N
    if out is None:
        out = torch.empty((M, N), dtype=dt, device=x.device)
    else:
        out_ld = _matrix(out, "out", dt, M, N)
    lib = load()
    wbytes = lib.zs_grouped_matmul_workspace_bytes(d, M, K, N, G) if _copies(w, perm) else 0
    workspace = _workspace(wbytes, w.device)
    st = lib.zs_grouped_matmul_ws(d, x.data_ptr(), x_ld, wp, rp, pp, M, K, N, G, out.data_ptr(), out_ld, _ptr(workspace), wbytes,
                                _stream(None))
    if st:
        _check("zs_grouped_matmul_ws", st)
    return out


def zs_grouped_matmul_dx(dy: torch.Tensor, w: torch.Tensor, row_ptr: torch.Tensor, perm: torch.Tensor | None = None,
                         out=None, stream=None) -> torch.Tensor:
    """dx[i] = w[g(i)]^T dy[i]: the gradient of zs_grouped_matmul in x, (M, K)."""
    if stream is not None:
        return _on(stream, zs_grouped_matmul_dx, dy, w, row_ptr, perm, out)
    if out is None:
        dx = _fast.matmul(dy, w, row_ptr, perm, True)
        if dx is not NotImplemented:
            return dx
    device = _elsewhere(dy, w, row_ptr, perm, out)
    if device is not None:
        with torch.cuda.device(device):
            return zs_grouped_matmul_dx(dy, w, row_ptr, perm, out)
    M, _ = _rows(dy, "dy")
    d, G, N, K, wp, rp, pp = _groups(w, row_ptr, perm, M)
    dt = w.dtype
    dy_ld = _matrix(dy, "dy", dt, M, N)
    out_ld = K
    if out is None:
        out = torch.empty((M, K), dtype=dt, device=dy.device)
    else:
        out_ld = _matrix(out, "out", dt, M, K)
    lib = load()
    wbytes = lib.zs_grouped_matmul_workspace_bytes(d, M, K, N, G) if _copies(w, perm) else 0
    workspace = _workspace(wbytes, w.device)
    st = lib.zs_grouped_matmul_dx_ws(d, dy.data_ptr(), dy_ld, wp, rp, pp, M, K, N, G, out.data_ptr(), out_ld, _ptr(workspace), wbytes,
                                   _stream(None))
    if st:
        _check("zs_grouped_matmul_dx_ws", st)
    return out


def zs_grouped_matmul_dw_workspace_bytes(dtype: torch.dtype, M: int, K: int, N: int, G: int) -> int:
    return int(load().zs_grouped_matmul_dw_workspace_bytes(DTYPES[dtype], M, K, N, G))


def zs_grouped_matmul_dw(dy: torch.Tensor, x: torch.Tensor, row_ptr: torch.Tensor, perm: torch.Tensor | None = None,
                         out=None, workspace=None, stream=None) -> torch.Tensor:
    """dw[g] = sum over the rows of group g of dy[i] x[i]^T: the gradient of
    zs_grouped_matmul in w, (G, N, K) with G = row_ptr.numel() - 1."""
    if stream is not None:
        return _on(stream, zs_grouped_matmul_dw, dy, x, row_ptr, perm, out, workspace)
    if out is None and workspace is None:
        dw = _fast.dw(dy, x, row_ptr, perm)
        if dw is not NotImplemented:
            return dw
    device = _elsewhere(dy, x, row_ptr, perm, out, workspace)
    if device is not None:
        with torch.cuda.device(device):
            return zs_grouped_matmul_dw(dy, x, row_ptr, perm, out, workspace)
    M, K = _rows(x, "x")
    _, N = _rows(dy, "dy")
    G = row_ptr.numel() - 1
    d, dt, dev = _dtype(x, "x"), x.dtype, x.device
    x_ld = _matrix(x, "x", dt, M, K)
    dy_ld = _matrix(dy, "dy", dt, M, N)
    rp = _array(row_ptr, "row_ptr", torch.int32, (G + 1,))
    pp = None if perm is None else _array(perm, "perm", torch.int32, (M,))
    if out is None:
        out = torch.empty((G, N, K), dtype=dt, device=dev)
    op = _array(out, "out", dt, (G, N, K))
    lib = load()
    if workspace is None:
        wbytes = lib.zs_grouped_matmul_dw_workspace_bytes(d, M, K, N, G)
        if _copies(out, perm):
            wbytes += lib.zs_grouped_matmul_dw_copy_bytes(d, M, K, N, G)
        if wbytes:
            workspace = torch.empty(wbytes, dtype=torch.uint8, device=dev)
    else:
        wbytes = workspace.numel() * workspace.element_size()
    st = lib.zs_grouped_matmul_dw(d, dy.data_ptr(), dy_ld, x.data_ptr(), x_ld, rp, pp, M, K, N, G, op, _ptr(workspace),
                                  wbytes, _stream(None))
    if st:
        _check("zs_grouped_matmul_dw", st)
    return out


def zs_grouped_matmul_backward(dy: torch.Tensor, x: torch.Tensor, w: torch.Tensor, row_ptr: torch.Tensor,
                               perm: torch.Tensor | None = None, stream=None):
    """Both gradients of zs_grouped_matmul: (dx (M, K), dw (G, N, K))."""
    if stream is not None:
        return _on(stream, zs_grouped_matmul_backward, dy, x, w, row_ptr, perm)
    return (zs_grouped_matmul_dx(dy, w, row_ptr, perm),
            zs_grouped_matmul_dw(dy, x, row_ptr, perm))


def _norm_operands(h, x, gate, w_post, scale, w_pre, kind):
    """Checks the operands of the residual norms; returns (dtype, kind, M, C, the
    arguments h..w_pre of the C call)."""
    M, C = _rows(h, "h")
    d, dt = _dtype(h, "h"), h.dtype
    k = NORM_KINDS.get(kind)
    if k is None:
        raise ValueError(f"kind must be one of {sorted(NORM_KINDS)}, got {kind!r}")
    h_ld = _matrix(h, "h", dt, M, C)
    x_ld = _matrix(x, "x", dt, M, C)
    gate_ptr, gate_ld, gate_cols = None, 0, 0
    if gate is not None:
        gate_cols = gate.shape[1] if gate.dim() == 2 else 0
        if gate_cols != 1 and gate_cols != C:
            raise ValueError(f"gate must have shape {(M, C)} or {(M, 1)}, got {tuple(gate.shape)}")
        gate_ld = _matrix(gate, "gate", dt, M, gate_cols)
        gate_ptr = gate.data_ptr()
    f32, shape = torch.float32, (C,)
    return d, k, M, C, (h.data_ptr(), h_ld, x.data_ptr(), x_ld, gate_ptr, gate_ld, gate_cols,
                        _array(w_post, "w_post", f32, shape), _array(scale, "scale", f32, shape),
                        _array(w_pre, "w_pre", f32, shape))


def zs_norm_gate_residual(h: torch.Tensor, x: torch.Tensor, gate: torch.Tensor | None, w_post: torch.Tensor,
                          scale: torch.Tensor, w_pre: torch.Tensor, eps: float = 1e-6, kind: str = "rms",
                          want_stats: bool = True, stream=None):
    """y = x + scale * sigmoid(gate) * (norm(h) * w_post), u = norm(y) * w_pre.

    h, x (M, C) float32, bfloat16 or float16 (row-strided views allowed), gate the
    same, (M, 1), or None; w_post, scale, w_pre (C,) float32; kind "rms" or "layer".
    Returns (y, u, stats): stats (M, 4) float32 is what the backward reads (None
    when want_stats is False)."""
    if stream is not None:
        return _on(stream, zs_norm_gate_residual, h, x, gate, w_post, scale, w_pre, eps, kind, want_stats)
    if kind in NORM_KINDS:
        r = _fast.norm(h, x, gate, w_post, scale, w_pre, eps, NORM_KINDS[kind], want_stats)
        if r is not NotImplemented:
            return r
    device = _elsewhere(h, x, gate, w_post, scale, w_pre)
    if device is not None:
        with torch.cuda.device(device):
            return zs_norm_gate_residual(h, x, gate, w_post, scale, w_pre, eps, kind, want_stats)
    d, k, M, C, args = _norm_operands(h, x, gate, w_post, scale, w_pre, kind)
    dt, dev = h.dtype, h.device
    y = torch.empty((M, C), dtype=dt, device=dev)
    u = torch.empty((M, C), dtype=dt, device=dev)
    stats = torch.empty((M, 4), dtype=torch.float32, device=dev) if want_stats else None
    st = load().zs_norm_gate_residual(d, k, *args, eps, M, C, y.data_ptr(), u.data_ptr(),
                                      stats.data_ptr() if want_stats else None, _stream(None))
    if st:
        _check("zs_norm_gate_residual", st)
    return y, u, stats


def zs_norm_gate_residual_backward(dy: torch.Tensor | None, du: torch.Tensor | None, h: torch.Tensor, x: torch.Tensor,
                                   gate: torch.Tensor | None, w_post: torch.Tensor, scale: torch.Tensor,
                                   w_pre: torch.Tensor, stats: torch.Tensor, kind: str = "rms", stream=None):
    """Gradients of zs_norm_gate_residual for the cotangents dy of y and du of u (None:
    zeros): (dh, dx, dgate, dw_post, dscale, dw_pre); dgate is None without a gate."""
    if stream is not None:
        return _on(stream, zs_norm_gate_residual_backward, dy, du, h, x, gate, w_post, scale, w_pre, stats, kind)
    if kind in NORM_KINDS:
        r = _fast.norm_backward(dy, du, h, x, gate, w_post, scale, w_pre, stats, NORM_KINDS[kind])
        if r is not NotImplemented:
            return r
    device = _elsewhere(dy, du, h, x, gate, w_post, scale, w_pre, stats)
    if device is not None:
        with torch.cuda.device(device):
            return zs_norm_gate_residual_backward(dy, du, h, x, gate, w_post, scale, w_pre, stats, kind)
    d, k, M, C, args = _norm_operands(h, x, gate, w_post, scale, w_pre, kind)
    dt, dev, f32 = h.dtype, h.device, torch.float32
    dy_ld = 0 if dy is None else _matrix(dy, "dy", dt, M, C)
    du_ld = 0 if du is None else _matrix(du, "du", dt, M, C)
    stats_ptr = _array(stats, "stats", f32, (M, 4))
    dh = torch.empty((M, C), dtype=dt, device=dev)
    dx = torch.empty((M, C), dtype=dt, device=dev)
    dgate = None if gate is None else torch.empty((M, args[6]), dtype=dt, device=dev)
    sums = [torch.empty((C,), dtype=f32, device=dev) for _ in range(3)]
    lib = load()
    need = lib.zs_norm_gate_residual_backward_workspace_bytes(M, C)
    workspace = _workspace(need, dev)
    st = lib.zs_norm_gate_residual_backward(
        d, k, None if dy is None else dy.data_ptr(), dy_ld, None if du is None else du.data_ptr(), du_ld, *args, stats_ptr,
        M, C, dh.data_ptr(), dx.data_ptr(), None if gate is None else dgate.data_ptr(), *(t.data_ptr() for t in sums),
        _ptr(workspace), need, _stream(None))
    if st:
        _check("zs_norm_gate_residual_backward", st)
    return dh, dx, dgate, *sums


class _AdamWTensor(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("grad", ctypes.c_void_p), ("exp_avg", ctypes.c_void_p),
                ("exp_avg_sq", ctypes.c_void_p), ("exp_avg_scale", ctypes.c_void_p),
                ("exp_avg_sq_scale", ctypes.c_void_p), ("numel", ctypes.c_int64)]


class _AdamWHyper(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("weight_decay", ctypes.c_double), ("step", ctypes.c_int64)]


class AdamWPlan:
    """The tensors of an AdamW step, checked once: lists of parameters, gradients and
    states, on one device, every parameter and gradient of one type.

    32-bit states: exp_avg and exp_avg_sq float32 of the parameters' sizes.  8-bit
    states: torch.float8_e4m3fn of the parameters' sizes (exp_avg_sq holds the root of
    the second moment), with exp_avg_scale and exp_avg_sq_scale float32 of
    ceil(numel / 256) elements each.  Every tensor is contiguous; the plan is of the
    memory that it has when the plan is made, which it holds, and ``zs_adamw_step``
    updates that.  ``set_grads`` puts other gradients (of the same sizes) in place of the
    plan's."""

    def __init__(self, params, grads, exp_avg, exp_avg_sq, exp_avg_scale=None, exp_avg_sq_scale=None):
        self.params, self.exp_avg, self.exp_avg_sq = list(params), list(exp_avg), list(exp_avg_sq)
        n = len(self.params)
        if not n:
            raise ValueError("a plan needs at least one parameter")
        if (exp_avg_scale is None) != (exp_avg_sq_scale is None):
            raise ValueError("8-bit states take both lists of scales, 32-bit states none")
        self.state_bits = 32 if exp_avg_scale is None else 8
        self.scales = [] if exp_avg_scale is None else [list(exp_avg_scale), list(exp_avg_sq_scale)]
        self.dtype = _dtype(self.params[0], "params[0]")
        self.device = self.params[0].device
        self._index = self.device.index
        self._table = (_AdamWTensor * n)()
        state_dtype = torch.float32 if self.state_bits == 32 else torch.float8_e4m3fn
        for lst, name in ((self.exp_avg, "exp_avg"), (self.exp_avg_sq, "exp_avg_sq"),
                          *zip(self.scales, ("exp_avg_scale", "exp_avg_sq_scale"))):
            if len(lst) != n:
                raise ValueError(f"{name} has {len(lst)} tensors, params {n}")
        for i, p in enumerate(self.params):
            e = self._table[i]
            self._one(p, f"params[{i}]", self.params[0].dtype, p.shape)
            self._one(self.exp_avg[i], f"exp_avg[{i}]", state_dtype, p.shape)
            self._one(self.exp_avg_sq[i], f"exp_avg_sq[{i}]", state_dtype, p.shape)
            e.param, e.exp_avg, e.exp_avg_sq = _ptr(p), _ptr(self.exp_avg[i]), _ptr(self.exp_avg_sq[i])
            e.numel = p.numel()
            if self.scales:
                for lst, name in zip(self.scales, ("exp_avg_scale", "exp_avg_sq_scale")):
                    self._one(lst[i], f"{name}[{i}]", torch.float32, (-(-p.numel() // ADAMW_BLOCK),))
                    setattr(e, name, _ptr(lst[i]))
        self._table_ptr = ctypes.addressof(self._table)
        self._shapes, self._param_at = [p.shape for p in self.params], [p.data_ptr() for p in self.params]
        written = sorted((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size())
                         for t in (*self.params, *self.exp_avg, *self.exp_avg_sq, *sum(self.scales, [])) if t.numel() and t.data_ptr())
        if any(end > start for (_, end), (start, _) in zip(written, written[1:])):
            raise ValueError("parameters and states must not overlap, nor be given twice")
        # a tensor's memory may be taken from it (t.data = other): it is held by itself
        self._memory = [t.untyped_storage() for t in (*self.params, *self.exp_avg, *self.exp_avg_sq, *sum(self.scales, []))]
        self.set_grads(grads)

    def _one(self, t, name, dtype, shape):
        if t.dtype is dtype and t.shape == shape and t.get_device() == self._index and t.is_contiguous():
            return
        _need(t, name, dtype, tuple(shape))
        if t.device != self.device:
            raise ValueError(f"{name} is on {t.device}, the plan on {self.device}")

    def set_grads(self, grads) -> None:
        grads = list(grads)
        if len(grads) != len(self.params):
            raise ValueError(f"grads has {len(grads)} tensors, params {len(self.params)}")
        dtype = self.params[0].dtype
        for i, (g, shape) in enumerate(zip(grads, self._shapes)):
            self._one(g, f"grads[{i}]", dtype, shape)
        self.grads, self._grad_at = grads, [g.data_ptr() for g in grads]
        for i, at in enumerate(self._grad_at):
            self._table[i].grad = at or None
        self._grad_memory = [g.untyped_storage() for g in grads]

    def has_grads(self, grads) -> bool:
        """Whether these tensors, where they are now, are the plan's gradients."""
        return [g.data_ptr() for g in grads] == self._grad_at and [g.shape for g in grads] == self._shapes

    def has_params(self, params) -> bool:
        """Whether these tensors, where they are now, are the plan's parameters."""
        return [p.data_ptr() for p in params] == self._param_at


def zs_adamw_step(plan: AdamWPlan, step: int, lr: float, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
                  weight_decay: float = 0.01, grad_scale: torch.Tensor | None = None, stream=None,
                  seed: int | None = None) -> None:
    """One AdamW step (number ``step``, from 1) over the plan's tensors, in place.
    grad_scale: one float32 element on the device that multiplies every gradient.
    8-bit states are rounded to nearest, which leaves a second moment where it is when
    it shrinks slowly, or with a ``seed`` at random by bits that follow from it and the
    step, as a training run needs them."""
    scale_ptr = None
    if grad_scale is not None:
        if grad_scale.numel() != 1 or grad_scale.dtype != torch.float32 or grad_scale.device != plan.device:
            raise ValueError(f"grad_scale must be one float32 element on {plan.device}")
        scale_ptr = grad_scale.data_ptr()
    if stream is not None and isinstance(stream, torch.cuda.Stream):
        _one_device((plan.params[0],), stream.device)
    if plan._index != _current_device():   # a launch is the current device's
        with torch.cuda.device(plan.device):
            return zs_adamw_step(plan, step, lr, beta1, beta2, eps, weight_decay, grad_scale, stream, seed)
    hyper = _AdamWHyper(lr, beta1, beta2, eps, weight_decay, step)
    if seed is None:
        st = load().zs_adamw_step(plan._table_ptr, len(plan.params), plan.dtype, plan.state_bits, ctypes.addressof(hyper),
                                  scale_ptr, _stream(stream))
    else:
        st = load().zs_adamw_step_seeded(plan._table_ptr, len(plan.params), plan.dtype, plan.state_bits,
                                         ctypes.addressof(hyper), seed & (1 << 64) - 1, scale_ptr, _stream(stream))
    if st:
        _check("zs_adamw_step", st)


# ---------------------------------------------------------------------------
# A block whose rows go to several experts: embedding, routing, the way to the
# experts' grouped products and back, dropout.

SCORE_KINDS = {"softmax": 0, "sigmoid": 1}


def _int(value, name: str, lo: int, hi: int) -> int:
    """An integer in [lo, hi]: what the C call's argument can hold."""
    value = operator.index(value)
    if not lo <= value <= hi:
        raise ValueError(f"{name} must be in [{lo}, {hi}], got {value}")
    return value


_I32, _U32 = (1 << 31) - 1, (1 << 32) - 1


def zs_embedding(w: torch.Tensor, ids: torch.Tensor, scale: float = 1.0, stream=None) -> torch.Tensor:
    """y[i] = scale * w[ids[i]]: w (V, C) float32, bfloat16 or float16 (a row-strided view
    allowed), ids (M,) int32; rows of ids outside [0, V) are zeros.  Returns y (M, C)."""
    if stream is not None:
        return _on(stream, zs_embedding, w, ids, scale)
    y = _fast.embedding(w, ids, scale)
    if y is not NotImplemented:
        return y
    device = _elsewhere(w, ids)
    if device is not None:
        with torch.cuda.device(device):
            return zs_embedding(w, ids, scale)
    V, C = _rows(w, "w")
    d, M = _dtype(w, "w"), ids.numel()
    ld = _matrix(w, "w", w.dtype, V, C)
    ip = _array(ids, "ids", torch.int32, (M,))
    y = torch.empty((M, C), dtype=w.dtype, device=w.device)
    st = load().zs_embedding(d, _ptr(w), ld, ip, M, _int(V, "V", 0, _I32), _int(C, "C", 0, _I32), scale, _ptr(y), C, _stream(None))
    if st:
        _check("zs_embedding", st)
    return y


def zs_embedding_backward(dy: torch.Tensor, row_ptr: torch.Tensor, perm: torch.Tensor, scale: float = 1.0,
                          stream=None) -> torch.Tensor:
    """dw[v] = scale * the sum of dy over the rows that hold v: the gradient of zs_embedding in
    w, (V, C) of dy's type, from the CSR (row_ptr (V+1,), perm (M,)) of zs_build_csr(ids, V)."""
    if stream is not None:
        return _on(stream, zs_embedding_backward, dy, row_ptr, perm, scale)
    dw = _fast.embedding_backward(dy, row_ptr, perm, scale)
    if dw is not NotImplemented:
        return dw
    device = _elsewhere(dy, row_ptr, perm)
    if device is not None:
        with torch.cuda.device(device):
            return zs_embedding_backward(dy, row_ptr, perm, scale)
    M, C = _rows(dy, "dy")
    d, V = _dtype(dy, "dy"), row_ptr.numel() - 1
    _int(V, "V = row_ptr.numel() - 1", 0, _I32), _int(C, "C", 0, _I32)
    ld = _matrix(dy, "dy", dy.dtype, M, C)
    rp, pp = _array(row_ptr, "row_ptr", torch.int32, (V + 1,)), _array(perm, "perm", torch.int32, (M,))
    dw = torch.empty((V, C), dtype=dy.dtype, device=dy.device)
    lib = load()
    need = lib.zs_embedding_backward_workspace_bytes(d, M, V, C)
    workspace = _workspace(need, dy.device)
    st = lib.zs_embedding_backward(d, _ptr(dy), ld, rp, pp, M, V, C, scale, _ptr(dw), _ptr(workspace), need, _stream(None))
    if st:
        _check("zs_embedding_backward", st)
    return dw


def _score(score: str) -> int:
    kind = SCORE_KINDS.get(score)
    if kind is None:
        raise ValueError(f"score must be one of {sorted(SCORE_KINDS)}, got {score!r}")
    return kind


def zs_route(logits: torch.Tensor, k: int, bias: torch.Tensor | None = None, score: str = "softmax", groups: int = 1,
             top_groups: int | None = None, group_top: int = 1, renormalise: bool = True, scale: float = 1.0, stream=None):
    """The k experts of each row with the largest score + bias among its best groups of
    experts, and their weights.

    logits (M, E) float32, bfloat16 or float16 (a row-strided view allowed; -inf closes an
    expert to a row), bias (E,) float32 or None (it counts for the choice alone), score
    "softmax" or "sigmoid".  The experts are in ``groups`` groups in a row; a group's value is
    the sum of its ``group_top`` (1 or 2) largest score + bias, and only the ``top_groups``
    groups with the largest values are open (None: all).  Returns (ids (M, k) int32, weights
    (M, k) float32): ids in descending order, equal ones by index, -1 behind the last open
    expert; weights scale * score, of scores divided by their sum over the row's choices with
    ``renormalise``."""
    if stream is not None:
        return _on(stream, zs_route, logits, k, bias, score, groups, top_groups, group_top, renormalise, scale)
    if score in SCORE_KINDS:
        r = _fast.route(logits, k, bias, SCORE_KINDS[score], groups, groups if top_groups is None else top_groups, group_top,
                        renormalise, scale)
        if r is not NotImplemented:
            return r
    device = _elsewhere(logits, bias)
    if device is not None:
        with torch.cuda.device(device):
            return zs_route(logits, k, bias, score, groups, top_groups, group_top, renormalise, scale)
    kind = _score(score)
    M, E = _rows(logits, "logits")
    d = _dtype(logits, "logits")
    ld = _matrix(logits, "logits", logits.dtype, M, E)
    bp = None if bias is None else _array(bias, "bias", torch.float32, (E,))
    k, groups = _int(k, "k", 1, E), _int(groups, "groups", 1, _I32)
    top_groups = groups if top_groups is None else _int(top_groups, "top_groups", 1, _I32)
    ids = torch.empty((M, k), dtype=torch.int32, device=logits.device)
    weights = torch.empty((M, k), dtype=torch.float32, device=logits.device)
    st = load().zs_route(d, kind, _ptr(logits), ld, bp, M, _int(E, "E", 0, _I32), k, groups, top_groups,
                         _int(group_top, "group_top", 1, 2), bool(renormalise), scale, _ptr(ids), _ptr(weights), _stream(None))
    if st:
        _check("zs_route", st)
    return ids, weights


def zs_route_backward(dweights: torch.Tensor, logits: torch.Tensor, ids: torch.Tensor, score: str = "softmax",
                      renormalise: bool = True, scale: float = 1.0, stream=None) -> torch.Tensor:
    """The gradient of zs_route's weights in the logits, the choice ``ids`` held fixed:
    dlogits (M, E) of the logits' type for the cotangent dweights (M, k) float32."""
    if stream is not None:
        return _on(stream, zs_route_backward, dweights, logits, ids, score, renormalise, scale)
    if score in SCORE_KINDS:
        r = _fast.route_backward(dweights, logits, ids, SCORE_KINDS[score], renormalise, scale)
        if r is not NotImplemented:
            return r
    device = _elsewhere(dweights, logits, ids)
    if device is not None:
        with torch.cuda.device(device):
            return zs_route_backward(dweights, logits, ids, score, renormalise, scale)
    kind = _score(score)
    M, E = _rows(logits, "logits")
    _, k = _rows(ids, "ids")
    d = _dtype(logits, "logits")
    ld = _matrix(logits, "logits", logits.dtype, M, E)
    ip, gp = _array(ids, "ids", torch.int32, (M, k)), _array(dweights, "dweights", torch.float32, (M, k))
    dlogits = torch.empty((M, E), dtype=logits.dtype, device=logits.device)
    st = load().zs_route_backward(d, kind, gp, _ptr(logits), ld, ip, M, _int(E, "E", 0, _I32), k, bool(renormalise), scale,
                                  _ptr(dlogits), _stream(None))
    if st:
        _check("zs_route_backward", st)
    return dlogits


def zs_dispatch(x: torch.Tensor, row_ptr: torch.Tensor, perm: torch.Tensor, k: int, stream=None):
    """Rows to their experts: with (row_ptr (G+1,), perm (M*k,)) the CSR zs_build_csr gives for the
    flattened ids (M, k) of zs_route, xs[p] = x[perm[p] // k] (zeros from position row_ptr[G]),
    in the order of zs_grouped_matmul without a perm, and slot[perm[p]] = p (-1 without a group).
    x (M, C) float32, bfloat16 or float16 (a row-strided view allowed).  Returns (xs (M*k, C),
    slot (M, k) int32)."""
    if stream is not None:
        return _on(stream, zs_dispatch, x, row_ptr, perm, k)
    r = _fast.dispatch(x, row_ptr, perm, k)
    if r is not NotImplemented:
        return r
    device = _elsewhere(x, row_ptr, perm)
    if device is not None:
        with torch.cuda.device(device):
            return zs_dispatch(x, row_ptr, perm, k)
    M, C = _rows(x, "x")
    d, k, G = _dtype(x, "x"), _int(k, "k", 1, _I32), row_ptr.numel() - 1
    ld = _matrix(x, "x", x.dtype, M, C)
    rp, pp = _array(row_ptr, "row_ptr", torch.int32, (G + 1,)), _array(perm, "perm", torch.int32, (M * k,))
    xs = torch.empty((M * k, C), dtype=x.dtype, device=x.device)
    slot = torch.empty((M, k), dtype=torch.int32, device=x.device)
    st = load().zs_dispatch(d, _ptr(x), ld, rp, pp, M, k, _int(G, "G = row_ptr.numel() - 1", 0, _I32), _int(C, "C", 0, _I32), _ptr(xs),
                            _ptr(slot), _stream(None))
    if st:
        _check("zs_dispatch", st)
    return xs, slot


def zs_combine(h: torch.Tensor, slot: torch.Tensor, weights: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """And back: y[i] = the sum over j of weights[i, j] * h[slot[i, j]]; slots outside [0, R) add
    nothing.  h (R, C) float32, bfloat16 or float16 (a row-strided view allowed), slot (M, k)
    int32, weights (M, k) float32.  Without weights it is the gradient of zs_dispatch in x."""
    if stream is not None:
        return _on(stream, zs_combine, h, slot, weights)
    y = _fast.combine(h, slot, weights)
    if y is not NotImplemented:
        return y
    device = _elsewhere(h, slot, weights)
    if device is not None:
        with torch.cuda.device(device):
            return zs_combine(h, slot, weights)
    R, C = _rows(h, "h")
    M, k = _rows(slot, "slot")
    d = _dtype(h, "h")
    ld = _matrix(h, "h", h.dtype, R, C)
    sp = _array(slot, "slot", torch.int32, (M, k))
    wp = None if weights is None else _array(weights, "weights", torch.float32, (M, k))
    y = torch.empty((M, C), dtype=h.dtype, device=h.device)
    st = load().zs_combine(d, _ptr(h), ld, sp, wp, M, _int(k, "k", 1, _I32), R, _int(C, "C", 0, _I32), _ptr(y), C, _stream(None))
    if st:
        _check("zs_combine", st)
    return y


def zs_combine_backward(dy: torch.Tensor, h: torch.Tensor, slot: torch.Tensor, weights: torch.Tensor, row_ptr: torch.Tensor,
                        stream=None):
    """Gradients of zs_combine with weights, for the slots and the CSR's row_ptr of zs_dispatch:
    (dh (M*k, C), zeros from position row_ptr[G]; dweights (M, k) float32, 0 without a slot)."""
    if stream is not None:
        return _on(stream, zs_combine_backward, dy, h, slot, weights, row_ptr)
    r = _fast.combine_backward(dy, h, slot, weights, row_ptr)
    if r is not NotImplemented:
        return r
    device = _elsewhere(dy, h, slot, weights, row_ptr)
    if device is not None:
        with torch.cuda.device(device):
            return zs_combine_backward(dy, h, slot, weights, row_ptr)
    _, C = _rows(h, "h")
    M, k = _rows(slot, "slot")
    d, dt, G = _dtype(h, "h"), h.dtype, row_ptr.numel() - 1
    h_ld = _matrix(h, "h", dt, M * k, C)
    dy_ld = _matrix(dy, "dy", dt, M, C)
    sp, wp = _array(slot, "slot", torch.int32, (M, k)), _array(weights, "weights", torch.float32, (M, k))
    rp = _array(row_ptr, "row_ptr", torch.int32, (G + 1,))
    dh = torch.empty((M * k, C), dtype=dt, device=h.device)
    dweights = torch.empty((M, k), dtype=torch.float32, device=h.device)
    st = load().zs_combine_backward(d, _ptr(dy), dy_ld, _ptr(h), h_ld, sp, wp, rp, M, _int(k, "k", 1, _I32),
                                    _int(G, "G = row_ptr.numel() - 1", 0, _I32), _int(C, "C", 0, _I32), _ptr(dh), _ptr(dweights),
                                    _stream(None))
    if st:
        _check("zs_combine_backward", st)
    return dh, dweights


def zs_dropout(h: torch.Tensor, p: float, seed: int, call: int = 0, step: int | torch.Tensor = 0,
               residual: torch.Tensor | None = None, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """residual + dropout(h): elements are dropped with probability p (to 1 / 65536), the others
    divided by 1 - p.  The mask follows from the elements' numbers in their order, the seed (64
    bits), ``call`` (32 bits: which of a step's dropouts this is) and ``step``: a number, or one
    int64 element on the device, which a captured call reads at each replay.  It is drawn again
    where it is needed: the gradient in h is zs_dropout(dy, p, seed, call, step).

    h float32, bfloat16 or float16, of any shape where it is contiguous, or a matrix with
    contiguous rows; residual and out like h (out may be h or residual)."""
    if stream is not None:
        return _on(stream, zs_dropout, h, p, seed, call, step, residual, out)
    if out is None:
        y = _fast.dropout(h, p, seed, call, step, residual)
        if y is not NotImplemented:
            return y
    device = _elsewhere(h, residual, out, step)
    if device is not None:
        with torch.cuda.device(device):
            return zs_dropout(h, p, seed, call, step, residual, out)
    d, shape = _dtype(h, "h"), h.shape
    if out is None:
        out = torch.empty(shape, dtype=h.dtype, device=h.device)
    given = {"h": h, "residual": residual, "out": out}
    if h.dim() == 2:
        M, C = shape
        at = {n: (None, 0) if t is None else (_ptr(t), _matrix(t, n, h.dtype, M, C)) for n, t in given.items()}
    else:
        C = int(shape[-1]) if h.dim() else 1
        M = h.numel() // C if C else 0
        at = {n: (None, 0) if t is None else (_array(t, n, h.dtype, shape) or None, C) for n, t in given.items()}
    call, step_ptr = _int(call, "call", 0, _U32), None
    if isinstance(step, torch.Tensor):
        if not step.is_cuda or step.dtype != torch.int64 or step.numel() != 1:
            raise ValueError("step must be a number or one int64 element on the device")
        step_ptr, step = step.data_ptr(), 0
    if M * C == 0:
        return out
    st = load().zs_dropout(d, *at["h"], *at["residual"], M, _int(C, "C", 0, _I32), p, operator.index(seed) & (1 << 64) - 1, call,
                           _int(step, "step", -1 << 63, (1 << 63) - 1), step_ptr, *at["out"], _stream(None))
    if st:
        _check("zs_dropout", st)
    return out
