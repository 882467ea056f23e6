"""ctypes binding of the operators in include/moe_proj.h (argument marshalling only).

What a server of many requests has around the two halves of a layer: the
residual's addition and the RMS norm, in bf16 and in E4M3 with scales
(moe_proj_norm), the FP8 projection that takes such rows (moe_proj_fp8), and
each request's own low-rank adapter beside a projection (moe_proj_lora).  As in
capi.py, every function checks dtype, shape, device and contiguity of its
tensors, passes their device pointers and torch's current HIP stream, and raises
MoeMlpError on a non-zero status; the library does all of the computing.

bind_norm, bind_fp8 and bind_lora check and marshal once and return a callable
that issues the call again on the same buffers (serving loops), on the stream
given when binding, or with none given on torch's current stream of the buffers'
device at the time of each call.  Calls of one bind_lora callable share its
workspace: two of them must not run at the same time, and a graph that has
captured one needs the callable for as long as it is replayed.

E4M3 tensors are torch.uint8, or torch.float8_e4m3fn.
"""
from __future__ import annotations

import ctypes
import dataclasses
from typing import Optional

import torch

from . import attention, capi
from .attention import _bytes_on_stream, _one_device
from .capi import _check, _check_tensor, _ptr

BLOCK = capi.FP8_BLOCK
NORM_MAX_HIDDEN = 16384
LORA_MAX_RANK = 256
MAX_FEATURES = 1 << 20

EXPORTED = ("moe_proj_norm", "moe_proj_fp8", "moe_proj_lora_workspace_size", "moe_proj_lora")


class moe_proj_adapters(ctypes.Structure):
    _fields_ = [("a", ctypes.c_void_p), ("b", ctypes.c_void_p), ("ranks", ctypes.c_void_p),
                ("scales", ctypes.c_void_p), ("n_adapters", ctypes.c_int64), ("max_rank", ctypes.c_int32),
                ("in_features", ctypes.c_int32), ("out_features", ctypes.c_int32)]


_READY = False


def _lib() -> ctypes.CDLL:
    global _READY
    L = capi.lib()
    if not _READY:
        vp, i64, sz, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
        ap = ctypes.POINTER(moe_proj_adapters)
        L.moe_proj_norm.argtypes = [vp, i64, vp, vp, f32, i64, i64, vp, vp, vp, vp, vp]
        L.moe_proj_fp8.argtypes = [vp, vp, vp, vp, i64, i64, i64, vp, vp]
        L.moe_proj_lora_workspace_size.argtypes = [ap, i64, ctypes.POINTER(sz)]
        L.moe_proj_lora.argtypes = [ap, vp, i64, i64, vp, vp, i64, vp, i64, vp, sz, vp]
        for n in EXPORTED:
            getattr(L, n).restype = ctypes.c_int
        _READY = True
    return L


def _callable(*args):
    _lib()
    return attention._callable(*args)


@dataclasses.dataclass
class Adapters:
    """Low-rank adapters of one projection: out += scales[a] * (x a^T) b^T."""
    a: torch.Tensor                         # [n, max_rank, in_features] bf16
    b: torch.Tensor                         # [n, out_features, max_rank] bf16
    ranks: Optional[torch.Tensor] = None    # [n] i32, up to max_rank; None: max_rank
    scales: Optional[torch.Tensor] = None   # [n] f32; None: ones

    def check(self) -> None:
        n, r, k = self.a.shape if isinstance(self.a, torch.Tensor) and self.a.dim() == 3 else (-1, -1, -1)
        _check_tensor(self.a, "adapters.a", (n, r, k), torch.bfloat16)
        out = self.b.shape[1] if isinstance(self.b, torch.Tensor) and self.b.dim() == 3 else -1
        _check_tensor(self.b, "adapters.b", (n, out, r), torch.bfloat16)
        if self.ranks is not None:
            _check_tensor(self.ranks, "adapters.ranks", (n,), torch.int32)
        if self.scales is not None:
            _check_tensor(self.scales, "adapters.scales", (n,), torch.float32)

    def c(self) -> moe_proj_adapters:
        n, r, k = self.a.shape
        return moe_proj_adapters(_ptr(self.a), _ptr(self.b), _ptr(self.ranks), _ptr(self.scales), n, r, k,
                                 self.b.shape[1])


def _check_bytes(t, name, shape) -> None:
    """An E4M3 tensor."""
    f8 = isinstance(t, torch.Tensor) and t.dtype == torch.float8_e4m3fn
    _check_tensor(t, name, shape, torch.float8_e4m3fn if f8 else torch.uint8)


def _rows(t, name, width, T=None) -> int:
    """Checks a bf16 matrix whose rows are `width` long and may be apart (columns of a wider tensor); its stride."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {torch.bfloat16}")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a device (HIP) tensor")
    if t.dim() != 2 or t.shape[1] != width or (T is not None and t.shape[0] != T) or \
            (t.shape[0] and width > 1 and t.stride(1) != 1):
        raise ValueError(f"{name}: shape {tuple(t.shape)} with strides {t.stride()}, expected "
                         f"{'' if T is None else T} rows of {width} values")
    return t.stride(0) if t.shape[0] > 1 else width


def bind_norm(x: torch.Tensor, weight: Optional[torch.Tensor], eps: float, residual: Optional[torch.Tensor] = None,
              h_out: Optional[torch.Tensor] = None, y_out: Optional[torch.Tensor] = None,
              q_out: Optional[torch.Tensor] = None, q_scale: Optional[torch.Tensor] = None, stream=None):
    """moe_proj_norm on these buffers, as a callable (its stream: see the module)."""
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError("x must be a [T, hidden] tensor")
    T, H = x.shape
    stride = _rows(x, "x", H)
    for n, t in (("residual", residual), ("h_out", h_out), ("y_out", y_out)):
        if t is not None:
            _check_tensor(t, n, (T, H), torch.bfloat16)
    if weight is not None:
        _check_tensor(weight, "weight", (H,), torch.float32)
    if q_out is not None:
        _check_bytes(q_out, "q_out", (T, H))
    if q_scale is not None:
        _check_tensor(q_scale, "q_scale", (T, -(-H // BLOCK)), torch.float32)
    _one_device(x=x, weight=weight, residual=residual, h_out=h_out, y_out=y_out, q_out=q_out, q_scale=q_scale)
    args = (x.data_ptr(), stride, _ptr(residual), _ptr(weight), ctypes.c_float(eps), T, H, _ptr(h_out), _ptr(y_out),
            _ptr(q_out), _ptr(q_scale))
    return _callable("moe_proj_norm", args, stream, x.device.index,
                     (x, weight, residual, h_out, y_out, q_out, q_scale))


def bind_fp8(x: torch.Tensor, x_scale: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor, y: torch.Tensor,
             stream=None):
    """moe_proj_fp8 on these buffers, as a callable (its stream: see the module)."""
    T, K = x.shape if isinstance(x, torch.Tensor) and x.dim() == 2 else (-1, -1)
    N = w.shape[0] if isinstance(w, torch.Tensor) and w.dim() == 2 else -1
    _check_bytes(x, "x", (T, K))
    _check_bytes(w, "w", (N, K))
    _check_tensor(x_scale, "x_scale", (T, K // BLOCK), torch.float32)
    _check_tensor(w_scale, "w_scale", (-(-N // BLOCK), K // BLOCK), torch.float32)
    _check_tensor(y, "y", (T, N), torch.bfloat16)
    _one_device(x=x, x_scale=x_scale, w=w, w_scale=w_scale, y=y)
    args = (x.data_ptr(), x_scale.data_ptr(), w.data_ptr(), w_scale.data_ptr(), T, N, K, y.data_ptr())
    return _callable("moe_proj_fp8", args, stream, x.device.index, (x, x_scale, w, w_scale, y))


def moe_proj_lora_workspace_size(adapters: Adapters, T: int) -> int:
    """Bytes for T tokens, or fewer."""
    n = ctypes.c_size_t(0)
    _check(_lib().moe_proj_lora_workspace_size(ctypes.byref(adapters.c()), int(T), ctypes.byref(n)),
           "moe_proj_lora_workspace_size")
    return n.value


def lora_workspace(adapters: Adapters, T: int, device="cuda") -> torch.Tensor:
    """A workspace tensor of the size the library asks for (allocated by torch)."""
    return torch.empty(max(1, moe_proj_lora_workspace_size(adapters, T)), dtype=torch.uint8, device=device)


def bind_lora(adapters: Adapters, x: torch.Tensor, adapter: torch.Tensor, base: torch.Tensor,
              out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None, stream=None):
    """moe_proj_lora on these buffers (out None: into base), as a callable (its stream: see the module)."""
    adapters.check()
    T = adapter.shape[0] if isinstance(adapter, torch.Tensor) and adapter.dim() == 1 else -1
    _check_tensor(adapter, "adapter", (T,), torch.int32)
    out = base if out is None else out
    K, N = adapters.a.shape[2], adapters.b.shape[1]
    xs, bs, os = (_rows(t, n, w, T) for n, t, w in (("x", x, K), ("base", base, N), ("out", out, N)))
    own = ws is None
    if own:
        ws = _bytes_on_stream(moe_proj_lora_workspace_size(adapters, T), x.device, stream)
    _check_tensor(ws, "workspace", None, torch.uint8)
    _one_device(a=adapters.a, b=adapters.b, ranks=adapters.ranks, scales=adapters.scales, x=x, adapter=adapter,
                base=base, out=out, workspace=ws)
    c = adapters.c()
    args = (ctypes.byref(c), x.data_ptr(), xs, T, adapter.data_ptr(), base.data_ptr(), bs, out.data_ptr(), os,
            ws.data_ptr(), ws.numel())
    return _callable("moe_proj_lora", args, stream, x.device.index, (c, adapters, x, adapter, base, out, ws),
                     ws if own else None)


def moe_proj_norm(x: torch.Tensor, weight: Optional[torch.Tensor], eps: float,
                  residual: Optional[torch.Tensor] = None, h_out: Optional[torch.Tensor] = None,
                  y_out: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None,
                  q_scale: Optional[torch.Tensor] = None, stream=None) -> None:
    """h = x + residual to h_out, its RMS norm to y_out (bf16) and to q_out with q_scale (E4M3, a scale per 128
    columns); every output is optional, but one of y_out and q_out is needed."""
    bind_norm(x, weight, eps, residual, h_out, y_out, q_out, q_scale, stream)()


def moe_proj_fp8(x: torch.Tensor, x_scale: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor, y: torch.Tensor,
                 stream=None) -> None:
    """y [T, N] = x w^T of E4M3 rows x [T, K] (scales [T, K / 128]) and weights w [N, K] (scales per 128 x 128)."""
    bind_fp8(x, x_scale, w, w_scale, y, stream)()


def moe_proj_lora(adapters: Adapters, x: torch.Tensor, adapter: torch.Tensor, base: torch.Tensor,
                  out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None, stream=None) -> None:
    """out [T, out_features] (None: base itself) = base + the tokens' own adapters of x; adapter [T] names them, any
    number that none has: no adapter."""
    bind_lora(adapters, x, adapter, base, out, ws, stream)()
