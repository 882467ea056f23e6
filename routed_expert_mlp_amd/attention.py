"""ctypes binding of the attention operators in include/moe_attn.h (argument marshalling only).

The attention half of the decoder layer whose MLP half capi.py binds: head
norms, rotation and cache append of new tokens (moe_attn_prepare), attention of
a few new tokens per sequence over the paged cache (moe_attn_decode) and of
prompts or pieces of prompts (moe_attn_prefill).  As in capi.py, every function
checks dtype, shape, device and contiguity of its tensors, passes their device
pointers and torch's current HIP stream, and raises MoeMlpError on a non-zero
status; the library does all of the computing.

bind_prepare, bind_decode and bind_prefill check and marshal once and return a
callable that issues the call again on the same buffers (serving loops).  It
goes to the stream given when binding; with none given, to torch's current
stream of the buffers' device at the time of each call, so that it can be
called, or captured, under another stream than it was bound under.  Calls of one
callable share its workspace: two of them must not run at the same time, and a
graph that has captured one needs the callable for as long as it is replayed.
"""
from __future__ import annotations

import ctypes
import dataclasses
from typing import Optional

import torch

from . import capi
from .capi import _check, _check_tensor, _ptr, _stream

ROPE_HALF = 0
ROPE_INTERLEAVED = 1
MAX_HEADS = 1024
DECODE_MAX_Q = 8

EXPORTED = ("moe_attn_prepare", "moe_attn_workspace_size", "moe_attn_workspace_bound", "moe_attn_decode",
            "moe_attn_prefill")


class moe_attn_config(ctypes.Structure):
    _fields_ = [("n_heads", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("rotary_dim", ctypes.c_int32), ("rope_style", ctypes.c_int32),
                ("window", ctypes.c_int32), ("n_sinks", ctypes.c_int32), ("norm_eps", ctypes.c_float),
                ("scale", ctypes.c_float)]


class moe_attn_cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("n_pages", ctypes.c_int64)]


_READY = False


def _lib() -> ctypes.CDLL:
    global _READY
    L = capi.lib()
    if not _READY:
        vp, i64, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t
        cfgp, cp = ctypes.POINTER(moe_attn_config), ctypes.POINTER(moe_attn_cache)
        L.moe_attn_prepare.argtypes = [cfgp, cp, vp, i64, i64, vp, vp, vp, i64, vp, vp, vp, vp]
        L.moe_attn_workspace_size.argtypes = [cfgp, i64, i64, i64, i64, ctypes.c_int, ctypes.POINTER(sz)]
        L.moe_attn_workspace_bound.argtypes = L.moe_attn_workspace_size.argtypes
        L.moe_attn_decode.argtypes = [cfgp, cp, vp, i64, i64, vp, vp, i64, i64, vp, vp, sz, vp]
        L.moe_attn_prefill.argtypes = [cfgp, cp, vp, i64, vp, i64, i64, vp, vp, i64, i64, vp, vp, sz, vp]
        for n in EXPORTED:
            getattr(L, n).restype = ctypes.c_int
        _READY = True
    return L


@dataclasses.dataclass(frozen=True)
class AttnConfig:
    """Geometry and constants of one attention layer; every field explicit (no defaults)."""
    n_heads: int
    n_kv_heads: int
    head_dim: int        # 64, 128 or 256
    page_size: int       # 16, 32, 64, 128 or 256
    rotary_dim: int      # 0 or a multiple of 16 up to head_dim
    rope_style: int      # ROPE_HALF or ROPE_INTERLEAVED
    norm_eps: float
    scale: float         # multiplies q . k
    window: int          # latest keys a query sees; 0 = all
    n_sinks: int         # first keys that stay visible beside a window

    def c(self) -> moe_attn_config:
        return moe_attn_config(**dataclasses.asdict(self))


@dataclasses.dataclass
class KVCache:
    """Pages of keys and values in the library's layout (see include/moe_attn.h)."""
    k: torch.Tensor      # [n_pages, n_kv_heads, head_dim / 8, page_size, 8] bf16
    v: torch.Tensor      # [n_pages, n_kv_heads, page_size / 8, head_dim, 8] bf16

    def check(self, cfg: AttnConfig) -> None:
        n = self.k.shape[0] if isinstance(self.k, torch.Tensor) and self.k.dim() else 0
        k, v = cache_shapes(cfg, n)
        _check_tensor(self.k, "cache.k", k, torch.bfloat16)
        _check_tensor(self.v, "cache.v", v, torch.bfloat16)

    def c(self) -> moe_attn_cache:
        return moe_attn_cache(_ptr(self.k), _ptr(self.v), self.k.shape[0])


def cache_shapes(cfg: AttnConfig, n_pages: int):
    """Shapes of KVCache.k and KVCache.v."""
    return ((n_pages, cfg.n_kv_heads, cfg.head_dim // 8, cfg.page_size, 8),
            (n_pages, cfg.n_kv_heads, cfg.page_size // 8, cfg.head_dim, 8))


def new_cache(cfg: AttnConfig, n_pages: int, device="cuda") -> KVCache:
    """An empty cache (allocated by torch; contents need no initialisation)."""
    k, v = cache_shapes(cfg, n_pages)
    return KVCache(torch.empty(k, dtype=torch.bfloat16, device=device),
                   torch.empty(v, dtype=torch.bfloat16, device=device))


def moe_attn_workspace_size(cfg: AttnConfig, T: int, B: int, max_q: int, max_len: int, prefill: bool) -> int:
    """Bytes for T new tokens of B sequences, at most max_q of one, each of at most max_len tokens in all; of exactly
    these sizes, since smaller ones may need more (moe_attn_workspace_bound)."""
    return _size("moe_attn_workspace_size", cfg, T, B, max_q, max_len, prefill)


def moe_attn_workspace_bound(cfg: AttnConfig, T: int, B: int, max_q: int, max_len: int, prefill: bool) -> int:
    """Bytes for every call of these sizes or smaller ones: for a workspace that is allocated once."""
    return _size("moe_attn_workspace_bound", cfg, T, B, max_q, max_len, prefill)


def _size(name, cfg, T, B, max_q, max_len, prefill) -> int:
    n = ctypes.c_size_t(0)
    _check(getattr(_lib(), name)(ctypes.byref(cfg.c()), int(T), int(B), int(max_q), int(max_len),
                                 int(bool(prefill)), ctypes.byref(n)), name)
    return n.value


def workspace(cfg: AttnConfig, T: int, B: int, max_q: int, max_len: int, prefill: bool,
              device="cuda") -> torch.Tensor:
    """A workspace tensor of the size the library asks for (allocated by torch)."""
    return torch.empty(max(1, moe_attn_workspace_size(cfg, T, B, max_q, max_len, prefill)), dtype=torch.uint8,
                       device=device)


def _one_device(**tensors) -> None:
    here = torch.cuda.current_device()
    for name, t in tensors.items():
        if t is not None and t.device.index != here:
            raise ValueError(f"{name} is on {t.device}, the current device is cuda:{here}")


def _ws_on_stream(cfg, T, B, max_q, max_len, prefill, device, stream) -> torch.Tensor:
    """A workspace that torch's allocator ties to the stream that the call runs on."""
    handle = _stream(stream)
    if handle == torch.cuda.current_stream().cuda_stream:
        return workspace(cfg, T, B, max_q, max_len, prefill, device)
    with torch.cuda.stream(torch.cuda.ExternalStream(handle)):
        return workspace(cfg, T, B, max_q, max_len, prefill, device)


def _callable(name: str, args, stream, device: int, keep, ws: Optional[torch.Tensor] = None):
    """args: all but the stream; ws: the workspace if it is the callable's own, allocated on the stream current now."""
    fn = getattr(_lib(), name)
    # looked up and converted once: a call of the smallest sizes is bound by what it does on the host
    handle_of, device_now = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
    args = tuple(to(a) if a is None or isinstance(a, int) else a for to, a in zip(fn.argtypes, args))
    fixed = None if stream is None else _stream(stream)
    home = handle_of(device)

    def call():
        if device_now() != device:
            raise ValueError(f"{name}: bound on cuda:{device}, the current device is cuda:{device_now()}")
        handle = handle_of(device) if fixed is None else fixed
        if ws is not None and fixed is None and handle != home:
            ws.record_stream(torch.cuda.current_stream(device))      # not handed out again before this call ends
        st = fn(*args, handle)
        if st:
            _check(st, name)
    call.keep = keep         # the buffers outlive the callable
    return call


def bind_prepare(cfg: AttnConfig, cache: KVCache, qkv: torch.Tensor, q_norm_w: Optional[torch.Tensor],
                 k_norm_w: Optional[torch.Tensor], cos_sin: Optional[torch.Tensor],
                 positions: Optional[torch.Tensor], slots: torch.Tensor, q_out: torch.Tensor, stream=None):
    """moe_attn_prepare on these buffers, as a callable (its stream: see the module)."""
    D, width = cfg.head_dim, (cfg.n_heads + 2 * cfg.n_kv_heads) * cfg.head_dim
    if not isinstance(qkv, torch.Tensor) or qkv.dim() != 2:
        raise ValueError("qkv must be a [T, (n_heads + 2 n_kv_heads) * head_dim] tensor")
    T = qkv.shape[0]
    if qkv.dtype != torch.bfloat16:
        raise TypeError(f"qkv: dtype {qkv.dtype}, expected {torch.bfloat16}")
    if qkv.device.type != "cuda":
        raise ValueError("qkv must be a device (HIP) tensor")
    if qkv.shape[1] != width or (T and qkv.stride(1) != 1):
        raise ValueError(f"qkv: shape {tuple(qkv.shape)} with strides {qkv.stride()}, expected rows of {width} values")
    stride = qkv.stride(0) if T > 1 else width
    cache.check(cfg)
    for n, t in (("q_norm_w", q_norm_w), ("k_norm_w", k_norm_w)):
        if t is not None:
            _check_tensor(t, n, (D,), torch.float32)
    P = 0
    if cos_sin is not None:
        P = cos_sin.shape[0] if cos_sin.dim() == 2 else -1
        _check_tensor(cos_sin, "cos_sin", (P, cfg.rotary_dim), torch.float32)
    if positions is not None:
        _check_tensor(positions, "positions", (T,), torch.int32)
    _check_tensor(slots, "slots", (T,), torch.int64)
    _check_tensor(q_out, "q_out", (T, cfg.n_heads, D), torch.bfloat16)
    _one_device(qkv=qkv, k=cache.k, v=cache.v, q_norm_w=q_norm_w, k_norm_w=k_norm_w, cos_sin=cos_sin,
                positions=positions, slots=slots, q_out=q_out)
    c, cc = cfg.c(), cache.c()
    args = (ctypes.byref(c), ctypes.byref(cc), qkv.data_ptr(), stride, T, _ptr(q_norm_w), _ptr(k_norm_w),
            _ptr(cos_sin), P, _ptr(positions), slots.data_ptr(), q_out.data_ptr())
    return _callable("moe_attn_prepare", args, stream, qkv.device.index,
                     (c, cc, cache, qkv, q_norm_w, k_norm_w, cos_sin, positions, slots, q_out))


def bind_decode(cfg: AttnConfig, cache: KVCache, q: torch.Tensor, seq_lens: torch.Tensor, page_table: torch.Tensor,
                max_len: int, out: torch.Tensor, ws: Optional[torch.Tensor] = None, stream=None):
    """moe_attn_decode on these buffers, as a callable (its stream: see the module)."""
    B, n = (q.shape[0], q.shape[1]) if q.dim() == 4 else (-1, -1)
    _check_tensor(q, "q", (B, n, cfg.n_heads, cfg.head_dim), torch.bfloat16)
    _check_tensor(out, "out", tuple(q.shape), torch.bfloat16)
    pages = _check_sequences(cfg, cache, B, seq_lens, page_table)
    own = ws is None
    if own:
        ws = _ws_on_stream(cfg, B * n, B, n, max_len, False, q.device, stream)
    _check_tensor(ws, "workspace", None, torch.uint8)
    _one_device(q=q, out=out, k=cache.k, v=cache.v, seq_lens=seq_lens, page_table=page_table, workspace=ws)
    c, cc = cfg.c(), cache.c()
    args = (ctypes.byref(c), ctypes.byref(cc), q.data_ptr(), B, n, seq_lens.data_ptr(), page_table.data_ptr(),
            pages, int(max_len), out.data_ptr(), ws.data_ptr(), ws.numel())
    return _callable("moe_attn_decode", args, stream, q.device.index, (c, cc, cache, q, seq_lens, page_table, out, ws),
                     ws if own else None)


def bind_prefill(cfg: AttnConfig, cache: KVCache, q: torch.Tensor, cu_q: torch.Tensor, max_q: int,
                 seq_lens: torch.Tensor, page_table: torch.Tensor, max_len: int, out: torch.Tensor,
                 ws: Optional[torch.Tensor] = None, stream=None):
    """moe_attn_prefill on these buffers, as a callable (its stream: see the module)."""
    T = q.shape[0] if q.dim() == 3 else -1
    _check_tensor(q, "q", (T, cfg.n_heads, cfg.head_dim), torch.bfloat16)
    _check_tensor(out, "out", tuple(q.shape), torch.bfloat16)
    B = cu_q.shape[0] - 1 if cu_q.dim() == 1 else -1
    if B < 0:
        raise ValueError("cu_q must be a [B + 1] tensor")
    _check_tensor(cu_q, "cu_q", (B + 1,), torch.int32)
    pages = _check_sequences(cfg, cache, B, seq_lens, page_table)
    own = ws is None
    if own:
        ws = _ws_on_stream(cfg, T, B, max_q, max_len, True, q.device, stream)
    _check_tensor(ws, "workspace", None, torch.uint8)
    _one_device(q=q, out=out, k=cache.k, v=cache.v, cu_q=cu_q, seq_lens=seq_lens, page_table=page_table,
                workspace=ws)
    c, cc = cfg.c(), cache.c()
    args = (ctypes.byref(c), ctypes.byref(cc), q.data_ptr(), T, cu_q.data_ptr(), B, int(max_q), seq_lens.data_ptr(),
            page_table.data_ptr(), pages, int(max_len), out.data_ptr(), ws.data_ptr(), ws.numel())
    return _callable("moe_attn_prefill", args, stream, q.device.index,
                     (c, cc, cache, q, cu_q, seq_lens, page_table, out, ws), ws if own else None)


def _check_sequences(cfg, cache, B, seq_lens, page_table) -> int:
    cache.check(cfg)
    _check_tensor(seq_lens, "seq_lens", (B,), torch.int32)
    pages = page_table.shape[1] if page_table.dim() == 2 else -1
    _check_tensor(page_table, "page_table", (B, pages), torch.int32)
    return pages


def moe_attn_prepare(cfg: AttnConfig, cache: KVCache, qkv: torch.Tensor, q_norm_w, k_norm_w, cos_sin, positions,
                     slots: torch.Tensor, q_out: torch.Tensor, stream=None) -> None:
    """Norm, rotate and append the tokens of qkv [T, (n_heads + 2 n_kv_heads) * head_dim]: queries to q_out
    [T, n_heads, head_dim], keys and values into the cache at `slots` (page * page_size + place)."""
    bind_prepare(cfg, cache, qkv, q_norm_w, k_norm_w, cos_sin, positions, slots, q_out, stream)()


def moe_attn_decode(cfg: AttnConfig, cache: KVCache, q: torch.Tensor, seq_lens: torch.Tensor,
                    page_table: torch.Tensor, max_len: int, out: torch.Tensor, ws: Optional[torch.Tensor] = None,
                    stream=None) -> None:
    """Attention of the last q.shape[1] tokens of every sequence over the cache: q, out [B, n_q, n_heads, head_dim]."""
    bind_decode(cfg, cache, q, seq_lens, page_table, max_len, out, ws, stream)()


def moe_attn_prefill(cfg: AttnConfig, cache: KVCache, q: torch.Tensor, cu_q: torch.Tensor, max_q: int,
                     seq_lens: torch.Tensor, page_table: torch.Tensor, max_len: int, out: torch.Tensor,
                     ws: Optional[torch.Tensor] = None, stream=None) -> None:
    """Causal attention of prompts (tokens cu_q[b] .. cu_q[b+1]-1 of q, the last of seq_lens[b]) over the cache."""
    bind_prefill(cfg, cache, q, cu_q, max_q, seq_lens, page_table, max_len, out, ws, stream)()
