"""GB300-native block-sparse ("splash") attention: Python binding of libbsa.so.

The functions here have the names of the C entry points in ``include/bsa.h``
(without the ``bsa_`` prefix) and do argument marshalling only: torch
supplies device memory and the current stream, and every step of the path
runs in the library's CUDA kernels.  When the library is missing every call
raises; nothing falls back to another implementation.

    info = mask_compile("causal", S, S)                     # MaskInfo (fwd orientation)
    o, lse = fwd(q, k, v, info)                              # bf16 O, fp32 logsumexp
    dkv = mask_compile("causal", S, S, orientation="dkv")
    dq, dk, dv = bwd(q, k, v, o, lse, do, info, dkv)

After a prompt, token by token over a cache held in 4 bits:

    cache = KV4Cache.empty(B, Hkv, capacity, D)
    kv4_append(cache, k, v, start, weights=key_weights(q, k, lse, dkv))
    kv4_append(cache, k1, v1, lens, positions=seen)          # each new token: slot lens[b], position seen[b]
    lens, seen = lens + 1, seen + 1
    o1, lse1 = kv4_fwd(q1, cache, lens, accumulate=True)
    lens, index = kv4_evict(cache, lens, keep, recent=recent, seen=seen)

Or over a cache in pages, which sequences take and give back as they grow and end, attending to all of it
or to the pages that promise the largest scores:

    cache = PagedCache.empty(pages, Hkv, page, D)
    table, free, used = paged_table(pages, B, M)
    lens, used, slots = paged_resize(table, free, used, lens, new_lens, page, T)
    paged_append(cache, k, v, slots)                         # k, v [B,Hkv,T,D]
    o, lse = paged_fwd(q, cache, table, lens)
    o, lse = paged_fwd(q, cache, table, lens, select=paged_select(q, cache, table, lens, keep))
"""
from __future__ import annotations

import contextlib
import ctypes as C
import math
from dataclasses import dataclass
from typing import Optional

import torch

from . import _abi
from ._abi import BsaError, check

__all__ = ["mask_compile", "MaskInfo", "fwd", "fwd_partial", "fwd_merge", "bwd", "bwd_noalloc", "bwd_rowsum",
           "bwd_dkv", "bwd_dq", "key_weights", "KV4Cache", "kv4_append", "kv4_fwd", "kv4_evict",
           "PagedCache", "paged_table", "paged_resize", "paged_append", "paged_select", "paged_fwd",
           "get_device_error", "set_wait_limit_ns", "debug_wait_timeout", "debug_selfcheck", "version", "BsaError",
           "library_path"]

_KINDS = {"dense": _abi.MASK_DENSE, "causal": _abi.MASK_CAUSAL, "local": _abi.MASK_LOCAL,
          "chunked": _abi.MASK_CHUNKED_CAUSAL, "full": _abi.MASK_FULL}
_ORIENT = {"fwd": _abi.ORIENT_FWD, "dkv": _abi.ORIENT_DKV}
_IDX_DTYPES = {1: torch.int8, 2: torch.int16, 4: torch.int32}


def library_path() -> str:
    return _abi.LIB_PATH


def version() -> str:
    return _abi.lib().bsa_version().decode()


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


class _DevArray:
    """A borrowed device array (no copy) usable with torch.as_tensor."""

    def __init__(self, ptr: int, shape, typestr: str):
        self.__cuda_array_interface__ = {"shape": tuple(shape), "typestr": typestr,
                                         "data": (ptr, False), "version": 3, "strides": None}


def _view(ptr: int, shape, dtype: torch.dtype) -> torch.Tensor:
    n = 1
    for s in shape:
        n *= s
    if n == 0 or not ptr:
        return torch.empty(shape, dtype=dtype, device="cuda")
    typestr = {torch.int8: "|i1", torch.uint8: "|u1", torch.int16: "<i2", torch.int32: "<i4"}[dtype]
    return torch.as_tensor(_DevArray(ptr, shape, typestr), device="cuda")


class MaskInfo:
    """A compiled mask owned by the library (freed when this object dies)."""

    def __init__(self, handle: int):
        self._h = C.c_void_p(handle)

    @property
    def handle(self) -> C.c_void_p:
        if not self._h:
            raise RuntimeError("MaskInfo was destroyed")
        return self._h

    def desc(self) -> _abi.MaskInfoDesc:
        d = _abi.MaskInfoDesc()
        check(_abi.lib().bsa_mask_info_view(self.handle, C.byref(d)), "bsa_mask_info_view")
        return d

    def arrays(self) -> dict:
        """Borrowed device views of the MaskInfo arrays (valid while self lives)."""
        d = self.desc()
        shp = (d.heads, d.rows, d.width)
        out = {
            "block_mask": _view(d.block_mask, shp, torch.int8),
            "data_next": _view(d.data_next, shp, _IDX_DTYPES[d.data_next_bytes]),
            "mask_next": None if not d.mask_next else _view(d.mask_next, shp, _IDX_DTYPES[d.mask_next_bytes]),
            "partial_mask_blocks": None if not d.partial_mask_blocks else
            _view(d.partial_mask_blocks, (d.num_partial, 128, 128), torch.uint8),
            "q_sequence": _view(d.q_sequence, (d.q_len,), torch.int32),
            "row_len": _view(d.row_len, (d.heads * d.rows,), torch.int32),
            "row_order": _view(d.row_order, (d.heads * d.rows,), torch.int32),
        }
        return out

    def to_host(self) -> dict:
        """Copies of every array plus the counts, as numpy (for inspection and tests)."""
        torch.cuda.synchronize()
        d = self.desc()
        out = {k: (None if v is None else v.cpu().numpy()) for k, v in self.arrays().items()}
        out.update(width=d.width, cols=d.cols, num_partial=d.num_partial, n_empty=d.n_empty,
                   n_partial=d.n_partial, n_full=d.n_full, heads=d.heads, rows=d.rows)
        return out

    def destroy(self) -> None:
        if self._h:
            _abi.lib().bsa_mask_info_destroy(self._h)
            self._h = C.c_void_p(None)

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass


def mask_compile(kind: str, q_len: int, kv_len: int, *, mask_heads: int = 1, local_left: Optional[int] = None,
                 local_right: Optional[int] = None, chunk: int = 0, dense: Optional[torch.Tensor] = None,
                 shrink: bool = True, orientation: str = "fwd", stream=None) -> MaskInfo:
    """bsa_mask_compile.  ``dense`` is a CUDA uint8 tensor [mask_heads, q_len, kv_len] (or 2-D)."""
    spec = _abi.MaskSpec()
    spec.kind = _KINDS[kind]
    spec.q_len, spec.kv_len = q_len, kv_len
    spec.mask_heads = mask_heads
    spec.local_left = -1 if local_left is None else local_left
    spec.local_right = -1 if local_right is None else local_right
    spec.chunk = chunk
    if dense is not None:
        if dense.dtype != torch.uint8 or not dense.is_cuda or not dense.is_contiguous():
            raise ValueError("dense mask must be a contiguous CUDA uint8 tensor")
        spec.mask_heads = 1 if dense.dim() == 2 else dense.shape[0]
        spec.dense = dense.data_ptr()
    opts = _abi.MaskOpts(128, 128, 1 if shrink else 0, _ORIENT[orientation])
    out = C.c_void_p()
    check(_abi.lib().bsa_mask_compile(C.byref(spec), C.byref(opts), _stream(stream), C.byref(out)),
          "bsa_mask_compile")
    return MaskInfo(out.value)


def _check_bf16(name: str, t: torch.Tensor) -> None:
    if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA bfloat16 tensor")


def _sink_fields(sinks: Optional[torch.Tensor], Hkv: int):
    """(pointer, count, per-kv-head flag) of an fp32 CUDA sinks tensor [Hkv, n] or [n]."""
    if sinks is None:
        return None, 0, 0
    if sinks.dtype != torch.float32 or not sinks.is_cuda or not sinks.is_contiguous():
        raise ValueError("sinks must be a contiguous CUDA float32 tensor")
    if sinks.dim() == 2:
        if sinks.shape[0] != Hkv:
            raise ValueError("a 2-D sinks tensor must be [Hkv, num_sinks]")
        return _ptr(sinks), sinks.shape[1], 1
    if sinks.dim() != 1:
        raise ValueError("sinks must be [Hkv, num_sinks] or [num_sinks]")
    return _ptr(sinks), sinks.shape[0], 0


def fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, info: MaskInfo, *, o: Optional[torch.Tensor] = None,
        lse: Optional[torch.Tensor] = None, softmax_scale: Optional[float] = None,
        logits_soft_cap: Optional[float] = None, sinks: Optional[torch.Tensor] = None, stream=None):
    """bsa_fwd.  q [B,Hq,S,D], k/v [B,Hkv,Skv,D] bf16 -> (o bf16 [B,Hq,S,D], lse fp32 [B,Hq,S]).
    Optional soft cap c (scores -> c*tanh(s/c)) and sinks (fp32 [Hkv, n] or [n])."""
    for n, t in (("q", q), ("k", k), ("v", v)):
        _check_bf16(n, t)
    B, Hq, S, D = q.shape
    Hkv, Skv = k.shape[1], k.shape[2]
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, Hq, S), dtype=torch.float32, device=q.device)
    sp, sn, skv = _sink_fields(sinks, Hkv)
    a = _abi.FwdArgs(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, Hq, Hkv, D, S, Skv,
                     math.nan if softmax_scale is None else softmax_scale, logits_soft_cap or 0.0, sp, sn, skv)
    check(_abi.lib().bsa_fwd(C.byref(a), info.handle, _stream(stream)), "bsa_fwd")
    return o, lse


def fwd_partial(q: torch.Tensor, k_shard: torch.Tensor, v_shard: torch.Tensor, info: MaskInfo, kv_offset: int, *,
                softmax_scale: Optional[float] = None, logits_soft_cap: Optional[float] = None, stream=None):
    """bsa_fwd_partial: attention of q over one key shard (k_shard / v_shard hold keys
    kv_offset .. kv_offset + Skv_shard - 1 of the MaskInfo's key axis).
    -> (o_acc fp32 [B,Hq,S,D], m fp32 [B,Hq,S], l fp32 [B,Hq,S])."""
    for n, t in (("q", q), ("k", k_shard), ("v", v_shard)):
        _check_bf16(n, t)
    B, Hq, S, D = q.shape
    Hkv, Skv = k_shard.shape[1], k_shard.shape[2]
    o_acc = torch.empty((B, Hq, S, D), dtype=torch.float32, device=q.device)
    m = torch.empty((B, Hq, S), dtype=torch.float32, device=q.device)
    l = torch.empty((B, Hq, S), dtype=torch.float32, device=q.device)
    a = _abi.FwdPartialArgs(_ptr(q), _ptr(k_shard), _ptr(v_shard), _ptr(o_acc), _ptr(m), _ptr(l), B, Hq, Hkv, D, S,
                            Skv, kv_offset, math.nan if softmax_scale is None else softmax_scale,
                            logits_soft_cap or 0.0)
    check(_abi.lib().bsa_fwd_partial(C.byref(a), info.handle, _stream(stream)), "bsa_fwd_partial")
    return o_acc, m, l


def fwd_merge(o_acc: torch.Tensor, m: torch.Tensor, l: torch.Tensor, stream=None):
    """bsa_fwd_merge over stacked shards: o_acc [n, B,Hq,S,D], m / l [n, B,Hq,S] fp32
    -> (o bf16 [B,Hq,S,D], lse fp32 [B,Hq,S])."""
    for n_, t in (("o_acc", o_acc), ("m", m), ("l", l)):
        if t.dtype != torch.float32 or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{n_} must be a contiguous CUDA float32 tensor")
    n = o_acc.shape[0]
    D = o_acc.shape[-1]
    rows = o_acc[0].numel() // D
    o = torch.empty(o_acc.shape[1:], dtype=torch.bfloat16, device=o_acc.device)
    lse = torch.empty(m.shape[1:], dtype=torch.float32, device=o_acc.device)
    a = _abi.MergeArgs(n, _ptr(o_acc), _ptr(m), _ptr(l), _ptr(o), _ptr(lse), rows, D)
    check(_abi.lib().bsa_fwd_merge(C.byref(a), _stream(stream)), "bsa_fwd_merge")
    return o, lse


@dataclass
class _BwdBufs:
    args: _abi.BwdArgs
    dq: torch.Tensor
    dk: torch.Tensor
    dv: torch.Tensor
    dsum: torch.Tensor
    dsinks: Optional[torch.Tensor] = None


def _bwd_args(q, k, v, o, lse, do, dq, dk, dv, dsum, softmax_scale, grad_fp32, logits_soft_cap=None,
              sinks=None) -> _BwdBufs:
    for n, t in (("q", q), ("k", k), ("v", v), ("o", o), ("do", do)):
        _check_bf16(n, t)
    B, Hq, S, D = q.shape
    Hkv, Skv = k.shape[1], k.shape[2]
    gdt = torch.float32 if grad_fp32 else torch.bfloat16
    dq = torch.empty(q.shape, dtype=gdt, device=q.device) if dq is None else dq
    dk = torch.empty(k.shape, dtype=gdt, device=q.device) if dk is None else dk
    dv = torch.empty(v.shape, dtype=gdt, device=q.device) if dv is None else dv
    dsum = torch.empty((B, Hq, S), dtype=torch.float32, device=q.device) if dsum is None else dsum
    sp, sn, skv = _sink_fields(sinks, Hkv)
    dsinks = None if sinks is None else torch.empty_like(sinks)
    a = _abi.BwdArgs(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(do), _ptr(dq), _ptr(dk), _ptr(dv),
                     _ptr(dsum), B, Hq, Hkv, D, S, Skv, math.nan if softmax_scale is None else softmax_scale,
                     1 if grad_fp32 else 0, logits_soft_cap or 0.0, sp, _ptr(dsinks), sn, skv)
    return _BwdBufs(a, dq, dk, dv, dsum, dsinks)


def bwd(q, k, v, o, lse, do, fwd_info: MaskInfo, dkv_info: MaskInfo, *, dq=None, dk=None, dv=None, dsum=None,
        softmax_scale=None, grad_fp32: bool = False, logits_soft_cap=None, sinks=None, stream=None):
    """bsa_bwd: rowsum, then dK/dV, then dQ.  Returns (dq, dk, dv), plus dsinks when sinks are given."""
    b = _bwd_args(q, k, v, o, lse, do, dq, dk, dv, dsum, softmax_scale, grad_fp32, logits_soft_cap, sinks)
    check(_abi.lib().bsa_bwd(C.byref(b.args), fwd_info.handle, dkv_info.handle, _stream(stream)), "bsa_bwd")
    return (b.dq, b.dk, b.dv) if sinks is None else (b.dq, b.dk, b.dv, b.dsinks)


def bwd_noalloc(q, k, v, o, lse, do, fwd_info: MaskInfo, dkv_info: MaskInfo, *, dq, dk, dv, softmax_scale=None,
                grad_fp32: bool = False, logits_soft_cap=None, sinks=None, dsinks=None, stream=None):
    """bsa_bwd_noalloc: the backward pass with no device allocation inside the
    library (its rowsum scratch is a fixed 4 MiB device array); the caller
    supplies the gradient buffers (and ``dsinks``, the sinks' shape, when the
    sinks' gradient is wanted)."""
    for n, t in (("q", q), ("k", k), ("v", v), ("o", o), ("do", do)):
        _check_bf16(n, t)
    B, Hq, S, D = q.shape
    Hkv, Skv = k.shape[1], k.shape[2]
    sp, sn, skv = _sink_fields(sinks, Hkv)
    a = _abi.BwdArgs(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(do), _ptr(dq), _ptr(dk), _ptr(dv),
                     None, B, Hq, Hkv, D, S, Skv, math.nan if softmax_scale is None else softmax_scale,
                     1 if grad_fp32 else 0, logits_soft_cap or 0.0, sp, _ptr(dsinks), sn, skv)
    check(_abi.lib().bsa_bwd_noalloc(C.byref(a), fwd_info.handle, dkv_info.handle, _stream(stream)),
          "bsa_bwd_noalloc")
    return (dq, dk, dv) if dsinks is None else (dq, dk, dv, dsinks)


def bwd_rowsum(o, do, *, dsum=None, stream=None) -> torch.Tensor:
    """bsa_bwd_rowsum: dsum[b,h,s] = sum_d dO*O (fp32)."""
    _check_bf16("o", o)
    _check_bf16("do", do)
    B, H, S, D = o.shape
    dsum = torch.empty((B, H, S), dtype=torch.float32, device=o.device) if dsum is None else dsum
    a = _abi.BwdArgs(_ptr(o), _ptr(o), _ptr(o), _ptr(o), _ptr(dsum), _ptr(do), _ptr(o), _ptr(o), _ptr(o),
                     _ptr(dsum), B, H, H, D, S, S, math.nan, 0)
    check(_abi.lib().bsa_bwd_rowsum(C.byref(a), _stream(stream)), "bsa_bwd_rowsum")
    return dsum


def bwd_dkv(q, k, v, o, lse, do, dsum, dkv_info: MaskInfo, *, dk=None, dv=None, softmax_scale=None,
            grad_fp32=False, stream=None):
    b = _bwd_args(q, k, v, o, lse, do, None, dk, dv, dsum, softmax_scale, grad_fp32)
    check(_abi.lib().bsa_bwd_dkv(C.byref(b.args), dkv_info.handle, _stream(stream)), "bsa_bwd_dkv")
    return b.dk, b.dv


def bwd_dq(q, k, v, o, lse, do, dsum, fwd_info: MaskInfo, *, dq=None, softmax_scale=None, grad_fp32=False,
           stream=None):
    b = _bwd_args(q, k, v, o, lse, do, dq, None, None, dsum, softmax_scale, grad_fp32)
    check(_abi.lib().bsa_bwd_dq(C.byref(b.args), fwd_info.handle, _stream(stream)), "bsa_bwd_dq")
    return b.dq


_INLINE = contextlib.nullcontext()


@contextlib.contextmanager
def _elsewhere(device, stream):
    with torch.cuda.device(device):
        if stream is None:
            yield
        else:
            with torch.cuda.stream(stream):
                yield


_raw_stream, _current_device = (getattr(torch._C, "_cuda_" + x, None) for x in ("getCurrentRawStream", "getDevice"))


def _place(device: torch.device, index: int, stream):
    """(context, stream handle) of a call on tensors of `device`: inside the
    context the device and the stream are current, so that what the call
    allocates belongs to the stream it is used on."""
    if stream is None:
        handle = _raw_stream(index)
        return (_INLINE if index == _current_device() else _elsewhere(device, None)), handle
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=device) if int(stream) else torch.cuda.default_stream(device)
    if stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, the tensors are on {device}")
    return _elsewhere(device, stream), stream.cuda_stream


def _need(name: str, t: torch.Tensor, dtype: torch.dtype, index: int, shape) -> int:
    """The address of a contiguous CUDA tensor of a type and shape on a device."""
    if t.dtype is not dtype or t.get_device() != index or t.shape != shape or not t.is_contiguous():
        if t.dtype != dtype or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA {str(dtype)[6:]} tensor")
        if t.get_device() != index:
            raise ValueError(f"{name} is on {t.device}, the call's other tensors are on cuda:{index}")
        raise ValueError(f"{name} must be {list(shape)}, not {list(t.shape)}")
    return t.data_ptr()


def _rows(name: str, t: torch.Tensor, index: int):
    """Strides (batch, head, token) of a 4-D bf16 CUDA tensor whose last axis is contiguous."""
    if t.dtype is not torch.bfloat16 or t.get_device() < 0 or t.dim() != 4:
        raise ValueError(f"{name} must be a 4-D CUDA bfloat16 tensor")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, the call's other tensors are on cuda:{index}")
    sb, sh, st, sd = t.stride()
    if (sb | sh | st) & 7 or sd != 1 or t.data_ptr() & 15:
        # (the stride of an axis of length 1 says nothing)
        sb, sh, st, sd = (1 if i == 3 and n == 1 else 0 if n == 1 else s
                          for i, (n, s) in enumerate(zip(t.shape, (sb, sh, st, sd))))
        if (sb | sh | st) & 7 or sd != 1 or t.data_ptr() & 15:
            raise ValueError(f"{name} needs a contiguous last axis, other strides that are multiples of 8 and "
                             "16-byte alignment")
    return sb, sh, st


def _lens(name: str, t: Optional[torch.Tensor], B: int, index: int) -> int:
    return 0 if t is None else _need(name, t, torch.int32, index, (B,))


# a workspace for one call, on the stream that the call uses (an allocation by way of a tensor, which serves where torch
# does not offer these, costs three times as much beside a launch)
_raw_alloc, _raw_free = (getattr(torch._C, "_cuda_cudaCachingAllocator_raw_" + x, None) for x in ("alloc", "delete"))


def _workspace(need: int, device) -> Optional[torch.Tensor]:
    return torch.empty(need, dtype=torch.uint8, device=device) if need else None


# workspace sizes of calls made before, by the shape of the call (host arithmetic, nothing of the data)
_workspace_sizes: dict = {}


def _workspace_size(entry: str, key, args) -> int:
    key = (entry, key)
    need = _workspace_sizes.get(key)
    if need is None:
        args = args if isinstance(args, bytes) else args()
        n = C.c_size_t(0)
        check(getattr(_abi.lib(), entry + "_workspace")(args, C.byref(n)), entry)
        if len(_workspace_sizes) > 4096:
            _workspace_sizes.clear()
        need = _workspace_sizes[key] = n.value
    return need


def key_weights(q: torch.Tensor, k: torch.Tensor, lse: torch.Tensor, dkv_info: MaskInfo, *,
                q_lens: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                softmax_scale: Optional[float] = None, logits_soft_cap: Optional[float] = None, stream=None) -> torch.Tensor:
    """bsa_key_weights: the attention weight each key of a prompt has received.
    q [B,Hq,S,D], k [B,Hkv,Skv,D] bf16, lse fp32 [B,Hq,S] from ``fwd``, the mask's "dkv" MaskInfo
    -> fp32 [B,Hkv,Skv].  ``q_lens`` (int32 [B]): queries past it are padding and not counted."""
    for n, t in (("q", q), ("k", k)):
        _check_bf16(n, t)
        if t.dim() != 4:
            raise ValueError(f"{n} must be 4-D")
    B, Hq, S, D = q.shape
    Hkv, Skv = k.shape[1], k.shape[2]
    if k.shape != (B, Hkv, Skv, D) or k.device != q.device:
        raise ValueError("k must be [B, Hkv, Skv, D] on q's device")
    index = q.get_device()
    a = _abi.KeyWeightsArgs(_ptr(q), _ptr(k), _need("lse", lse, torch.float32, index, (B, Hq, S)),
                            _lens("q_lens", q_lens, B, index) or None, None, None, 0, B, Hq, Hkv,
                            D, S, Skv, math.nan if softmax_scale is None else softmax_scale, logits_soft_cap or 0.0)
    ctx, handle = _place(q.device, index, stream)
    with ctx:
        if out is None:
            out = torch.empty((B, Hkv, Skv), dtype=torch.float32, device=q.device)
        a.weights = _need("out", out, torch.float32, index, (B, Hkv, Skv))
        need = C.c_size_t(0)
        check(_abi.lib().bsa_key_weights_workspace(C.byref(a), dkv_info.handle, C.byref(need)), "bsa_key_weights")
        ws = _workspace(need.value, q.device)
        a.workspace, a.workspace_bytes = _ptr(ws), need.value
        check(_abi.lib().bsa_key_weights(C.byref(a), dkv_info.handle, handle), "bsa_key_weights")
    return out


class KV4Cache:
    """A key/value cache held in 4 bits (bsa_kv4_cache): the buffers, which the caller owns.

    k_codes, v_codes: uint8 [B, Hkv, capacity, D/2]; k_scales, v_scales: bf16 [B, Hkv, capacity, D/32];
    weights: fp32 [B, Hkv, capacity] accumulated attention weights, or None; positions: int32
    [B, Hkv, capacity] the tokens' positions, or None.  capacity is a multiple of 16."""

    __slots__ = ("k_codes", "k_scales", "v_codes", "v_scales", "weights", "positions", "B", "Hkv", "D", "capacity",
                 "device", "index", "_c")

    def __init__(self, k_codes: torch.Tensor, k_scales: torch.Tensor, v_codes: torch.Tensor, v_scales: torch.Tensor,
                 weights: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None):
        if k_codes.dim() != 4:
            raise ValueError("k_codes must be [B, Hkv, capacity, D/2]")
        B, H, n, half = shape = k_codes.shape
        index = k_codes.get_device()
        if index < 0:
            raise ValueError("k_codes must be a contiguous CUDA uint8 tensor")
        scales, slots = (B, H, n, half // 16), (B, H, n)
        self._c = _abi.KV4_CACHE.pack(
            _need("k_codes", k_codes, torch.uint8, index, shape), _need("k_scales", k_scales, torch.bfloat16, index, scales),
            _need("v_codes", v_codes, torch.uint8, index, shape), _need("v_scales", v_scales, torch.bfloat16, index, scales),
            0 if weights is None else _need("weights", weights, torch.float32, index, slots),
            0 if positions is None else _need("positions", positions, torch.int32, index, slots), B, H, 2 * half, n)
        self.k_codes, self.k_scales, self.v_codes, self.v_scales = k_codes, k_scales, v_codes, v_scales
        self.weights, self.positions = weights, positions
        self.B, self.Hkv, self.D, self.capacity, self.device, self.index = B, H, 2 * half, n, k_codes.device, index

    @classmethod
    def empty(cls, B: int, Hkv: int, capacity: int, D: int, device="cuda", weights: bool = True) -> "KV4Cache":
        """A cache without tokens; without ``weights`` it has neither weights nor positions."""
        def new(shape, dtype):
            return torch.zeros(shape, dtype=dtype, device=device)
        codes, scales = (B, Hkv, capacity, D // 2), (B, Hkv, capacity, D // 32)
        return cls(new(codes, torch.uint8), new(scales, torch.bfloat16), new(codes, torch.uint8),
                   new(scales, torch.bfloat16), new((B, Hkv, capacity), torch.float32) if weights else None,
                   new((B, Hkv, capacity), torch.int32) if weights else None)


def kv4_append(cache: KV4Cache, k: torch.Tensor, v: torch.Tensor, start: torch.Tensor, *,
               n_new: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None,
               weights: Optional[torch.Tensor] = None, values: bool = False, stream=None):
    """bsa_kv4_append: tokens of k, v (bf16 [B,Hkv,T,D], any strides with a contiguous last axis) into slots
    start[b] + t (int32 [B] on the device).  ``n_new``: tokens past it are padding; ``positions``: position of token
    0 (default start, which is right until tokens are evicted: from then on a sequence holds fewer tokens than it has
    had, and eviction's ``recent`` goes by positions); ``weights`` fp32 [B,Hkv,T]: initial accumulated weights
    (default 0; a cache without weights or positions keeps none).  With ``values``
    returns what the cache now holds, (k, v) bf16 [B,Hkv,T,D], 0 for padding."""
    dev, index = cache.device, cache.index
    B, H, T, D = k.shape if k.dim() == 4 else (0, 0, 0, 0)
    if (B, H, D) != (cache.B, cache.Hkv, cache.D) or v.shape != k.shape:
        raise ValueError("k and v must both be [B, Hkv, T, D] with the cache's B, Hkv and D")
    ks, vs = _rows("k", k, index), _rows("v", v, index)
    w0 = 0 if weights is None else _need("weights", weights, torch.float32, index, (B, H, T))
    if start is None:
        raise ValueError("start is missing")
    ctx, handle = _place(dev, index, stream)
    with ctx:
        kv = vv = None
        if values:
            kv = torch.empty((B, H, T, D), dtype=torch.bfloat16, device=dev)
            vv = torch.empty_like(kv)
        args = cache._c + _abi.KV4_APPEND_REST.pack(
            k.data_ptr(), v.data_ptr(), *ks, *vs, T, _lens("start", start, B, index), _lens("n_new", n_new, B, index),
            _lens("positions", positions, B, index), w0, kv.data_ptr() if values else 0, vv.data_ptr() if values else 0)
        check(_abi.lib().bsa_kv4_append(args, handle), "bsa_kv4_append")
    return (kv, vv) if values else None


def kv4_fwd(q: torch.Tensor, cache: KV4Cache, lens: torch.Tensor, *, q_lens: Optional[torch.Tensor] = None,
            o: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None, softmax_scale: Optional[float] = None,
            logits_soft_cap: Optional[float] = None, sinks: Optional[torch.Tensor] = None, accumulate: bool = False,
            stream=None):
    """bsa_kv4_fwd: attention of T new tokens over the cache.  q bf16 [B,Hq,T,D] (any strides with a contiguous last
    axis, e.g. a transposed [B,T,Hq,D]), lens int32 [B] on the device: keys held, the new tokens' own included
    -> (o bf16 [B,Hq,T,D], lse fp32 [B,Hq,T]).  ``q_lens``: new tokens per sequence (default T).  With
    ``accumulate`` every key's probabilities are added to cache.weights."""
    dev, index = cache.device, cache.index
    qs = _rows("q", q, index)
    B, Hq, T, D = q.shape
    if B != cache.B or D != cache.D:
        raise ValueError("q must be [B, Hq, T, D] with the cache's B and D")
    if lens is None:
        raise ValueError("lens is missing")
    sp, sn, skv = (0, 0, 0) if sinks is None else _sink_fields(sinks, cache.Hkv)
    if sinks is not None and sinks.device != dev:
        raise ValueError(f"sinks is on {sinks.device}, the call's other tensors are on {dev}")
    ctx, handle = _place(dev, index, stream)
    with ctx:
        if o is None:
            o = torch.empty((B, Hq, T, D), dtype=torch.bfloat16, device=dev)
        elif o.shape != q.shape:
            raise ValueError("o must have q's shape")
        if lse is None:
            lse = torch.empty((B, Hq, T), dtype=torch.float32, device=dev)
        head = (q.data_ptr(), o.data_ptr(), _need("lse", lse, torch.float32, index, (B, Hq, T)), *qs, *_rows("o", o, index),
                Hq, T, _lens("lens", lens, B, index), _lens("q_lens", q_lens, B, index),
                math.nan if softmax_scale is None else softmax_scale, logits_soft_cap or 0.0, sp, sn, skv,
                1 if accumulate else 0)
        pack = _abi.KV4_FWD_REST.pack
        need = _workspace_size("bsa_kv4_fwd", (index, B, cache.Hkv, D, cache.capacity, Hq, T, accumulate),
                               cache._c + pack(*head, 0, 0))
        ws = _workspace(need, dev)
        check(_abi.lib().bsa_kv4_fwd(cache._c + pack(*head, 0 if ws is None else ws.data_ptr(), need), handle), "bsa_kv4_fwd")
    return o, lse


def kv4_evict(cache: KV4Cache, lens: torch.Tensor, keep: int, *, recent: int = 0, seen: Optional[torch.Tensor] = None,
              out: Optional[KV4Cache] = None, values: bool = False, stream=None):
    """bsa_kv4_evict: keep the ``keep`` slots of largest accumulated weight of every sequence and key head, the last
    ``recent`` positions (of ``seen`` tokens, default lens) before all others.  In place, or into ``out`` (another
    cache of at least ``keep`` slots).  -> (new lens int32 [B], index int32 [B,Hkv,keep]: the slot each kept token
    had, -1 past the new length), with ``values`` also (k, v) bf16 [B,Hkv,keep,D] of the kept slots."""
    dev, index = cache.device, cache.index
    dst = cache if out is None else out
    if dst.index != index:
        raise ValueError(f"out is on {dst.device}, the cache is on {dev}")
    if lens is None:
        raise ValueError("lens is missing")
    B, H, D = cache.B, cache.Hkv, cache.D
    caches, pack = cache._c + dst._c, _abi.KV4_EVICT_REST.pack
    head = (_lens("lens", lens, B, index), _lens("seen", seen, B, index), keep, recent)
    need = _workspace_size("bsa_kv4_evict", (index, B, H, D, cache.capacity, dst.capacity, keep, recent, caches[:8] == dst._c[:8]),
                           caches + pack(*head, 0, 0, 0, 0, 0, 0))
    ctx, handle = _place(dev, index, stream)
    with ctx:
        new_lens = torch.empty((B,), dtype=torch.int32, device=dev)
        slots = torch.empty((B, H, keep), dtype=torch.int32, device=dev)
        kv = vv = None
        if values:
            kv = torch.empty((B, H, keep, D), dtype=torch.bfloat16, device=dev)
            vv = torch.empty_like(kv)
        ws = _workspace(need, dev)
        check(_abi.lib().bsa_kv4_evict(
            caches + pack(*head, new_lens.data_ptr(), slots.data_ptr(), kv.data_ptr() if values else 0,
                          vv.data_ptr() if values else 0, 0 if ws is None else ws.data_ptr(), need), handle), "bsa_kv4_evict")
    return (new_lens, slots, kv, vv) if values else (new_lens, slots)


def _pages(name: str, t: torch.Tensor, index: int):
    """Strides (page, head, token) of a cache tensor [pages, Hkv, page, D]."""
    strides = sp, sh, st = _rows(name, t, index)
    if (sp <= 0 or sh <= 0 or st <= 0) and (min(strides) < 0 or any(n > 1 and s == 0 for n, s in zip(t.shape, strides))):
        raise ValueError(f"{name} must not have several rows in one place")
    return strides


class PagedCache:
    """A key/value cache in pages (bsa_paged_cache): the buffers, which the caller owns.

    k, v: bf16 [pages, Hkv, page, D], any strides with a contiguous last axis (e.g. [pages, page, Hkv, D]
    transposed); bounds: bf16 [pages, Hkv, 2, D], an upper and a lower bound of each channel of a page's keys, which
    ``paged_append`` keeps and ``paged_select`` reads, or None.  page is 16, 32, 64, 128 or 256."""

    __slots__ = ("k", "v", "bounds", "pages", "Hkv", "page", "D", "device", "index", "_c")

    def __init__(self, k: torch.Tensor, v: torch.Tensor, bounds: Optional[torch.Tensor] = None):
        index, shape = k.get_device(), k.shape
        if index < 0 or len(shape) != 4:
            raise ValueError("k must be a CUDA bfloat16 tensor [pages, Hkv, page, D]")
        if v.shape != shape:
            raise ValueError("v must have k's shape")
        P, H, page, D = shape
        self._c = _abi.PAGED_CACHE.pack(
            k.data_ptr(), v.data_ptr(), *_pages("k", k, index), *_pages("v", v, index),
            0 if bounds is None else _need("bounds", bounds, torch.bfloat16, index, (P, H, 2, D)), P, H, D, page)
        self.k, self.v, self.bounds = k, v, bounds
        self.pages, self.Hkv, self.page, self.D, self.device, self.index = P, H, page, D, k.device, index

    @classmethod
    def empty(cls, pages: int, Hkv: int, page: int, D: int, device="cuda", bounds: bool = True) -> "PagedCache":
        """A cache without tokens; without ``bounds`` it keeps none."""
        def new(*shape):
            return torch.zeros(shape, dtype=torch.bfloat16, device=device)
        return cls(new(pages, Hkv, page, D), new(pages, Hkv, page, D), new(pages, Hkv, 2, D) if bounds else None)


def paged_table(pages: int, B: int, M: int, device="cuda"):
    """(table int32 [B, M], free int32 [pages], used int32 [1]) of a cache of `pages` pages that holds no sequence yet."""
    return (torch.full((B, M), -1, dtype=torch.int32, device=device), torch.arange(pages, dtype=torch.int32, device=device),
            torch.zeros((1,), dtype=torch.int32, device=device))


def _table(table: torch.Tensor, B: int, index: int) -> int:
    if table.dim() != 2:
        raise ValueError("table must be [B, M]")
    return _need("table", table, torch.int32, index, (B, table.shape[1]))


def paged_resize(table: torch.Tensor, free: torch.Tensor, used: torch.Tensor, lens: torch.Tensor, new_lens: torch.Tensor,
                 page: int, T: int, *, stream=None):
    """bsa_paged_resize: sequences of ``lens`` tokens get ``new_lens`` (int32 [B], 0 for one that has ended); pages go back
    to the free stack and from it into the rows of ``table`` (int32 [B, M]) and ``free`` (int32 [pages], entries used[0] ..
    are free), both in place; a page that rows share is given back by each of them (nothing counts references).  -> (lens
    int32 [B] that they now have, used int32 [1], slots int32 [B, T]: where the tokens lens[b] + i go, -1 behind the last).
    Where the pages do not suffice a sequence, and every later one that needs any, keeps its length."""
    index = table.get_device()
    if index < 0:
        raise ValueError("table must be a contiguous CUDA int32 tensor")
    if lens is None or new_lens is None:
        raise ValueError("lens and new_lens are missing")
    B = table.shape[0]
    head = (_table(table, B, index), _need("free", free, torch.int32, index, (free.numel(),)),
            _need("used", used, torch.int32, index, (1,)), _lens("lens", lens, B, index), _lens("new_lens", new_lens, B, index))
    ctx, handle = _place(table.device, index, stream)
    with ctx:
        out, used_out = torch.empty_like(lens), torch.empty_like(used)
        slots = torch.empty((B, max(T, 0)), dtype=torch.int32, device=table.device)
        check(_abi.lib().bsa_paged_resize(
            _abi.PAGED_RESIZE.pack(*head, out.data_ptr(), used_out.data_ptr(), slots.data_ptr(), B, table.shape[1], T, free.numel(),
                                   page), handle), "bsa_paged_resize")
    return out, used_out, slots


def paged_append(cache: PagedCache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, *, stream=None) -> None:
    """bsa_paged_append: tokens of k, v (bf16 [B,Hkv,T,D], any strides with a contiguous last axis) into ``slots`` (int32
    [B, T] on the device, negative: padding), as ``paged_resize`` gives them; the bounds of their pages are
    renewed if the cache has any.  Without bounds the slots may come in any order."""
    index = cache.index
    B, H, T, D = k.shape if k.dim() == 4 else (0, 0, 0, 0)
    if (H, D) != (cache.Hkv, cache.D) or v.shape != k.shape:
        raise ValueError("k and v must both be [B, Hkv, T, D] with the cache's Hkv and D")
    ks, vs = _rows("k", k, index), _rows("v", v, index)
    args = cache._c + _abi.PAGED_APPEND_REST.pack(k.data_ptr(), v.data_ptr(), *ks, *vs,
                                                  _need("slots", slots, torch.int32, index, (B, T)), B, T)
    ctx, handle = _place(cache.device, index, stream)
    with ctx:
        check(_abi.lib().bsa_paged_append(args, handle), "bsa_paged_append")


def paged_select(q: torch.Tensor, cache: PagedCache, table: torch.Tensor, lens: torch.Tensor, keep: int, *, first: int = 1,
                 recent: int = 1, q_lens: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """bsa_paged_select: for every new token and key head the ``keep`` pages with the largest bound on q.k (q rounded to
    8 bits), the ``first`` and the last ``recent`` ones that it sees among them.  q bf16 [B,Hq,T,D] (any strides with a
    contiguous last axis), lens int32 [B] with the new tokens' own keys included -> int32 [B,Hkv,T,keep], numbers of the
    sequence's pages in increasing order, -1 behind the last; for ``paged_fwd``'s ``select``."""
    dev, index = cache.device, cache.index
    qs = _rows("q", q, index)
    B, Hq, T, D = q.shape
    if D != cache.D:
        raise ValueError("q must be [B, Hq, T, D] with the cache's D")
    if lens is None:
        raise ValueError("lens is missing")
    head = (q.data_ptr(), *qs, _table(table, B, index), _lens("lens", lens, B, index), _lens("q_lens", q_lens, B, index))
    ctx, handle = _place(dev, index, stream)
    with ctx:
        out = torch.empty((B, cache.Hkv, T, max(keep, 0)), dtype=torch.int32, device=dev)
        args = cache._c + _abi.PAGED_SELECT_REST.pack(*head, out.data_ptr(), B, Hq, table.shape[1], T, keep, first, recent)
        check(_abi.lib().bsa_paged_select(args, handle), "bsa_paged_select")
    return out


def paged_fwd(q: torch.Tensor, cache: PagedCache, table: torch.Tensor, lens: torch.Tensor, *,
              q_lens: Optional[torch.Tensor] = None, select: Optional[torch.Tensor] = None, local_left: Optional[int] = None,
              chunk: Optional[int] = None, o: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
              softmax_scale: Optional[float] = None, logits_soft_cap: Optional[float] = None,
              sinks: Optional[torch.Tensor] = None, stream=None):
    """bsa_paged_fwd: attention of T new tokens over their sequences' pages.  q bf16 [B,Hq,T,D] (any strides with a
    contiguous last axis), table int32 [B, M], lens int32 [B] on the device: keys held, the new tokens' own included
    -> (o bf16 [B,Hq,T,D], lse fp32 [B,Hq,T]).  ``q_lens``: new tokens per sequence (default T).  ``local_left`` or
    ``chunk``: the local or chunked causal mask instead of the causal one.  ``select`` (int32 [B,Hkv,T,keep] from
    ``paged_select``): only the pages listed for each query."""
    dev, index = cache.device, cache.index
    qs = _rows("q", q, index)
    B, Hq, T, D = q.shape
    if D != cache.D:
        raise ValueError("q must be [B, Hq, T, D] with the cache's D")
    if lens is None:
        raise ValueError("lens is missing")
    if local_left is not None and chunk is not None:
        raise ValueError("local_left and chunk exclude each other")
    kind = _abi.MASK_LOCAL if local_left is not None else _abi.MASK_CHUNKED_CAUSAL if chunk is not None else _abi.MASK_CAUSAL
    keep = 0
    if select is not None:
        if select.dim() != 4 or select.shape[3] < 1:
            raise ValueError("select must be [B, Hkv, T, keep]")
        keep = select.shape[3]
    sp, sn, skv = (0, 0, 0) if sinks is None else _sink_fields(sinks, cache.Hkv)
    if sinks is not None and sinks.device != dev:
        raise ValueError(f"sinks is on {sinks.device}, the call's other tensors are on {dev}")
    tp, M = _table(table, B, index), table.shape[1]
    ctx, handle = _place(dev, index, stream)
    with ctx:
        if o is None:
            o = torch.empty_like(q) if q.is_contiguous() else torch.empty((B, Hq, T, D), dtype=torch.bfloat16, device=dev)
            os = (Hq * T * D, T * D, D)
        elif o.shape != q.shape:
            raise ValueError("o must have q's shape")
        else:
            os = _rows("o", o, index)
        if lse is None:
            lse = torch.empty((B, Hq, T), dtype=torch.float32, device=dev)
        else:
            _need("lse", lse, torch.float32, index, (B, Hq, T))
        head = (q.data_ptr(), o.data_ptr(), lse.data_ptr(), *qs, *os, tp, _lens("lens", lens, B, index), _lens("q_lens", q_lens, B, index),
                0 if select is None else _need("select", select, torch.int32, index, (B, cache.Hkv, T, keep)), B, Hq, M, T, keep,
                kind, -1 if local_left is None else local_left, chunk or 0, math.nan if softmax_scale is None else softmax_scale,
                logits_soft_cap or 0.0, sp, sn, skv)
        pack = _abi.PAGED_FWD_REST.pack
        need = _workspace_size("bsa_paged_fwd", (index, B, cache.Hkv, D, cache.page, Hq, M, T, keep, kind, local_left, chunk), lambda: cache._c + pack(*head, 0, 0))
        own = _raw_alloc(need, handle) if need and _raw_alloc and _raw_free else 0
        held = _workspace(0 if own else need, dev)
        try:
            check(_abi.lib().bsa_paged_fwd(cache._c + pack(*head, own or _ptr(held) or 0, need), handle), "bsa_paged_fwd")
        finally:
            if own:
                _raw_free(own)
    return o, lse


def get_device_error(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device error word; raises if non-zero."""
    w = C.c_uint32(0)
    st = _abi.lib().bsa_get_device_error(_stream(stream), C.byref(w))
    if st != _abi.OK:
        raise BsaError(st, f"device error word {w.value:#x}")
    return w.value


def set_wait_limit_ns(ns: int) -> None:
    check(_abi.lib().bsa_set_wait_limit_ns(ns), "bsa_set_wait_limit_ns")


def debug_wait_timeout(stream=None) -> None:
    check(_abi.lib().bsa_debug_wait_timeout(_stream(stream)), "bsa_debug_wait_timeout")


def debug_selfcheck(stream=None) -> None:
    """bsa_debug_selfcheck: out-of-range indices through the range checks
    (recorded only by the range-checked build)."""
    check(_abi.lib().bsa_debug_selfcheck(_stream(stream)), "bsa_debug_selfcheck")
