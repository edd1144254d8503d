"""Binding of the entry points between the QKV product and the output
projection: normalisation and rotation of queries and keys, the paged cache,
and attention of drafted tokens over it (``include/skg.h`` has the contract).

Rows are tensors [T, heads, head_dim] whose heads are adjacent; tokens may be
any multiple of 16 bytes apart, so the parts of a fused QKV buffer are taken as
they lie.  Every tensor of a call has to be on the current device.
"""

from __future__ import annotations

import ctypes
import math

import torch

from . import OK, Q8_1_BLOCK_BYTES, _stream, check, lib

# skg_kv_fmt
KV_BF16, KV_Q8_0, KV_Q4_0 = range(3)
# skg_dtype
F32, BF16 = range(2)
_DTYPE = {torch.float32: F32, torch.bfloat16: BF16}


class _Cache(ctypes.Structure):
    _fields_ = [("fmt", ctypes.c_int32), ("heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("pages", ctypes.c_int64), ("k", ctypes.c_void_p),
                ("v", ctypes.c_void_p)]


class _Rope(ctypes.Structure):
    _fields_ = [("rot", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("norm", ctypes.c_int32),
                ("eps", ctypes.c_float), ("pos", ctypes.c_void_p), ("inv_freq", ctypes.c_void_p),
                ("gq", ctypes.c_void_p), ("gk", ctypes.c_void_p)]


def kv_bytes(fmt: int, heads: int, head_dim: int, page_size: int, pages: int) -> int:
    """Bytes of one of a cache's two buffers (0: invalid description)."""
    return int(lib.skg_kv_bytes(fmt, heads, head_dim, page_size, pages))


class KvCache:
    """A paged cache over two buffers of the caller, kept alive by this handle.

    k and v are contiguous GPU tensors of any type, of equal size, holding a
    whole number of pages; the layout of their bytes is in ``include/skg.h``.
    """

    def __init__(self, fmt: int, heads: int, head_dim: int, page_size: int, k, v):
        page = kv_bytes(fmt, heads, head_dim, page_size, 1)
        if page == 0:
            check(lib.skg_kv_store(ctypes.byref(_Cache(fmt, heads, head_dim, page_size, 1, None, None)), 0, 1, None, 0,
                                   None, 0, None, None))
        for name, t in (("k", k), ("v", v)):
            if not t.is_cuda:
                raise ValueError(f"{name} must be on the GPU")
            if not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous")
        size = k.numel() * k.element_size()
        if size != v.numel() * v.element_size() or k.get_device() != v.get_device():
            raise ValueError("k and v must be of one size, on one device")
        if size == 0 or size % page:
            raise ValueError(f"buffers of {size} bytes are not whole pages of {page} bytes")
        if max(k.data_ptr(), v.data_ptr()) < min(k.data_ptr(), v.data_ptr()) + size:
            raise ValueError("k and v overlap")
        self.fmt, self.heads, self.head_dim, self.page_size = fmt, heads, head_dim, page_size
        self.pages = size // page
        self.k, self.v = k, v
        self._device = k.get_device()
        self._c = _Cache(fmt, heads, head_dim, page_size, self.pages, k.data_ptr(), v.data_ptr())
        self._ref = ctypes.byref(self._c)


def kv_cache(fmt: int, heads: int, head_dim: int, page_size: int, pages: int, device=None) -> KvCache:
    """A cache over two new buffers (contents undefined until stored)."""
    size = kv_bytes(fmt, heads, head_dim, page_size, pages)
    if size == 0:
        check(lib.skg_kv_store(ctypes.byref(_Cache(fmt, heads, head_dim, page_size, pages, None, None)), 0, 1, None, 0,
                               None, 0, None, None))
    k, v = (torch.empty(size, dtype=torch.uint8, device=device or torch.device("cuda")) for _ in range(2))
    return KvCache(fmt, heads, head_dim, page_size, k, v)


# A decode step's small calls cost more here than on the GPU (a launch is 2 to
# 4 us of the host's time, torch.cuda.current_stream() alone 2.8), so what every
# call does is kept short: the stream's handle without a Stream object around
# it, and no checks of tensors that are made here.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _on_stream(stream, dev: int) -> int:
    return _raw_stream(dev) if stream is None and _raw_stream is not None else _stream(stream)


def _device(t, what: str) -> int:
    """The current device, which has to be t's."""
    if not t.is_cuda:
        raise ValueError(f"{what} must be on the GPU")
    dev = torch.cuda.current_device()
    if t.get_device() != dev:
        raise ValueError(f"{what} is on device {t.get_device()}, the current device is {dev}")
    return dev


def _dtype(t, what: str) -> int:
    dt = _DTYPE.get(t.dtype)
    if dt is None:
        raise ValueError(f"{what} must be float32 or bfloat16 (got {t.dtype})")
    return dt


def _rows(t, what: str, shape, dtype, dev: int):
    """Pointer and token stride (elements) of rows [T, heads, D]."""
    if t.shape != shape:
        raise ValueError(f"{what} must be {list(shape)} (got {list(t.shape)})")
    if t.dtype != dtype:
        raise ValueError(f"{what} must be {dtype} (got {t.dtype})")
    if t.get_device() != dev:
        raise ValueError(f"{what} must be on the current GPU")
    T, heads, D = shape
    ld, head, one = t.stride()
    if one != 1 or (head != D and heads > 1):
        raise ValueError(f"the heads of {what} must be adjacent (strides {list(t.stride())})")
    return t.data_ptr(), ld if T > 1 else heads * D


def _flat(t, what: str, n: int, dtypes, dev: int) -> int:
    """Pointer of a contiguous tensor of n elements at least."""
    if t.dtype not in dtypes:
        raise ValueError(f"{what} must be {dtypes[0]} (got {t.dtype})")
    if t.get_device() != dev:
        raise ValueError(f"{what} must be on the current GPU")
    if not t.is_contiguous() or t.numel() < n:
        raise ValueError(f"{what} must be contiguous and hold {n} elements (it holds {t.numel()})")
    return t.data_ptr()


_I32, _I64, _F32, _MASK = (torch.int32,), (torch.int64,), (torch.float32,), (torch.int64, torch.uint64)


def _on(stream, tensors):
    """Tells the allocator of tensors made here that `stream`, not the current
    stream, uses them."""
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()
    if stream.cuda_stream != torch.cuda.current_stream().cuda_stream:
        for t in tensors:
            t.record_stream(stream)


def _rope(T: int, hq: int, hk: int, D: int, pos, inv_freq, gq, gk, eps: float, norm: bool, interleaved: bool, dev: int):
    rot = 0 if inv_freq is None else 2 * inv_freq.numel()
    r = _Rope(rot, interleaved, norm, eps, None, None, None, None)
    if rot:
        if pos is None:
            raise ValueError("pos is required")
        r.pos = _flat(pos, "pos", T, _I32, dev)
        r.inv_freq = _flat(inv_freq, "inv_freq", 1, _F32, dev)
    if norm:
        if gq is not None and hq:
            r.gq = _flat(gq, "gq", D, _F32, dev)
        if gk is not None and hk:
            r.gk = _flat(gk, "gk", D, _F32, dev)
    return r


def cache_args(cache: KvCache):
    """The skg_kv_cache argument of direct calls of ``lib`` (by reference)."""
    return cache._ref


def rope_args(head_dim: int, pos, inv_freq, gq=None, gk=None, eps: float = 1e-6, norm: bool = False,
              interleaved: bool = False):
    """The skg_rope argument of direct calls of ``lib`` (by reference), for
    pos.numel() tokens; the tensors have to outlive it."""
    return ctypes.byref(_rope(pos.numel(), 1, 1, head_dim, pos, inv_freq, gq, gk, eps, norm, interleaved,
                              _device(pos, "pos")))


def qk_norm_rope(q, k, pos, inv_freq, gq=None, gk=None, eps: float = 1e-6, norm: bool = False,
                 interleaved: bool = False, qo=None, ko=None, stream=None):
    """RMSNorm (norm=True, gains gq / gk [D] or None) of every head of q
    [T, hq, D] and k [T, hk, D] and their rotation by pos[t] * inv_freq[i], in
    one pass.  The first 2 * len(inv_freq) elements of a head are turned, in
    adjacent pairs (interleaved) or in pairs half of them apart.  Either of q
    and k may be None; qo=q, ko=k work in place.  Returns (qo, ko).
    """
    x = q if q is not None else k
    if x is None:
        raise ValueError("q or k is required")
    dev = _device(x, "q" if q is not None else "k")
    dt = _dtype(x, "q" if q is not None else "k")
    for t in (q, k):
        if t is not None and t.dim() != 3:
            raise ValueError(f"rows must be [T, heads, head_dim] (got {list(t.shape)})")
    T, _, D = x.shape
    hq, hk = 0 if q is None else q.shape[1], 0 if k is None else k.shape[1]
    r = _rope(T, hq, hk, D, pos, inv_freq, gq, gk, eps, norm, interleaved, dev)
    qp = kp = qop = kop = None
    ldq = ldk = ldqo = ldko = 0
    mine = []
    if q is not None:
        shape = (T, hq, D)
        qp, ldq = _rows(q, "q", shape, x.dtype, dev)
        if qo is None:
            qo = x.new_empty(shape)
            mine.append(qo)
            qop, ldqo = qo.data_ptr(), hq * D
        else:
            qop, ldqo = _rows(qo, "qo", shape, x.dtype, dev)
    if k is not None:
        shape = (T, hk, D)
        kp, ldk = _rows(k, "k", shape, x.dtype, dev)
        if ko is None:
            ko = x.new_empty(shape)
            mine.append(ko)
            kop, ldko = ko.data_ptr(), hk * D
        else:
            kop, ldko = _rows(ko, "ko", shape, x.dtype, dev)
    if stream is not None:
        _on(stream, mine)
    st = lib.skg_qk_norm_rope(dt, T, hq, hk, D, qp, ldq, kp, ldk, ctypes.byref(r), qop, ldqo, kop, ldko,
                              _on_stream(stream, dev))
    if st != OK:
        check(st)
    return (qo if q is not None else None), (ko if k is not None else None)


def kv_store(cache: KvCache, k, v, slots, stream=None) -> None:
    """Encodes rows k and v [T, heads, D] into slots[t] (int64) of the cache; a
    slot outside it (a padded token's -1) is skipped."""
    dev = _device(k, "k")
    dt = _dtype(k, "k")
    if cache._device != dev:
        raise ValueError("the cache must be on the current GPU")
    if k.dim() != 3:
        raise ValueError(f"rows must be [T, heads, head_dim] (got {list(k.shape)})")
    T = k.shape[0]
    shape = (T, cache.heads, cache.head_dim)
    kp, ldk = _rows(k, "k", shape, k.dtype, dev)
    vp, ldv = _rows(v, "v", shape, k.dtype, dev)
    st = lib.skg_kv_store(cache._ref, dt, T, kp, ldk, vp, ldv, _flat(slots, "slots", T, _I64, dev),
                          _on_stream(stream, dev))
    if st != OK:
        check(st)


def kv_load(cache: KvCache, slots, dtype=torch.float32, k=None, v=None, stream=None):
    """The values in slots [T] (int64) as rows [T, heads, D] of `dtype` (or of
    the given k and v); zeros for a slot outside the cache.  Returns (k, v)."""
    dev = _device(slots, "slots")
    T = slots.numel()
    if cache._device != dev:
        raise ValueError("the cache must be on the current GPU")
    shape = (T, cache.heads, cache.head_dim)
    mine = []
    if k is None:
        k = torch.empty(shape, dtype=dtype if v is None else v.dtype, device=slots.device)
        mine.append(k)
    if v is None:
        v = k.new_empty(shape)
        mine.append(v)
    dt = _dtype(k, "k")
    kp, ldk = _rows(k, "k", shape, k.dtype, dev)
    vp, ldv = _rows(v, "v", shape, k.dtype, dev)
    if stream is not None:
        _on(stream, mine)
    st = lib.skg_kv_load(cache._ref, dt, T, _flat(slots, "slots", T, _I64, dev), kp, ldk, vp, ldv,
                         _on_stream(stream, dev))
    if st != OK:
        check(st)
    return k, v


def qkv_rope_store(cache: KvCache, q, k, v, slots, pos, inv_freq, gq=None, gk=None, eps: float = 1e-6,
                   norm: bool = False, interleaved: bool = False, qo=None, stream=None):
    """qk_norm_rope of q, and kv_store of the normalised and rotated k and of
    v, in one launch.  Returns qo."""
    dev = _device(q, "q")
    dt = _dtype(q, "q")
    if q.dim() != 3:
        raise ValueError(f"q must be [T, heads, head_dim] (got {list(q.shape)})")
    T, hq, D = q.shape
    if cache._device != dev or cache.head_dim != D:
        raise ValueError("the cache must be on the current GPU and have q's head_dim")
    r = _rope(T, hq, cache.heads, D, pos, inv_freq, gq, gk, eps, norm, interleaved, dev)
    qp, ldq = _rows(q, "q", (T, hq, D), q.dtype, dev)
    shape = (T, cache.heads, D)
    kp, ldk = _rows(k, "k", shape, q.dtype, dev)
    vp, ldv = _rows(v, "v", shape, q.dtype, dev)
    if qo is None:
        qo = q.new_empty((T, hq, D))
        qop, ldqo = qo.data_ptr(), hq * D
        if stream is not None:
            _on(stream, [qo])
    else:
        qop, ldqo = _rows(qo, "qo", (T, hq, D), q.dtype, dev)
    st = lib.skg_qkv_rope_store(cache._ref, dt, T, hq, qp, ldq, kp, ldk, vp, ldv, ctypes.byref(r),
                                _flat(slots, "slots", T, _I64, dev), qop, ldqo, _on_stream(stream, dev))
    if st != OK:
        check(st)
    return qo


def tree_attn_workspace(cache: KvCache, dtype, T: int, n_seqs: int, hq: int, max_draft: int, width: int,
                        max_kv: int = 0) -> int:
    """Bytes of workspace that a tree_attn call of these counts needs (0: none)."""
    return int(lib.skg_tree_attn_workspace(cache._ref, _DTYPE[dtype], T, n_seqs, hq, max_draft, width, max_kv))


def tree_attn(cache: KvCache, q, table, ctx, cu=None, mask=None, max_draft: int | None = None, max_kv: int = 0,
              scale: float | None = None, o=None, oq=None, workspace=None, stream=None):
    """Attention of the drafted tokens q [T, hq, D] of len(ctx) sequences.

    table [n_seqs, width] (int32) names each sequence's pages, ctx [n_seqs]
    (int32) its context; its tokens are rows cu[b]..cu[b+1]-1 (int32; None:
    equally many each), whose keys and values follow the context in the cache.
    mask [T] (int64 or uint64 bits) says which drafted tokens of its sequence
    a token sees; None: itself and those before it.  max_draft bounds the
    tokens of a sequence (64 at most; needed with cu unless T is small enough);
    max_kv bounds its keys.  scale defaults to 1 / sqrt(D).

    o: True or None to allocate [T, hq, D], a tensor to write into, False to
    skip it; oq: True or a tensor (uint8 [T, hq * D / 32, 36]) for the Q8_1
    blocks of o.  Returns o, or (o, oq) if oq was asked for.

    workspace: tree_attn_workspace(...) bytes that no other call uses at the
    time; None allocates it.
    """
    dev = _device(q, "q")
    dt = _dtype(q, "q")
    if q.dim() != 3:
        raise ValueError(f"q must be [T, heads, head_dim] (got {list(q.shape)})")
    T, hq, D = q.shape
    if cache._device != dev or cache.head_dim != D:
        raise ValueError("the cache must be on the current GPU and have q's head_dim")
    n = ctx.numel()
    if table.dim() != 2 or table.shape[0] != n:
        raise ValueError(f"table must be [{n}, width] (got {list(table.shape)})")
    width = table.shape[1]
    if max_draft is None:
        max_draft = (T // n if n else 0) if cu is None else min(T, 64)
    shape = (T, hq, D)
    qp, ldq = _rows(q, "q", shape, q.dtype, dev)
    mine = []
    if o is None or o is True:
        o = q.new_empty(shape)
        mine.append(o)
        op, ldo = o.data_ptr(), hq * D
    elif o is False:
        o, op, ldo = None, None, 0
    else:
        op, ldo = _rows(o, "o", shape, q.dtype, dev)
    oqp = None
    if oq is None or oq is False:
        oq = None
    else:
        nq = T * (hq * D // 32) * Q8_1_BLOCK_BYTES
        if oq is True:
            oq = torch.empty((T, hq * D // 32, Q8_1_BLOCK_BYTES), dtype=torch.uint8, device=q.device)
            mine.append(oq)
        oqp = _flat(oq, "oq", nq, (torch.uint8,), dev)
    size = lib.skg_tree_attn_workspace(cache._ref, dt, T, n, hq, max_draft, width, max_kv)
    wp = None
    if size:
        if workspace is None:
            workspace = torch.empty(size, dtype=torch.uint8, device=q.device)
            mine.append(workspace)
        elif workspace.get_device() != dev or not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous, on the current GPU")
        wp, size = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    if stream is not None:
        _on(stream, mine)
    st = lib.skg_tree_attn(
        cache._ref, dt, T, n, hq, max_draft, qp, ldq, None if cu is None else _flat(cu, "cu", n + 1, _I32, dev),
        _flat(ctx, "ctx", n, _I32, dev), _flat(table, "table", n * width, _I32, dev), width, max_kv,
        None if mask is None else _flat(mask, "mask", T, _MASK, dev), 1 / math.sqrt(D) if scale is None else scale,
        op, ldo, oqp, wp, size, _on_stream(stream, dev))
    if st != OK:
        check(st)
    return o if oq is None else (o, oq)
