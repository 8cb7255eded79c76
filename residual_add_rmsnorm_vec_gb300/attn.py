"""Tensor-level entry points of the attention path over the C ABI of
include/rmsnorm_attn.h (marshalling only): QK norm with multi-axis rotary
positions, the append to a paged E4M3 cache, and the attention over it.
Nothing here computes: a failed call raises ``RmsnError``.

The usual call (tensors of the current device, the current stream) is
marshalled natively (binding/attn_fast.cpp), with the same checks; what that
does not take comes back here, which makes the call or raises the error.
"""
from __future__ import annotations

import contextlib
import ctypes
import decimal
import functools
import math

import torch

from . import _attn_lib as _al
from . import _lib
from .api import _IN, _check

_CODES = (torch.uint8, torch.float8_e4m3fn)


# (cudaStream_t of the current stream of a device index; no Stream object)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


@contextlib.contextmanager
def _other(device, stream):
    """Device and stream of a call that names a stream, or whose tensors are
    on another device than the current one: outputs and workspaces are
    allocated, and the launch made, with both current.  Yields (cudaStream_t,
    keep): keep(t) holds a new output's memory back from other streams' use
    while the caller's stream still works on it."""
    caller = torch.cuda.current_stream(device)
    if stream is None:
        stream = caller
    elif stream.device != device:
        raise ValueError(f"stream must be on {device}, got {stream.device}")
    with torch.cuda.stream(stream):
        yield stream.cuda_stream, (lambda t: t.record_stream(caller)) if stream != caller else None


class _Fixed:
    """The attributes in ``_fixed`` are set once, by ``_set``: what a call reads
    beside the tensors (their shapes, addresses, device) cannot fall out of step
    with them.  A subclass may have others."""

    __slots__ = ()
    _fixed: tuple = ()

    def __setattr__(self, name, value):
        if name in self._fixed:
            raise AttributeError(f"{type(self).__name__}.{name} cannot be changed: make another")
        object.__setattr__(self, name, value)

    def __delattr__(self, name):
        if name in self._fixed:
            raise AttributeError(f"{type(self).__name__}.{name} cannot be removed")
        object.__delattr__(self, name)

    def _set(self, **values):
        for name, value in values.items():
            object.__setattr__(self, name, value)


class RopeTable(_Fixed):
    """Frequencies of the rotary pairs: ``turns`` (int64 bit patterns of 64-bit
    fractions of a turn per position), ``axis`` (int32, the axis whose position
    turns the pair), both [rot_dim / 2] on the device; made by ``rope_table``.
    The attributes are fixed."""

    _fixed = __slots__ = ("turns", "axis", "rot_dim", "n_axes", "index")

    def __init__(self, turns: torch.Tensor, axis: torch.Tensor, n_axes: int):
        if turns.dim() != 1:
            raise ValueError("turns must be [rot_dim / 2]")
        self._set(turns=turns, axis=axis, rot_dim=2 * turns.numel(), n_axes=int(n_axes),
                  index=turns.get_device())
        self._pointers()

    def _pointers(self):
        """Addresses of turns and axis, which are still what they were made as
        (a tensor can be given other data in place)."""
        pairs = (self.rot_dim // 2,)
        _check("turns", self.turns, pairs, (torch.int64,))
        _check("axis", self.axis, pairs, (torch.int32,), self.turns.device)
        if self.turns.get_device() != self.index:
            raise ValueError(f"the table was moved to {self.turns.device}")
        return self.turns.data_ptr(), self.axis.data_ptr()

    def __reduce__(self):
        return type(self), (self.turns, self.axis, self.n_axes)


@functools.lru_cache(maxsize=16)
def _turns_per_radian(bits: int) -> int:
    """2^bits / (2 pi) to within a few units (pi by Machin's formula,
    16 atan(1/5) - 4 atan(1/239))."""
    def atan_of_one_over(n):
        term = total = (1 << bits) // n
        k = 1
        while term:
            term //= -n * n
            k += 2
            total += term // k
        return total

    bits += 16
    pi = 16 * atan_of_one_over(5) - 4 * atan_of_one_over(239)
    return (1 << (2 * bits - 1)) // pi >> 16


def _turn_bits(num: int, shift: int) -> int:
    """num / 2^shift radians in turns: the fraction of a turn, rounded to 64 bits."""
    # the whole turns, the 64 bits, and 64 to round by; in steps, for the cache
    bits = (max(0, abs(num).bit_length() - shift) + 191) // 64 * 64
    return ((num * _turns_per_radian(bits) >> (shift + bits - 65)) + 1 >> 1) % 2**64


def rope_table(rot_dim: int, *, base: float = 10000.0, sections=None, axis=None, inv_freq=None,
               device="cuda") -> RopeTable:
    """Table of ``rot_dim / 2`` rotary pairs.

    Pair p turns by ``inv_freq[p]`` radians per position, by default
    ``base ** (-2 p / rot_dim)``; the table holds either to the nearest 2^-64
    of a turn.  ``sections`` gives consecutive pairs to the
    axes (time, height, width, ...; they add up to rot_dim / 2); ``axis`` names
    each pair's axis instead; neither: one axis.
    """
    if rot_dim < 0 or rot_dim % 2:
        raise ValueError("rot_dim must be even and not negative")
    pairs = rot_dim // 2
    if sections is not None and axis is not None:
        raise ValueError("give sections or axis, not both")
    if sections is not None:
        if min(sections, default=0) < 0 or sum(sections) != pairs:
            raise ValueError(f"sections must add up to {pairs}, got {list(sections)}")
        n_axes = len(sections)
        axes = [i for i, n in enumerate(sections) for _ in range(n)]
    else:
        axes = [0] * pairs if axis is None else [int(i) for i in axis]
        if len(axes) != pairs or min(axes, default=0) < 0:
            raise ValueError(f"axis must name {pairs} axes")
        n_axes = max(axes, default=0) + 1
    if inv_freq is None:
        base = float(base)
        if not base > 0:
            raise ValueError("base must be positive")
        # fixed-point powers of one step; a base below 1 makes large ones
        large = max(0, 1 - math.frexp(base)[1])
        shift = 192 + 2 * large
        with decimal.localcontext(decimal.Context(prec=64 + large)):
            step = int(decimal.Decimal(base) ** (decimal.Decimal(-2) / max(rot_dim, 1)) * (1 << shift))
        freqs = [(1 << shift, shift)][:pairs]
        while len(freqs) < pairs:
            freqs.append((freqs[-1][0] * step >> shift, shift))
    else:
        freqs = [float(f) for f in inv_freq]
        if len(freqs) != pairs:
            raise ValueError(f"inv_freq must hold {pairs} values")
        if not all(math.isfinite(f) for f in freqs):
            raise ValueError("frequencies must be finite")
        freqs = [(n, d.bit_length() - 1) for n, d in map(float.as_integer_ratio, freqs)]
    bits = [_turn_bits(*f) for f in freqs]
    bits = [b - 2**64 if b >= 2**63 else b for b in bits]
    return RopeTable(torch.tensor(bits, dtype=torch.int64, device=device),
                     torch.tensor(axes, dtype=torch.int32, device=device), n_axes)


def _heads(name, t, head_dim):
    """(heads, token stride) of [T, H * head_dim] or [T, H, head_dim] with the
    heads of a token back to back."""
    shape, stride = t.shape, t.stride()
    if len(shape) == 2:
        width = shape[1]
        if width % head_dim:
            raise ValueError(f"{name}: rows must hold whole heads of head_dim elements")
        ok = stride[1] == 1 or width == 1
    elif len(shape) == 3:
        if shape[2] != head_dim:
            raise ValueError(f"{name}: rows must hold whole heads of head_dim elements")
        width = shape[1] * head_dim
        ok = (stride[2] == 1 or head_dim == 1) and (stride[1] == head_dim or shape[1] <= 1)
    else:
        raise ValueError(f"{name} must be [T, heads * head_dim] or [T, heads, head_dim]")
    if not ok:
        raise ValueError(f"{name}: a token's heads must lie back to back")
    return width // head_dim, (stride[0] if shape[0] > 1 else width)


def _like(name, out, x, dt, index):
    if out.shape != x.shape or out.dtype != dt or out.get_device() != index:
        raise ValueError(f"{name} must be like {name[0]}")
    return out


def qk_norm_rope(q: torch.Tensor | None, k: torch.Tensor | None, positions: torch.Tensor,
                 table: RopeTable, q_weight: torch.Tensor | None = None,
                 k_weight: torch.Tensor | None = None, *, head_dim: int, eps: float | None = None,
                 weight_offset: float = 0.0, interleaved: bool = False,
                 q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None,
                 stream: torch.cuda.Stream | None = None, pdl: bool = False):
    """QK norm and rotary positions of q and k in one launch
    (``rmsattn_qk_rope_fwd``).

    q is [T, Hq * head_dim] or [T, Hq, head_dim], likewise k (either may be
    None); both may be column slices of a fused qkv matrix.  positions is [T]
    for a table of one axis, else [n_axes, T] (``p.expand(n_axes, T)`` where
    all axes agree), int32 or int64.  ``eps``: the norm's; None leaves the norm (and the weights) out.  ``interleaved``:
    pairs are neighbouring elements, else halves of the first rot_dim.  The
    results go to q_out / k_out (new tensors where None; pass q and k
    themselves to work in place).  Returns ``(q_out, k_out)``.
    """
    if stream is None:
        done = (_al._fast or _al.load_fast()).qk_rope(
            q, k, positions, table.turns, table.axis, table.n_axes, q_weight, k_weight, head_dim,
            eps, weight_offset, interleaved, q_out, k_out, pdl)
        if done is not None:
            return done
    ref = q if q is not None else k
    if ref is None:
        return q_out, k_out
    if head_dim < 1:
        raise ValueError("head_dim must be positive")
    dt, index, T = ref.dtype, ref.get_device(), ref.shape[0]
    flags = _IN.get(dt)
    if flags is None:
        raise TypeError(f"unsupported dtype {dt}")
    rot, n_axes = table.rot_dim, table.n_axes
    if rot > head_dim:
        raise ValueError(f"the table turns {rot} elements of heads of {head_dim}")
    hq = qs = hk = ks = qos = kos = 0
    if q is not None:
        hq, qs = _heads("q", q, head_dim)
    if k is not None:
        hk, ks = _heads("k", k, head_dim)
        if q is not None and (k.shape[0] != T or k.dtype != dt or k.get_device() != index):
            raise ValueError("q and k need the same tokens, dtype and device")
    shape, pstride = positions.shape, positions.stride()
    if len(shape) == 2:
        if shape[0] != n_axes or shape[1] != T:
            raise ValueError(f"positions must be [{n_axes}, {T}], got {tuple(shape)}")
    elif len(shape) != 1 or n_axes != 1 or shape[0] != T:
        raise ValueError(f"positions must be [{n_axes}, {T}], got {tuple(shape)}")
    pdt = positions.dtype
    if pdt is torch.int64:
        flags |= _al.RMSATTN_POS_I64
    elif pdt is not torch.int32:
        raise TypeError(f"positions must be int32 or int64, got {pdt}")
    if T > 1 and pstride[-1] != 1:
        raise ValueError("positions of an axis must be contiguous")
    if index < 0:
        raise ValueError("q / k must be CUDA tensors")
    if positions.get_device() != index or table.index != index:
        raise ValueError(f"positions and table must be on {ref.device}")
    if eps is None:
        if q_weight is not None or k_weight is not None:
            raise ValueError("weights need the norm's eps")
        eps = 0.0
    else:
        flags |= _al.RMSATTN_NORM
        for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
            if w is not None and (w.dtype != dt or w.dim() != 1 or w.shape[0] != head_dim
                                  or w.get_device() != index or (head_dim > 1 and w.stride(0) != 1)):
                raise ValueError(f"{name} must be a contiguous [{head_dim}] {dt} on {ref.device}")
    if interleaved:
        flags |= _al.RMSATTN_INTERLEAVED
    if pdl:
        flags |= _lib.RMSN_PDL
    if stream is not None or index != torch._C._cuda_getDevice():
        with _other(ref.device, stream) as (_, keep):
            new_q, new_k = q is not None and q_out is None, k is not None and k_out is None
            q_out, k_out = qk_norm_rope(q, k, positions, table, q_weight, k_weight,
                                        head_dim=head_dim, eps=eps if flags & _al.RMSATTN_NORM else None,
                                        weight_offset=weight_offset, interleaved=interleaved,
                                        q_out=q_out, k_out=k_out, pdl=pdl)
            for t in (q_out if new_q else None, k_out if new_k else None):
                if t is not None and keep is not None:
                    keep(t)
        return q_out, k_out
    if q is not None:
        if q_out is None:
            q_out, qos = torch.empty(q.shape, dtype=dt, device=ref.device), hq * head_dim
        else:
            qos = _heads("q_out", _like("q_out", q_out, q, dt, index), head_dim)[1]
    if k is not None:
        if k_out is None:
            k_out, kos = torch.empty(k.shape, dtype=dt, device=ref.device), hk * head_dim
        else:
            kos = _heads("k_out", _like("k_out", k_out, k, dt, index), head_dim)[1]
    st = _al.load_attn().rmsattn_qk_rope_fwd(
        None if q is None else q.data_ptr(), None if k is None else k.data_ptr(),
        None if q_weight is None else q_weight.data_ptr(),
        None if k_weight is None else k_weight.data_ptr(),
        None if q is None else q_out.data_ptr(), None if k is None else k_out.data_ptr(),
        positions.data_ptr(), pstride[0] if n_axes > 1 else T, *table._pointers(), T,
        hq, hk, head_dim, rot, n_axes, qs, ks, qos, kos, eps, weight_offset, flags,
        _raw_stream(index))
    if st:
        raise _lib.RmsnError(st, "rmsattn_qk_rope_fwd")
    return q_out, k_out


class KVCache(_Fixed):
    """A paged cache of keys and values in E4M3 codes with one fp32 scale for
    every block of 16 tokens and head (``rmsattn_cache``): k and v are
    [n_pages, n_kv_heads, page_size, head_dim] uint8 (or float8_e4m3fn), the
    scales [n_pages, n_kv_heads, page_size / 16]; a token's value is code *
    scale.  The tensors are the caller's; pages may be strided (all layers of
    a model in one tensor), the rest of each tensor is contiguous.  The
    attributes are fixed; a tensor that was given other memory in place
    (``resize_`` of its storage, ``set_``) is looked at again by the next call."""

    _fixed = __slots__ = ("k", "v", "k_scale", "v_scale", "n_pages", "n_kv_heads", "page_size",
                          "head_dim", "device", "index", "_c", "_ref", "_addr", "_tensors")

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor,
                 v_scale: torch.Tensor):
        c = self._described(k, v, k_scale, v_scale)
        self._set(k=k, v=v, k_scale=k_scale, v_scale=v_scale, n_pages=c.n_pages,
                  n_kv_heads=c.n_kv_heads, page_size=c.page_size, head_dim=c.head_dim, device=k.device,
                  index=k.get_device(), _c=c, _ref=ctypes.byref(c), _addr=ctypes.addressof(c),
                  _tensors=(k, v, k_scale, v_scale))

    @staticmethod
    def _described(k, v, k_scale, v_scale):
        """The C ABI's description of the tensors, checked."""
        if k.dim() != 4:
            raise ValueError("k must be [n_pages, n_kv_heads, page_size, head_dim]")
        pages, heads, page, dim = k.shape
        if page % _al.RMSATTN_BLOCK or not page:
            raise ValueError(f"page_size must be a multiple of {_al.RMSATTN_BLOCK}, got {page}")
        if heads < 1 or dim < 1:
            raise ValueError(f"a cache needs heads and a head_dim, got {heads} of {dim}")
        shape = (pages, heads, page // _al.RMSATTN_BLOCK)
        for name, t, want, dtypes in (("k", k, k.shape, _CODES), ("v", v, k.shape, _CODES),
                                      ("k_scale", k_scale, shape, (torch.float32,)),
                                      ("v_scale", v_scale, shape, (torch.float32,))):
            if tuple(t.shape) != tuple(want):
                raise ValueError(f"{name} must have shape {tuple(want)}, got {tuple(t.shape)}")
            if t.dtype not in dtypes:
                raise TypeError(f"{name} must be one of {[str(d) for d in dtypes]}, got {t.dtype}")
            if t.device != k.device:
                raise ValueError(f"{name} must be on {k.device}, got {t.device}")
            # each page contiguous; pages any stride apart
            inner = 1
            for size, step in zip(want[:0:-1], t.stride()[:0:-1]):
                if size > 1 and step != inner:
                    break
                inner *= size
            else:
                end = t.storage_offset() + (pages - 1) * t.stride(0) + inner
                if pages and end * t.element_size() > t.untyped_storage().nbytes():
                    raise ValueError(f"{name} is larger than its storage")
                continue
            if pages:
                raise ValueError(f"{name}: each page must be contiguous")
        if pages > 1 and (k.stride(0) != v.stride(0) or k_scale.stride(0) != v_scale.stride(0)):
            raise ValueError("k and v need the same page stride, and so do their scales")
        return _al.RmsattnCache(
            k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), pages,
            k.stride(0) if pages > 1 else heads * page * dim,
            k_scale.stride(0) if pages > 1 else shape[1] * shape[2], heads, page, dim, 0)

    def __reduce__(self):
        return type(self), self._tensors

    def _current(self):
        """The description as the C ABI takes it, where the tensors lie now."""
        c, at = self._c, tuple(t.data_ptr() for t in self._tensors)
        if at != (c.k or 0, c.v or 0, c.k_scale or 0, c.v_scale or 0):
            now = self._described(*self._tensors)
            if (tuple(self.k.shape) != (self.n_pages, self.n_kv_heads, self.page_size, self.head_dim)
                    or self.k.device != self.device):
                raise ValueError("the cache's tensors have another shape or device than it was made for")
            ctypes.memmove(self._addr, ctypes.addressof(now), ctypes.sizeof(now))
        return self._ref

    @classmethod
    def empty(cls, n_pages: int, n_kv_heads: int, page_size: int, head_dim: int,
              device="cuda") -> "KVCache":
        """A cache of its own, uninitialised: nothing reads a block before its
        first token is appended."""
        codes = (n_pages, n_kv_heads, page_size, head_dim)
        scales = (n_pages, n_kv_heads, page_size // _al.RMSATTN_BLOCK)
        return cls(torch.empty(codes, dtype=torch.uint8, device=device),
                   torch.empty(codes, dtype=torch.uint8, device=device),
                   torch.empty(scales, dtype=torch.float32, device=device),
                   torch.empty(scales, dtype=torch.float32, device=device))


def _check_seqs(cache, block_table, lengths, n_seqs):
    """The table's row stride and width; both tensors as the kernels read them."""
    shape, stride = block_table.shape, block_table.stride()
    if len(shape) != 2 or shape[0] != n_seqs:
        raise ValueError(f"block_table must be [{n_seqs}, pages], got {tuple(shape)}")
    if block_table.dtype is not torch.int32 or lengths.dtype is not torch.int32:
        raise TypeError("block_table and lengths must be int32")
    if lengths.dim() != 1 or lengths.shape[0] != n_seqs:
        raise ValueError(f"lengths must be [{n_seqs}], got {tuple(lengths.shape)}")
    width = shape[1]
    if (width > 1 and stride[1] != 1) or (n_seqs > 1 and lengths.stride(0) != 1):
        raise ValueError("block_table rows and lengths must be contiguous")
    if block_table.get_device() != cache.index or lengths.get_device() != cache.index:
        raise ValueError(f"block_table and lengths must be on {cache.device}")
    return (stride[0] if n_seqs > 1 else width), width


def kv_cache_append_(cache: KVCache, k: torch.Tensor, v: torch.Tensor, block_table: torch.Tensor,
                     lengths: torch.Tensor, cu_seqlens: torch.Tensor | None = None, *,
                     stream: torch.cuda.Stream | None = None, pdl: bool = False) -> KVCache:
    """Append new keys and values to the cache (``rmsattn_kv_append``).

    k and v are [T, n_kv_heads, head_dim] or [T, n_kv_heads * head_dim]
    (column slices of a fused qkv matrix will do) in bf16, fp16 or fp32.
    Sequence s holds ``lengths[s]`` tokens before the call (lengths is not
    changed; a negative one leaves the sequence out) and gets rows
    ``cu_seqlens[s]`` to ``cu_seqlens[s + 1]``; without cu_seqlens, row s.
    ``block_table`` [n_seqs, pages] lists each sequence's pages.  Blocks of 16
    tokens share a scale: where a new token's magnitude exceeds it, the scale
    grows and the block's older codes are re-encoded.
    """
    if stream is None and (_al._fast or _al.load_fast()).kv_append(
            k, v, cache._addr, cache._tensors, cache.index, block_table, lengths, cu_seqlens, pdl):
        return cache
    hk, ks = _heads("k", k, cache.head_dim)
    hv, vs = _heads("v", v, cache.head_dim)
    T, dt, index = k.shape[0], k.dtype, cache.index
    if hk != cache.n_kv_heads or hv != hk:
        raise ValueError(f"k and v must hold {cache.n_kv_heads} heads")
    if v.shape[0] != T or v.dtype != dt:
        raise ValueError("k and v need the same tokens and dtype")
    flags = _IN.get(dt)
    if flags is None:
        raise TypeError(f"unsupported dtype {dt}")
    n = lengths.shape[0] if lengths.dim() == 1 else 0
    stride, width = _check_seqs(cache, block_table, lengths, n)
    if cu_seqlens is None:
        if T != n:
            raise ValueError(f"without cu_seqlens, k must have one row for each of {n} sequences")
    elif (cu_seqlens.dtype is not torch.int32 or cu_seqlens.dim() != 1
          or cu_seqlens.shape[0] != n + 1 or cu_seqlens.get_device() != index
          or (n and cu_seqlens.stride(0) != 1)):
        _check("cu_seqlens", cu_seqlens, (n + 1,), (torch.int32,), cache.device)
    if index < 0 or k.get_device() != index or v.get_device() != index:
        raise ValueError(f"k and v must be on the cache's CUDA device, {cache.device}")
    if stream is not None or index != torch._C._cuda_getDevice():
        with _other(cache.device, stream):
            return kv_cache_append_(cache, k, v, block_table, lengths, cu_seqlens, pdl=pdl)
    st = _al.load_attn().rmsattn_kv_append(
        cache._current(), k.data_ptr(), v.data_ptr(), ks, vs, block_table.data_ptr(), stride, width,
        lengths.data_ptr(), None if cu_seqlens is None else cu_seqlens.data_ptr(), T, n,
        flags | _lib.RMSN_PDL if pdl else flags, _raw_stream(index))
    if st:
        raise _lib.RmsnError(st, "rmsattn_kv_append")
    return cache


def _token_stride(name, t, n):
    """Elements between the tokens of [n_seqs, heads, head_dim] (n = 1) or
    [n_seqs, n, heads, head_dim], which must be evenly spaced with their heads
    back to back."""
    shape, stride = t.shape, t.stride()
    H, D = shape[-2], shape[-1]
    if stride[-1] != 1 or (H > 1 and stride[-2] != D):
        raise ValueError(f"{name}: a token's heads must lie back to back")
    if n > 1:
        if shape[0] > 1 and stride[0] != n * stride[1]:
            raise ValueError(f"{name}: the tokens must be evenly spaced")
        return stride[1]
    return stride[0] if shape[0] > 1 else H * D


def kv_cache_attention(q: torch.Tensor, cache: KVCache, block_table: torch.Tensor,
                       lengths: torch.Tensor, *, scale: float | None = None, window: int = 0,
                       sinks: int = 0, out: torch.Tensor | None = None,
                       stream: torch.cuda.Stream | None = None, pdl: bool = False) -> torch.Tensor:
    """Attention of one or a few query tokens per sequence over the cache
    (``rmsattn_kv_attention``).

    q is [n_seqs, Hq, head_dim], or [n_seqs, n, Hq, head_dim] for n query
    tokens a sequence (up to 32), bf16 or fp16, Hq a multiple of the cache's
    heads.  ``lengths`` counts each sequence's tokens in the cache, the
    queries' own among them; query i stands at position lengths - n + i and
    sees the tokens up to its own; with ``window``, of those only the last
    ``window`` and the sequence's first ``sinks``.  A query that sees nothing
    (length 0, a padded row) gives 0.  ``scale``: default 1 / sqrt(head_dim).
    Returns out, shaped like q.
    """
    if stream is None:
        done = (_al._fast or _al.load_fast()).kv_attention(
            q, cache._addr, cache._tensors, cache.index, block_table, lengths, scale, window, sinks, out, pdl)
        if done is not None:
            return done
    shape, dt, index = q.shape, q.dtype, cache.index
    if len(shape) == 3:
        B, H, D = shape
        n = 1
    elif len(shape) == 4:
        B, n, H, D = shape
    else:
        raise ValueError("q must be [n_seqs, heads, head_dim] or [n_seqs, n, heads, head_dim]")
    Hk = cache.n_kv_heads
    if D != cache.head_dim or H < 1 or H % Hk:
        raise ValueError(f"q must hold a multiple of {Hk} heads of {cache.head_dim}")
    if not 1 <= n <= _al.RMSATTN_MAX_QUERIES:
        raise ValueError(f"1 to {_al.RMSATTN_MAX_QUERIES} query tokens a sequence, got {n}")
    if dt is not torch.bfloat16 and dt is not torch.float16:
        raise TypeError(f"q must be bfloat16 or float16, got {dt}")
    if window < 0 or sinks < 0:
        raise ValueError("window and sinks must not be negative")
    # the C ABI's int64 would wrap; no table holds so many tokens
    window, sinks = min(window, 2**62), min(sinks, 2**62)
    stride, width = _check_seqs(cache, block_table, lengths, B)
    if index < 0 or q.get_device() != index:
        raise ValueError(f"q must be on the cache's CUDA device, {cache.device}")
    if stream is not None or index != torch._C._cuda_getDevice():
        with _other(cache.device, stream) as (_, keep):
            new = out is None
            out = kv_cache_attention(q, cache, block_table, lengths, scale=scale, window=window,
                                     sinks=sinks, out=out, pdl=pdl)
            if new and keep is not None:
                keep(out)
        return out
    qs = _token_stride("q", q, n)
    lib = _al.load_attn()
    if out is None:
        out, os = torch.empty(shape, dtype=dt, device=cache.device), H * D
    else:
        if out.shape != shape or out.dtype != dt or out.get_device() != index:
            raise ValueError("out must be like q")
        os = _token_stride("out", out, n)
    need = lib.rmsattn_kv_attention_workspace(B, n, H, Hk, D, width * cache.page_size, window, sinks)
    if need < 0:
        raise _lib.RmsnError(need, "rmsattn_kv_attention_workspace")
    # freed when this returns: the allocator hands it to later work of the
    # same stream only, which runs behind the kernels
    ws = torch.empty(need, dtype=torch.uint8, device=cache.device) if need else None
    flags = _IN[dt]
    st = lib.rmsattn_kv_attention(
        q.data_ptr(), cache._current(), block_table.data_ptr(), stride, width, lengths.data_ptr(),
        out.data_ptr(), qs, os, B, n, H, 1.0 / math.sqrt(D) if scale is None else scale, window,
        sinks, ws.data_ptr() if need else None, need, flags | _lib.RMSN_PDL if pdl else flags, _raw_stream(index))
    if st:
        raise _lib.RmsnError(st, "rmsattn_kv_attention")
    return out
