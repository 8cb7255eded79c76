"""Tensor-level entry points of the attention path over the C ABI of
include/rmsnorm_attn.h (marshalling only): QK norm with multi-axis rotary
positions, the append to a paged E4M3 cache, and the attention over it.
Nothing here computes: a failed call raises ``RmsnError``.
"""
from __future__ import annotations

import contextlib
import ctypes
import math

import torch

from . import _attn_lib as _al
from . import _lib
from .api import _IN, _check

_CODES = (torch.uint8, torch.float8_e4m3fn)


def _on(device, stream):
    """(cudaStream_t, stream to enter or None, caller's stream) of a call on
    `device`: outputs and workspaces are allocated, and the launch made, with
    that device and stream current."""
    caller = torch.cuda.current_stream(device)
    if stream is None:
        if device.index == torch.cuda.current_device():
            return caller.cuda_stream, None, caller
        stream = caller
    elif stream.device != device:
        raise ValueError(f"stream must be on {device}, got {stream.device}")
    return stream.cuda_stream, stream, caller


def _enter(s):
    return contextlib.nullcontext() if s is None else torch.cuda.stream(s)


def _new(shape, dtype, device, s, caller):
    """An output of a call on stream s (None: the caller's own): its memory
    comes from that stream's pool, and is not handed on while the caller's
    stream still works on it."""
    t = torch.empty(shape, dtype=dtype, device=device)
    if s is not None and s != caller:
        t.record_stream(caller)
    return t


class RopeTable:
    """Frequencies of the rotary pairs: ``turns`` (int64 bit patterns of 64-bit
    fractions of a turn per position), ``axis`` (int32, the axis whose position
    turns the pair), both [rot_dim / 2] on the device; made by ``rope_table``."""

    __slots__ = ("turns", "axis", "rot_dim", "n_axes")

    def __init__(self, turns: torch.Tensor, axis: torch.Tensor, n_axes: int):
        if turns.dim() != 1:
            raise ValueError("turns must be [rot_dim / 2]")
        _check("turns", turns, (turns.numel(),), (torch.int64,))
        _check("axis", axis, (turns.numel(),), (torch.int32,), turns.device)
        self.turns, self.axis = turns, axis
        self.rot_dim, self.n_axes = 2 * turns.numel(), int(n_axes)


def rope_table(rot_dim: int, *, base: float = 10000.0, sections=None, axis=None, inv_freq=None,
               device="cuda") -> RopeTable:
    """Table of ``rot_dim / 2`` rotary pairs.

    Pair p turns by ``inv_freq[p]`` radians per position, by default
    ``base ** (-2 p / rot_dim)``.  ``sections`` gives consecutive pairs to the
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
        if not base > 0:
            raise ValueError("base must be positive")
        freqs = [float(base) ** (-2.0 * p / rot_dim) for p in range(pairs)]
    else:
        freqs = [float(f) for f in inv_freq]
        if len(freqs) != pairs:
            raise ValueError(f"inv_freq must hold {pairs} values")
    if not all(math.isfinite(f) for f in freqs):
        raise ValueError("frequencies must be finite")
    bits = [int(math.ldexp(f / (2.0 * math.pi), 64)) % 2**64 for f in freqs]
    bits = [b - 2**64 if b >= 2**63 else b for b in bits]
    return RopeTable(torch.tensor(bits, dtype=torch.int64, device=device),
                     torch.tensor(axes, dtype=torch.int32, device=device), n_axes)


def _heads(name, t, head_dim):
    """(heads, token stride) of [T, H * head_dim] or [T, H, head_dim] with the
    heads of a token back to back."""
    if t.dim() == 2:
        width = t.shape[1]
        if width % head_dim:
            raise ValueError(f"{name}: rows must hold whole heads of head_dim elements")
        ok = t.stride(1) == 1 or width == 1
    elif t.dim() == 3:
        if t.shape[2] != head_dim:
            raise ValueError(f"{name}: rows must hold whole heads of head_dim elements")
        width = t.shape[1] * head_dim
        ok = (t.stride(2) == 1 or head_dim == 1) and (t.stride(1) == head_dim or t.shape[1] <= 1)
    else:
        raise ValueError(f"{name} must be [T, heads * head_dim] or [T, heads, head_dim]")
    if not ok:
        raise ValueError(f"{name}: a token's heads must lie back to back")
    return width // head_dim, (t.stride(0) if t.shape[0] > 1 else width)


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
    for a table of one axis, else [n_axes, T], int32 or int64.  ``eps``: the
    norm's; None leaves the norm (and the weights) out.  ``interleaved``:
    pairs are neighbouring elements, else halves of the first rot_dim.  The
    results go to q_out / k_out (new tensors where None; pass q and k
    themselves to work in place).  Returns ``(q_out, k_out)``.
    """
    ref = q if q is not None else k
    if ref is None:
        return q_out, k_out
    if head_dim < 1:
        raise ValueError("head_dim must be positive")
    dt, dev, T = ref.dtype, ref.device, ref.shape[0]
    if dt not in _IN:
        raise TypeError(f"unsupported dtype {dt}")
    if table.rot_dim > head_dim:
        raise ValueError(f"the table turns {table.rot_dim} elements of heads of {head_dim}")
    hq = qs = hk = ks = 0
    if q is not None:
        hq, qs = _heads("q", q, head_dim)
    if k is not None:
        hk, ks = _heads("k", k, head_dim)
        if q is not None and (k.shape[0] != T or k.dtype != dt or k.device != dev):
            raise ValueError("q and k need the same tokens, dtype and device")
    if positions.dim() == 1 and table.n_axes == 1:
        positions = positions[None]
    if tuple(positions.shape) != (table.n_axes, T):
        raise ValueError(f"positions must be [{table.n_axes}, {T}], got {tuple(positions.shape)}")
    if positions.dtype not in (torch.int32, torch.int64):
        raise TypeError(f"positions must be int32 or int64, got {positions.dtype}")
    if T > 1 and positions.stride(1) != 1:
        raise ValueError("positions of an axis must be contiguous")
    if not ref.is_cuda:
        raise ValueError("q / k must be CUDA tensors")
    if positions.device != dev or table.turns.device != dev:
        raise ValueError(f"positions and table must be on {dev}")
    flags = _IN[dt]
    if eps is None:
        if q_weight is not None or k_weight is not None:
            raise ValueError("weights need the norm's eps")
    else:
        flags |= _al.RMSATTN_NORM
        if q_weight is not None:
            _check("q_weight", q_weight, (head_dim,), (dt,), dev)
        if k_weight is not None:
            _check("k_weight", k_weight, (head_dim,), (dt,), dev)
    if interleaved:
        flags |= _al.RMSATTN_INTERLEAVED
    if positions.dtype == torch.int64:
        flags |= _al.RMSATTN_POS_I64
    if pdl:
        flags |= _lib.RMSN_PDL
    handle, s, caller = _on(dev, stream)
    with _enter(s):
        qos = kos = 0
        if q is not None:
            if q_out is None:
                q_out = _new(q.shape, dt, dev, s, caller)
            elif q_out.shape != q.shape or q_out.dtype != dt or q_out.device != dev:
                raise ValueError("q_out must be like q")
            qos = _heads("q_out", q_out, head_dim)[1]
        if k is not None:
            if k_out is None:
                k_out = _new(k.shape, dt, dev, s, caller)
            elif k_out.shape != k.shape or k_out.dtype != dt or k_out.device != dev:
                raise ValueError("k_out must be like k")
            kos = _heads("k_out", k_out, head_dim)[1]
        st = _al.load_attn().rmsattn_qk_rope_fwd(
            q.data_ptr() if q is not None else None, k.data_ptr() if k is not None else None,
            None if q_weight is None else q_weight.data_ptr(),
            None if k_weight is None else k_weight.data_ptr(),
            q_out.data_ptr() if q is not None else None,
            k_out.data_ptr() if k is not None else None,
            positions.data_ptr(), positions.stride(0) if table.n_axes > 1 else T,
            table.turns.data_ptr(), table.axis.data_ptr(), T, hq, hk, head_dim, table.rot_dim,
            table.n_axes, qs, ks, qos, kos, 0.0 if eps is None else eps, weight_offset, flags,
            handle)
    if st != _lib.RMSN_OK:
        raise _lib.RmsnError(st, "rmsattn_qk_rope_fwd")
    return q_out, k_out


class KVCache:
    """A paged cache of keys and values in E4M3 codes with one fp32 scale for
    every block of 16 tokens and head (``rmsattn_cache``): k and v are
    [n_pages, n_kv_heads, page_size, head_dim] uint8 (or float8_e4m3fn), the
    scales [n_pages, n_kv_heads, page_size / 16]; a token's value is code *
    scale.  The tensors are the caller's; pages may be strided (all layers of
    a model in one tensor), the rest of each tensor is contiguous."""

    __slots__ = ("k", "v", "k_scale", "v_scale", "n_pages", "n_kv_heads", "page_size", "head_dim",
                 "device", "_c")

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor,
                 v_scale: torch.Tensor):
        if k.dim() != 4:
            raise ValueError("k must be [n_pages, n_kv_heads, page_size, head_dim]")
        pages, heads, page, dim = k.shape
        if page % _al.RMSATTN_BLOCK or not page:
            raise ValueError(f"page_size must be a multiple of {_al.RMSATTN_BLOCK}, got {page}")
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
            if pages and not t[0].is_contiguous():
                raise ValueError(f"{name}: each page must be contiguous")
        if pages > 1 and (k.stride(0) != v.stride(0) or k_scale.stride(0) != v_scale.stride(0)):
            raise ValueError("k and v need the same page stride, and so do their scales")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.n_pages, self.n_kv_heads, self.page_size, self.head_dim = pages, heads, page, dim
        self.device = k.device
        self._c = _al.RmsattnCache(
            k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), pages,
            k.stride(0) if pages > 1 else heads * page * dim,
            k_scale.stride(0) if pages > 1 else shape[1] * shape[2], heads, page, dim, 0)

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
    if block_table.dim() != 2 or block_table.shape[0] != n_seqs:
        raise ValueError(f"block_table must be [{n_seqs}, pages], got {tuple(block_table.shape)}")
    if block_table.dtype != torch.int32 or lengths.dtype != torch.int32:
        raise TypeError("block_table and lengths must be int32")
    if lengths.dim() != 1 or lengths.shape[0] != n_seqs:
        raise ValueError(f"lengths must be [{n_seqs}], got {tuple(lengths.shape)}")
    if ((block_table.shape[1] > 1 and block_table.stride(1) != 1)
            or (n_seqs > 1 and lengths.stride(0) != 1)):
        raise ValueError("block_table rows and lengths must be contiguous")
    if block_table.device != cache.device or lengths.device != cache.device:
        raise ValueError(f"block_table and lengths must be on {cache.device}")


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
    hk, ks = _heads("k", k, cache.head_dim)
    hv, vs = _heads("v", v, cache.head_dim)
    T = k.shape[0]
    if hk != cache.n_kv_heads or hv != cache.n_kv_heads:
        raise ValueError(f"k and v must hold {cache.n_kv_heads} heads")
    if v.shape[0] != T or k.dtype != v.dtype:
        raise ValueError("k and v need the same tokens and dtype")
    if k.dtype not in _IN:
        raise TypeError(f"unsupported dtype {k.dtype}")
    _check_seqs(cache, block_table, lengths, lengths.shape[0] if lengths.dim() else 0)
    n = lengths.shape[0]
    if cu_seqlens is None:
        if T != n:
            raise ValueError(f"without cu_seqlens, k must have one row for each of {n} sequences")
    else:
        _check("cu_seqlens", cu_seqlens, (n + 1,), (torch.int32,), cache.device)
    if not k.is_cuda or k.device != cache.device or v.device != cache.device:
        raise ValueError(f"k and v must be on the cache's CUDA device {cache.device}")
    handle, s, caller = _on(cache.device, stream)
    with _enter(s):
        st = _al.load_attn().rmsattn_kv_append(
            ctypes.byref(cache._c), k.data_ptr(), v.data_ptr(), ks, vs, block_table.data_ptr(),
            block_table.stride(0) if n > 1 else block_table.shape[1], block_table.shape[1],
            lengths.data_ptr(), None if cu_seqlens is None else cu_seqlens.data_ptr(), T, n,
            _IN[k.dtype] | (_lib.RMSN_PDL if pdl else 0), handle)
    if st != _lib.RMSN_OK:
        raise _lib.RmsnError(st, "rmsattn_kv_append")
    return cache


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
    if q.dim() == 3:
        q4 = q.unsqueeze(1)
    elif q.dim() == 4:
        q4 = q
    else:
        raise ValueError("q must be [n_seqs, heads, head_dim] or [n_seqs, n, heads, head_dim]")
    B, n, H, D = q4.shape
    if D != cache.head_dim or H < 1 or H % cache.n_kv_heads:
        raise ValueError(f"q must hold a multiple of {cache.n_kv_heads} heads of {cache.head_dim}")
    if not 1 <= n <= _al.RMSATTN_MAX_QUERIES:
        raise ValueError(f"1 to {_al.RMSATTN_MAX_QUERIES} query tokens a sequence, got {n}")
    if q.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError(f"q must be bfloat16 or float16, got {q.dtype}")
    if window < 0 or sinks < 0:
        raise ValueError("window and sinks must not be negative")
    _check_seqs(cache, block_table, lengths, B)
    if not q.is_cuda or q.device != cache.device:
        raise ValueError(f"q must be on the cache's CUDA device {cache.device}")
    qs = _token_stride("q", q4)
    lib = _al.load_attn()
    handle, s, caller = _on(cache.device, stream)
    with _enter(s):
        if out is None:
            out = _new(q.shape, q.dtype, q.device, s, caller)
            os = H * D
        else:
            if out.shape != q.shape or out.dtype != q.dtype or out.device != q.device:
                raise ValueError("out must be like q")
            os = _token_stride("out", out if q.dim() == 4 else out.unsqueeze(1))
        need = lib.rmsattn_kv_attention_workspace(B, n, H, cache.n_kv_heads, D)
        if need < 0:
            raise _lib.RmsnError(need, "rmsattn_kv_attention_workspace")
        # freed when this returns: the allocator hands it to later work of the
        # same stream only, which runs behind the kernels
        ws = torch.empty(need, dtype=torch.uint8, device=q.device) if need else None
        st = lib.rmsattn_kv_attention(
            q.data_ptr(), ctypes.byref(cache._c), block_table.data_ptr(),
            block_table.stride(0) if B > 1 else block_table.shape[1], block_table.shape[1],
            lengths.data_ptr(), out.data_ptr(), qs, os, B, n, H,
            1.0 / math.sqrt(D) if scale is None else scale, window, sinks,
            None if ws is None else ws.data_ptr(), need,
            _IN[q.dtype] | (_lib.RMSN_PDL if pdl else 0), handle)
    if st != _lib.RMSN_OK:
        raise _lib.RmsnError(st, "rmsattn_kv_attention")
    return out


def _token_stride(name, t):
    """Elements between the tokens of [n_seqs, n, heads, head_dim], which must
    be evenly spaced with their heads back to back."""
    B, n, H, D = t.shape
    if t.stride(3) != 1 or (H > 1 and t.stride(2) != D):
        raise ValueError(f"{name}: a token's heads must lie back to back")
    if n > 1:
        step = t.stride(1)
        if B > 1 and t.stride(0) != n * step:
            raise ValueError(f"{name}: the tokens must be evenly spaced")
        return step
    return t.stride(0) if B > 1 else H * D
