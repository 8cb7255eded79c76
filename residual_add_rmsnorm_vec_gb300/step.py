"""Tensor-level entry points of the operators around the attention in a serving
step, over the C ABI of include/rmsnorm_attn.h (marshalling only): the step's
page plan, attention with a shared prefix, and the norms at a block's end.
Nothing here computes: a failed call raises ``RmsnError``.

As in attn.py, the usual call is marshalled natively (binding/attn_fast.cpp),
and what that does not take comes back here.
"""
from __future__ import annotations

import math
from typing import NamedTuple

import torch

from . import _attn_lib as _al
from . import _lib
from .api import _IN, _check
from .attn import KVCache, _check_seqs, _other, _raw_stream, _token_stride


class KVStep(NamedTuple):
    """What ``kv_pages_step_`` plans: ``cu_seqlens`` and ``before`` go to
    ``kv_cache_append_``, ``positions`` to ``qk_norm_rope``, ``after`` to the
    attention (and into the next step as its lengths), ``rows`` to
    ``fused_block_norms`` (a gate row for each sequence), ``slots`` are the rows'
    places in the cache, ``n_free`` the next step's free pages.  They may share one
    allocation."""
    cu_seqlens: torch.Tensor
    positions: torch.Tensor
    slots: torch.Tensor
    rows: torch.Tensor
    before: torch.Tensor
    after: torch.Tensor
    n_free: torch.Tensor


def kv_free_pages(n_pages: int, device="cuda"):
    """(free_pages, n_free) of a cache whose ``n_pages`` pages are all free: they
    are taken from the end of free_pages, page 0 first."""
    if n_pages < 0:
        raise ValueError("n_pages must not be negative")
    return (torch.arange(n_pages - 1, -1, -1, dtype=torch.int32, device=device),
            torch.full((1,), n_pages, dtype=torch.int32, device=device))


def _other_call(device, stream, call):
    """call() with device and stream current; its new tensors are held back from
    other streams' use while the caller's stream still works on them."""
    with _other(device, stream) as (_, keep):
        made, result = call()
        if keep is not None:
            for t in made:
                keep(t)
    return result


def kv_pages_step_(free_pages: torch.Tensor, n_free: torch.Tensor, block_table: torch.Tensor,
                   lengths: torch.Tensor, new_tokens: torch.Tensor, shared_pages: torch.Tensor | None = None, *,
                   page_size: int, n_rows: int, stream: torch.cuda.Stream | None = None,
                   pdl: bool = False) -> KVStep:
    """Plan a serving step from the requests' lengths (``rmsattn_pages_step``).

    Sequence s holds ``lengths[s]`` tokens and gets ``new_tokens[s]`` more, the
    next rows of the step's batch of ``n_rows``.  A negative ``new_tokens[s]``
    says that it is finished: its pages, from ``shared_pages[s]`` on, go back to
    the free ones (``free_pages``, of which the first ``n_free`` count).  Growing
    sequences take new pages from the end of the free ones into their row of
    ``block_table``.  A sequence for which pages, columns or rows are missing is
    left out: ``before`` is -1 and ``after`` its length as it was.  All tensors
    are int32; block_table and free_pages are changed in place, lengths and
    n_free are not: go on with the result's ``after`` and ``n_free``.
    """
    if stream is None:
        done = (_al._fast or _al.load_fast()).pages_step(
            free_pages, n_free, block_table, lengths, new_tokens, shared_pages, page_size, n_rows, pdl)
        if done is not None:
            return KVStep._make(done)
    device, i32 = free_pages.device, (torch.int32,)
    if free_pages.dim() != 1:
        raise ValueError("free_pages must be [n_pages]")
    if lengths.dim() != 1:
        raise ValueError("lengths must be [n_seqs]")
    n = lengths.shape[0]
    _check("free_pages", free_pages, free_pages.shape, i32)
    _check("n_free", n_free, (1,), i32, device)
    _check("lengths", lengths, (n,), i32, device)
    _check("new_tokens", new_tokens, (n,), i32, device)
    _check("shared_pages", shared_pages, (n,), i32, device)
    if block_table.dim() != 2 or block_table.shape[0] != n or block_table.dtype is not torch.int32:
        raise ValueError(f"block_table must be int32 [{n}, pages], got {block_table.dtype} {tuple(block_table.shape)}")
    if block_table.device != device or device.type != "cuda":
        raise ValueError("free_pages and block_table must be on one CUDA device")
    width = block_table.shape[1]
    if width > 1 and block_table.stride(1) != 1:
        raise ValueError("block_table rows must be contiguous")
    if page_size < _al.RMSATTN_BLOCK or page_size % _al.RMSATTN_BLOCK:
        raise ValueError(f"page_size must be a multiple of {_al.RMSATTN_BLOCK}, got {page_size}")
    if not 0 <= n_rows <= 1 << 29:
        raise ValueError(f"n_rows must be within [0, 2^29], got {n_rows}")
    if stream is not None or free_pages.get_device() != torch._C._cuda_getDevice():
        def call():
            step = kv_pages_step_(free_pages, n_free, block_table, lengths, new_tokens, shared_pages,
                                  page_size=page_size, n_rows=n_rows, pdl=pdl)
            return step, step
        return _other_call(device, stream, call)

    def new(size, dtype=torch.int32):
        return torch.empty(size, dtype=dtype, device=device)

    step = KVStep(new(n + 1), new(n_rows), new(n_rows, torch.int64), new(n_rows), new(n), new(n), new(1))
    lib = _al.load_attn()
    need = lib.rmsattn_pages_workspace(n)
    if need < 0:
        raise _lib.RmsnError(need, "rmsattn_pages_workspace")
    ws = new(need, torch.uint8) if need else None
    st = lib.rmsattn_pages_step(
        free_pages.data_ptr(), free_pages.shape[0], n_free.data_ptr(), block_table.data_ptr(),
        block_table.stride(0) if n > 1 else width, width, lengths.data_ptr(), new_tokens.data_ptr(),
        None if shared_pages is None else shared_pages.data_ptr(), n, page_size, n_rows,
        *(t.data_ptr() for t in step), ws.data_ptr() if need else None, need, _lib.RMSN_PDL if pdl else 0,
        _raw_stream(free_pages.get_device()))
    if st:
        raise _lib.RmsnError(st, "rmsattn_pages_step")
    return step


def kv_cache_prefix_attention(q: torch.Tensor, cache: KVCache, block_table: torch.Tensor, lengths: torch.Tensor,
                              prefix_lengths: torch.Tensor, groups: torch.Tensor | None = None, *,
                              scale: float | None = None, out: torch.Tensor | None = None,
                              stream: torch.cuda.Stream | None = None, pdl: bool = False) -> torch.Tensor:
    """Attention of one or a few query tokens per sequence over the cache, where
    groups of sequences share a long prefix (``rmsattn_kv_prefix_attention``).

    As ``kv_cache_attention`` (q, cache, block_table, lengths, scale, out), and
    the same result, but what a group shares is read once: group g, the sequences
    ``groups[g]`` to ``groups[g + 1] - 1`` (``groups`` int32 [n_groups + 1]; None:
    one group of all), has the same first ``prefix_lengths[g]`` tokens, in the
    same pages.  ``lengths`` and the rows of ``block_table`` count those too.  A
    sequence that does not see all of the prefix reads its own row alone.

    It takes some 25 us at the least: ``kv_cache_attention`` with the same arguments is
    the faster one up to about 200 MB of keys and values over all sequences' lengths
    (300 MB at head_dim 256).
    """
    if stream is None:
        done = (_al._fast or _al.load_fast()).kv_prefix_attention(
            q, cache._addr, cache._tensors, cache.index, block_table, lengths, prefix_lengths, groups, scale, out,
            pdl)
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
    stride, width = _check_seqs(cache, block_table, lengths, B)
    if index < 0 or q.get_device() != index:
        raise ValueError(f"q must be on the cache's CUDA device, {cache.device}")
    if prefix_lengths.dim() != 1:
        raise ValueError("prefix_lengths must be [n_groups]")
    n_groups = prefix_lengths.shape[0]
    _check("prefix_lengths", prefix_lengths, (n_groups,), (torch.int32,), cache.device)
    if groups is None:
        if n_groups != 1:
            raise ValueError(f"without groups, prefix_lengths must hold one length, got {n_groups}")
    else:
        _check("groups", groups, (n_groups + 1,), (torch.int32,), cache.device)
    if stream is not None or index != torch._C._cuda_getDevice():
        def call():
            o = kv_cache_prefix_attention(q, cache, block_table, lengths, prefix_lengths, groups, scale=scale,
                                          out=out, pdl=pdl)
            return [o] if out is None else [], o
        return _other_call(cache.device, stream, call)
    qs = _token_stride("q", q, n)
    lib = _al.load_attn()
    if out is None:
        out, os = torch.empty(shape, dtype=dt, device=cache.device), H * D
    else:
        if out.shape != shape or out.dtype != dt or out.get_device() != index:
            raise ValueError("out must be like q")
        os = _token_stride("out", out, n)
    need = lib.rmsattn_kv_prefix_attention_workspace(B, n, H, Hk, D, width * cache.page_size, n_groups)
    if need < 0:
        raise _lib.RmsnError(need, "rmsattn_kv_prefix_attention_workspace")
    # freed when this returns: the allocator hands it to later work of the
    # same stream only, which runs behind the kernels
    ws = torch.empty(need, dtype=torch.uint8, device=cache.device)
    st = lib.rmsattn_kv_prefix_attention(
        q.data_ptr(), cache._current(), block_table.data_ptr(), stride, width, lengths.data_ptr(),
        prefix_lengths.data_ptr(), None if groups is None else groups.data_ptr(), n_groups, out.data_ptr(), qs,
        os, B, n, H, 1.0 / math.sqrt(D) if scale is None else scale, ws.data_ptr(), need,
        _IN[dt] | _lib.RMSN_PDL if pdl else _IN[dt], _raw_stream(index))
    if st:
        raise _lib.RmsnError(st, "rmsattn_kv_prefix_attention")
    return out


def fused_block_norms(x: torch.Tensor, residual: torch.Tensor, post_weight: torch.Tensor | None = None,
                      weight: torch.Tensor | None = None, *, eps: float, gate: torch.Tensor | None = None,
                      gate_index: torch.Tensor | None = None, residual_scale: float = 1.0,
                      weight_offset: float = 0.0, out_dtype: str | None = None,
                      out: torch.Tensor | None = None, residual_out: torch.Tensor | None = None,
                      out_scale: torch.Tensor | None = None, stream: torch.cuda.Stream | None = None,
                      pdl: bool = False):
    """The end of a block and the begin of the next, in one launch
    (``rmsattn_block_norms``): the RMS norm of the block's output x [T, H], its
    gate, the residual update and the RMS norm of the updated residual::

        h   = residual_scale * residual + gate * norm(x, post_weight)
        out = norm(h, weight)

    residual is [T, H] of x's dtype, or fp32 over bf16 / fp16 x; the weights are
    [H] of x's dtype (None: 1), both plus ``weight_offset``.  ``gate``: None (1),
    [H], or rows [T, H]; with ``gate_index`` (int32 [T]) rows [n, H] of which
    token t takes row gate_index[t], and a token with a negative index is left
    out: its row stays as it is in an ``out``, ``residual_out`` or ``out_scale`` that
    is given, and is zeros in one that the call makes.  ``out_dtype``: x's, or
    "fp8" (E4M3 codes as uint8 with a scale for each token).  Returns
    ``(out, residual_out, out_scale)``, out_scale None without fp8.
    """
    if stream is None:
        done = (_al._fast or _al.load_fast()).block_norms(
            x, residual, post_weight, weight, eps, gate, gate_index, residual_scale, weight_offset, out_dtype, out,
            residual_out, out_scale, pdl)
        if done is not None:
            return done
    if x.dim() != 2:
        raise ValueError("x must be [n_tokens, hidden]")
    dt, device = x.dtype, x.device
    flags = _IN.get(dt)
    if flags is None:
        raise TypeError(f"unsupported dtype {dt}")
    if device.type != "cuda":
        raise ValueError("x must be a CUDA tensor")
    if out_dtype not in (None, "fp8", {torch.float32: "f32", torch.bfloat16: "bf16", torch.float16: "f16"}[dt]):
        raise ValueError(f"out_dtype must be x's or 'fp8', got {out_dtype!r}")
    fp8 = out_dtype == "fp8"
    T, H = x.shape
    if residual is None:
        raise ValueError("residual is needed")
    _check("x", x, (T, H), (dt,))
    _check("residual", residual, (T, H), (dt,) if dt is torch.float32 else (dt, torch.float32), device)
    _check("post_weight", post_weight, (H,), (dt,), device)
    _check("weight", weight, (H,), (dt,), device)
    _check("out", out, (T, H), (torch.uint8 if fp8 else dt,), device)
    _check("residual_out", residual_out, (T, H), (residual.dtype,), device)
    if out_scale is not None and not fp8:
        raise ValueError("out_scale is only written for the fp8 output")
    _check("out_scale", out_scale, (T,), (torch.float32,), device)
    n_gates = stride = 0
    if gate is None:
        if gate_index is not None:
            raise ValueError("gate_index needs a gate")
    elif gate.dim() == 1 and gate_index is None:
        _check("gate", gate, (H,), (dt,), device)
        n_gates = 1
    else:
        if gate.dim() != 2 or gate.shape[1] != H or gate.dtype != dt or gate.device != device:
            raise ValueError(f"gate must be [{H}] or rows of {H} elements, {dt} on {device}")
        n_gates = gate.shape[0]
        if gate_index is None and n_gates != T:
            raise ValueError(f"without gate_index, gate must have a row for each of {T} tokens, got {n_gates}")
        if H > 1 and gate.stride(1) != 1:
            raise ValueError("gate rows must be contiguous")
        stride = gate.stride(0) if n_gates > 1 else H
        if stride < H:
            raise ValueError("gate rows must not overlap (pass [H] for one row)")
        _check("gate_index", gate_index, (T,), (torch.int32,), device)
    if residual.dtype != dt:
        flags |= _lib.RMSN_RESIDUAL_F32
    if fp8:
        flags |= _al.RMSATTN_OUT_FP8
    if pdl:
        flags |= _lib.RMSN_PDL
    if stream is not None or x.get_device() != torch._C._cuda_getDevice():
        def call():
            done = fused_block_norms(x, residual, post_weight, weight, eps=eps, gate=gate, gate_index=gate_index,
                                     residual_scale=residual_scale, weight_offset=weight_offset,
                                     out_dtype=out_dtype, out=out, residual_out=residual_out, out_scale=out_scale,
                                     pdl=pdl)
            given = (out, residual_out, out_scale)
            return [t for t, g in zip(done, given) if t is not None and g is None], done
        return _other_call(device, stream, call)
    if gate_index is not None:  # rows that are left out of new outputs
        flags |= _al.RMSATTN_ZERO_OUT if out is None else 0
        flags |= _al.RMSATTN_ZERO_RESIDUAL if residual_out is None else 0
        flags |= _al.RMSATTN_ZERO_SCALE if fp8 and out_scale is None else 0
    if out is None:
        out = torch.empty((T, H), dtype=torch.uint8 if fp8 else dt, device=device)
    if residual_out is None:
        residual_out = torch.empty((T, H), dtype=residual.dtype, device=device)
    if fp8 and out_scale is None:
        out_scale = torch.empty((T,), dtype=torch.float32, device=device)

    def ptr(t):
        return None if t is None else t.data_ptr()

    st = _al.load_attn().rmsattn_block_norms(
        x.data_ptr(), residual.data_ptr(), ptr(post_weight), ptr(weight), ptr(gate), stride, ptr(gate_index),
        n_gates, out.data_ptr(), residual_out.data_ptr(), ptr(out_scale), T, H, eps, residual_scale, weight_offset,
        flags, _raw_stream(x.get_device()))
    if st:
        raise _lib.RmsnError(st, "rmsattn_block_norms")
    return out, residual_out, out_scale
