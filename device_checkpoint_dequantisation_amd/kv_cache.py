"""A cache of keys and values in 8 bits, the operator that writes it (st_kv_append) and the attention that reads it
(st_kv_attention).

    cache = QuantizedKvCache.empty(pages=4096, heads=8, head_dim=128, block=64)
    table, lengths                                   # int32 [seqs, blocks] page of each block, int32 [seqs] tokens
    lengths += 1                                     # one new token for each sequence
    kv_append(cache, k, v, table, lengths)           # k, v [seqs, 8, 128]
    o = kv_attention(q, cache, table, lengths)       # q [seqs, 32, 128]

Prompts, or chunks of them, lie one after the other with ``starts`` [seqs + 1].  Both operators run on the current stream (or
``stream``), allocate with torch, synchronise nothing and can be captured into a HIP graph: the table, the lengths and
the starts are read on the device.  They have no backward pass."""
from __future__ import annotations

import ctypes as C
import math
from dataclasses import dataclass

import torch

from ._lib import KvAppendArgs, KvAttentionArgs, check, lib
from .ops import _E4M3, _E8M0, _TYPE, _launch, _on_device, _overlaps, _span

BLOCKS = (16, 32, 64, 128)         # tokens of a page
HEAD_DIMS = (64, 128, 256)         # of kv_attention; kv_append takes every multiple of 32 up to 256


@dataclass
class QuantizedKvCache:
    """Pages of ``block`` tokens; a value is code * scale, with one power of two for a page and a head.
      k        float8_e4m3fn [pages, heads, block, head_dim]
      v        float8_e4m3fn [pages, heads, head_dim, block]
      k_scale, v_scale  float8_e8m0fnu [pages, heads]"""
    k: object
    v: object
    k_scale: object
    v_scale: object

    @classmethod
    def empty(cls, pages: int, heads: int, head_dim: int, block: int = 64, device="cuda") -> "QuantizedKvCache":
        """A cache of zeros."""
        new = lambda *s: torch.zeros(s, dtype=torch.uint8, device=device)   # noqa: E731
        return cls(new(pages, heads, block, head_dim).view(_E4M3), new(pages, heads, head_dim, block).view(_E4M3),
                   new(pages, heads).view(_E8M0), new(pages, heads).view(_E8M0))


def _check_cache(c, who: str):
    if not isinstance(c, QuantizedKvCache):
        raise ValueError(f"{who}: the cache is a {type(c).__name__}; a QuantizedKvCache is needed")
    k, v, ks, vs = c.k, c.v, c.k_scale, c.v_scale
    shape = k.shape
    if not (len(shape) == 4 and k.dtype == _E4M3 and k.is_contiguous()):
        raise ValueError(f"{who}: the cache's keys are {k.dtype} {tuple(shape)}, strides {k.stride()}")
    pages, heads, block, dim = shape
    if not (v.dtype == _E4M3 and v.shape == (pages, heads, dim, block) and v.is_contiguous()):
        raise ValueError(f"{who}: the cache's values are {v.dtype} {tuple(v.shape)}, strides {v.stride()}; "
                         f"{(pages, heads, dim, block)} are needed")
    for s in (ks, vs):
        if not (s.dtype == _E8M0 and s.shape == (pages, heads) and s.is_contiguous()):
            raise ValueError(f"{who}: the cache's scales are {s.dtype} {tuple(s.shape)}, strides {s.stride()}; {(pages, heads)} are needed")
    if block not in BLOCKS:
        raise ValueError(f"{who}: pages of {block} tokens; one of {BLOCKS} is needed")
    return pages, heads, block, dim


def _check_seqs(table, lengths, starts, max_new, tokens: int, who: str):
    """(seqs, max_new) of the arguments both operators share."""
    if not (table.dtype == torch.int32 and table.dim() == 2
            and (table.is_contiguous() or ((table.shape[1] <= 1 or table.stride(1) == 1)
                                           and (table.shape[0] <= 1 or table.stride(0) >= table.shape[1])))):
        raise ValueError(f"{who}: table {table.dtype} {tuple(table.shape)}, strides {table.stride()}; int32 [sequences, blocks] is needed")
    seqs = table.shape[0]
    if not (lengths.dtype == torch.int32 and lengths.shape == (seqs,) and lengths.is_contiguous()):
        raise ValueError(f"{who}: lengths {lengths.dtype} {tuple(lengths.shape)}, strides {lengths.stride()}; int32 [{seqs}] is needed")
    if starts is None:
        if seqs == 0 and tokens or seqs and tokens % seqs:
            raise ValueError(f"{who}: {tokens} tokens are not {seqs} equal parts; starts is needed")
        if max_new is not None:
            raise ValueError(f"{who}: max_new goes with starts")
        return seqs, tokens // seqs if seqs else 0
    if not (starts.dtype == torch.int32 and starts.shape == (seqs + 1,) and starts.is_contiguous()):
        raise ValueError(f"{who}: starts {starts.dtype} {tuple(starts.shape)}, strides {starts.stride()}; int32 [{seqs + 1}] is needed")
    if max_new is None:
        return seqs, tokens
    if not (isinstance(max_new, int) and max_new >= 0):
        raise ValueError(f"{who}: max_new {max_new!r} is not a number of tokens")
    return seqs, min(max_new, tokens)


def _heads(t, name: str, heads, dim: int, who: str):
    """Checks t [tokens, heads, dim] with adjacent elements of a head; a dimension of one has no stride to check."""
    if not (t.dim() == 3 and t.shape[2] == dim and (heads is None or t.shape[1] == heads)):
        raise ValueError(f"{who}: {name} is {tuple(t.shape)}; [tokens, {'heads' if heads is None else heads}, {dim}] is needed")
    if not (t.numel() == 0 or t.stride(2) == 1):
        raise ValueError(f"{who}: the last dimension of {name} must be contiguous (stride 1, got {t.stride(2)})")


def kv_append(cache: QuantizedKvCache, k, v, table, lengths, starts=None, max_new: int | None = None, stream=None) -> None:
    """Write new tokens' keys and values (``k``, ``v`` [tokens, heads, head_dim], bf16, fp16 or fp32) into the cache's pages.

    ``lengths`` [seqs] counts the new tokens in.  Sequence s has rows ``starts[s]`` to ``starts[s + 1] - 1`` (without
    ``starts``, the s-th of equal parts), its last tokens; ``max_new`` is at least the most of any sequence (default: all rows; a
    closer bound launches less).  Block j of the sequence lies on page ``table[s, j]``; tokens whose block has no page there (a
    number that is none, or past the table) are left out, and so are those a larger sequence has behind ``max_new``.

    A page and head has one power of two for its scale: the smallest >= amax / 448 over its finite values, but never less than
    that of tokens it holds already, whose codes are rounded to the new scale where it grows.  A value that is not finite becomes
    the NaN code.  A page that new tokens go to belongs to one block of one sequence; pages of earlier tokens may be shared."""
    who = "kv_append"
    pages, heads, block, dim = _check_cache(cache, who)
    if dim % 32 or dim == 0 or dim > 256:
        raise ValueError(f"{who}: head_dim {dim} is not a multiple of 32 up to 256")
    _heads(k, "k", heads, dim, who)
    _heads(v, "v", heads, dim, who)
    if not (k.dtype in _TYPE and v.dtype == k.dtype and v.shape == k.shape):
        raise ValueError(f"{who}: k {k.dtype} {tuple(k.shape)}, v {v.dtype} {tuple(v.shape)}; bf16, fp16 or fp32 of one shape are needed")
    _on_device(cache.k.device, (cache.k, cache.v, cache.k_scale, cache.v_scale, k, v, table, lengths, starts), who)
    tokens = k.shape[0]
    seqs, most = _check_seqs(table, lengths, starts, max_new, tokens, who)
    if tokens == 0 or seqs == 0 or most == 0 or heads == 0:
        return
    ck, cv, sk, sv = cache.k.data_ptr(), cache.v.data_ptr(), cache.k_scale.data_ptr(), cache.v_scale.data_ptr()
    codes, scales = pages * heads * block * dim, pages * heads
    (ka, kb), (va, vb) = _span(k), _span(v)
    for a, n in ((ck, codes), (cv, codes), (sk, scales), (sv, scales)):
        if a < kb and ka < a + n or a < vb and va < a + n:
            raise ValueError(f"{who}: the cache overlaps an input")
    k_pitch, k_head, _ = k.stride()
    v_pitch, v_head, _ = v.stride()
    args = KvAppendArgs(ka, va, ck, cv, sk, sv, table.data_ptr(), lengths.data_ptr(), None if starts is None else starts.data_ptr(),
                        pages, tokens, seqs, most, table.shape[1], table.stride(0), k_pitch, k_head, v_pitch, v_head, heads, dim, block,
                        _TYPE[k.dtype])
    _launch(lib().st_kv_append, args, cache.k.device, stream,
            (k, v, cache.k, cache.v, cache.k_scale, cache.v_scale, table, lengths, starts), who)


def kv_attention(q, cache: QuantizedKvCache, table, lengths, starts=None, max_new: int | None = None, scale: float | None = None,
                 causal: bool = True, window: int | None = None, out=None, stream=None):
    """softmax(scale * q k^T) v over the cache, for ``q`` [tokens, query heads, head_dim] in bf16 or fp16; the result has q's
    shape and type.  Query head h reads head h // (query heads / heads) of the cache; ``scale`` is 1 / sqrt(head_dim) by default.

    ``table``, ``lengths``, ``starts`` and ``max_new`` are those of :func:`kv_append`.  ``causal``: the queries are the last tokens of
    their sequence and each sees the tokens up to its own, with a ``window`` the last ``window`` of them; not causal: each sees all
    ``lengths[s]`` tokens, such as an encoder's, and a sequence may have more queries than tokens.  A query that sees no token, or only scores of minus infinity, gives 0.
    Tokens that a query does not see, and what pages hold behind a sequence's end, have no part in its result.
    A cache of no pages and a table of no blocks are refused.
    Rows that belong to no sequence (before ``starts[0]``, from ``starts[-1]`` on, behind ``max_new``) stay as they are in ``out`` and are
    0 without one.  Scores and sums are fp32; the softmax's numerators enter the second product with fp16's 11 bits, values
    exactly unless their page's scale is 2**-7 times the largest that the query sees or less, then to 2**-17 of that scale."""
    who = "kv_attention"
    pages, heads, block, dim = _check_cache(cache, who)
    if dim not in HEAD_DIMS:
        raise ValueError(f"{who}: head_dim {dim}; one of {HEAD_DIMS} is needed")
    _heads(q, "q", None, dim, who)
    if q.dtype not in (torch.bfloat16, torch.float16):
        raise ValueError(f"{who}: q is {q.dtype}; bf16 or fp16 is needed")
    if heads == 0 and q.shape[1] or heads and q.shape[1] % heads:
        raise ValueError(f"{who}: {q.shape[1]} query heads for {heads} heads of the cache")
    device = q.device
    _on_device(device, (q, cache.k, cache.v, cache.k_scale, cache.v_scale, table, lengths, starts, out), who)
    tokens = q.shape[0]
    seqs, most = _check_seqs(table, lengths, starts, max_new, tokens, who)
    scale = 1.0 / math.sqrt(dim) if scale is None else float(scale)
    if not 0.0 < scale < 1e30:
        raise ValueError(f"{who}: scale {scale} is not positive")
    if window is not None and not (isinstance(window, int) and window >= 1 and causal):
        raise ValueError(f"{who}: window {window!r}; a number of tokens from 1 on is needed, and causal attention")
    if out is None:
        # (with starts there may be rows of no sequence)
        out = torch.empty(q.shape, dtype=q.dtype, device=device) if starts is None else torch.zeros(q.shape, dtype=q.dtype, device=device)
    else:
        if not (out.dtype == q.dtype and out.shape == q.shape):
            raise ValueError(f"{who}: out {out.dtype} {tuple(out.shape)}; {q.dtype} {tuple(q.shape)} is needed")
        s0, s1, s2 = out.stride()
        if not (out.numel() == 0 or (s2 == 1 and (out.shape[1] <= 1 or s1 >= dim)
                                     and (tokens <= 1 or s0 >= (out.shape[1] - 1) * s1 + dim))):
            raise ValueError(f"{who}: out has strides {out.stride()}")
        if any(_overlaps(out, t) for t in (q, cache.k, cache.v, cache.k_scale, cache.v_scale, table, lengths, starts)):
            raise ValueError(f"{who}: out overlaps an input")
    if q.numel() == 0 or seqs == 0 or most == 0:
        return out
    if pages == 0 or table.shape[1] == 0:      # no query sees a token
        raise ValueError(f"{who}: a cache of {pages} pages and a table of {table.shape[1]} blocks")
    args = KvAttentionArgs(q.data_ptr(), out.data_ptr(), cache.k.data_ptr(), cache.v.data_ptr(), cache.k_scale.data_ptr(),
                           cache.v_scale.data_ptr(), table.data_ptr(), lengths.data_ptr(),
                           None if starts is None else starts.data_ptr(), None, 0, pages, tokens, seqs, most, table.shape[1],
                           table.stride(0), q.stride(0), q.stride(1), out.stride(0), out.stride(1), min(window or 0, 2 ** 31 - 1), scale, heads,
                           q.shape[1] // heads, dim, block, int(causal), _TYPE[q.dtype])
    need = C.c_uint64()
    check(lib().st_kv_attention_workspace_bytes(C.byref(args), C.byref(need)), who)
    work = None
    if need.value:
        work = q.new_empty(need.value, dtype=torch.uint8)
        args.workspace, args.workspace_bytes = work.data_ptr(), need.value
    _launch(lib().st_kv_attention, args, device, stream,
            (q, cache.k, cache.v, cache.k_scale, cache.v_scale, table, lengths, starts, out, work), who)
    return out
