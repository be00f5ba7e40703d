"""Tensor-level convenience over the paged-cache entry points
(include/gqa_paged.h): derives the dims from tensor shapes, checks the
tensors, keeps the scratch, and raises on a non-OK status.  Marshalling only;
the CUDA library does the work.

The cache is two pools of pages, ``k_pages`` and ``v_pages`` [pages, Hkv,
page_size, D], and an int32 ``block_table`` [B, columns] of each sequence's
pages.  New tokens come as token arrays [tokens, heads * D]; sequence b owns
rows ``cu_seqlens[b]`` to ``cu_seqlens[b + 1]`` (int32 [B + 1]) and has
``seqlens_k[b]`` (int32 [B]) tokens in the cache already.
``total_sequence_length`` and ``max_new_tokens`` are the host's upper bounds on
a sequence's length (new tokens included) and on its new tokens.

Every call runs on ``stream`` (default: the current stream of the pools'
device).  As everywhere in torch, tensors made on another stream must be
ordered before the call by the caller."""
from __future__ import annotations

import contextlib
import functools
from typing import Optional

import torch

from . import _binding as B
from .api import _DT, Workspace


def _check(cond, what: str):
    if not cond:
        raise ValueError(what)


def _tensor(name, t, dtype, ndim, device):
    """A dense CUDA tensor of the given type, rank and device."""
    if not (t.dtype is dtype and t.dim() == ndim and t.device == device and t.is_contiguous()):
        raise ValueError(f"{name}: expected a contiguous {ndim}-d {dtype} tensor on {device}, got "
                         f"{tuple(t.shape)} {t.dtype} on {t.device}, strides {t.stride()}")


def _pools(k_pages, v_pages=None):
    _check(k_pages.dtype in _DT, "k_pages: float16 or bfloat16")
    _check(k_pages.is_cuda, "k_pages: a CUDA tensor")
    _tensor("k_pages", k_pages, k_pages.dtype, 4, k_pages.device)
    if v_pages is not None:
        _tensor("v_pages", v_pages, k_pages.dtype, 4, k_pages.device)
        _check(v_pages.shape == k_pages.shape, "v_pages: the shape of k_pages")
    return k_pages.device, k_pages.dtype


def _lists(device, block_table, cu_seqlens, seqlens_k):
    _tensor("block_table", block_table, torch.int32, 2, device)
    batch = block_table.shape[0]
    if cu_seqlens is not None:
        _tensor("cu_seqlens", cu_seqlens, torch.int32, 1, device)
        _check(cu_seqlens.shape[0] == batch + 1, "cu_seqlens: one entry more than block_table has rows")
    _tensor("seqlens_k", seqlens_k, torch.int32, 1, device)
    _check(seqlens_k.shape[0] == batch, "seqlens_k: one entry for each row of block_table")
    return batch


@functools.lru_cache(maxsize=512)
def _dims(*fields):
    return B.make_paged_dims(*fields)


@functools.lru_cache(maxsize=512)
def _scratch_bytes(device_index, fields, total, window):
    return B.gqa_paged_workspace_size(_dims(*fields), total, window)


def _on(device, stream):
    """Context with `device` current, and the stream to launch on."""
    ctx = contextlib.nullcontext() if torch.cuda.current_device() == device.index else torch.cuda.device(device)
    return ctx, torch.cuda.current_stream(device) if stream is None else stream


def _scratch(workspace: Optional[Workspace], nbytes, device, stream):
    """Scratch for one call: the workspace's buffer of this stream, or, without
    one and while a graph is captured, a buffer of the call's own (captured
    graphs share no scratch with each other or with eager calls)."""
    if nbytes == 0:
        return None
    capturing = torch.cuda.is_current_stream_capturing()
    if workspace is not None and not capturing:
        key = (device, stream.cuda_stream)
        buf = workspace.paged.get(key)
        if buf is not None and buf.numel() >= nbytes:
            return buf
    with torch.cuda.stream(stream):
        buf = torch.empty(nbytes, dtype=torch.uint8, device=device)
    if workspace is not None and not capturing:
        workspace.paged[key] = buf
    return buf


def _raise(status, where):
    if status != B.GQA_OK:
        raise B.GqaError(status, where)


def paged_append(query, key, value, k_pages, v_pages, block_table, cu_seqlens, seqlens_k, total_sequence_length,
                 q_norm_weight=None, k_norm_weight=None, norm_eps=1e-6, cos_cache=None, sin_cache=None,
                 positions=None, query_out=None, stream=None, rotary_interleaved=0):
    """The new rows enter the cache: per-head RMS norm (where a weight [D] is
    given) and rotation (where cos/sin [rows, D/2] are given; at ``positions``,
    int32 [tokens], or at the rows' slots) of queries and keys in one pass,
    keys and values written to their pages.  key and value None: packed QKV in
    query.  Returns the queries [tokens, H*D] (``query_out``, which may be
    ``query`` itself unless packed)."""
    device, dt = _pools(k_pages, v_pages)
    batch = _lists(device, block_table, cu_seqlens, seqlens_k)
    num_pages, hkv, page, D = k_pages.shape
    _tensor("query", query, dt, 2, device)
    tokens, width = query.shape
    _check(width % D == 0, "query: a multiple of the head size wide")
    H = width // D - (2 * hkv if key is None and value is None else 0)
    _check((key is None) == (value is None), "key and value: both or neither")
    if key is not None:
        for name, t in (("key", key), ("value", value)):
            _tensor(name, t, dt, 2, device)
            _check(t.shape == (tokens, hkv * D), f"{name}: [tokens, Hkv * D]")
    for name, t in (("q_norm_weight", q_norm_weight), ("k_norm_weight", k_norm_weight)):
        if t is not None:
            _tensor(name, t, dt, 1, device)
            _check(t.shape[0] == D, f"{name}: [D]")
    rows = 0
    if cos_cache is not None:
        _check(sin_cache is not None and sin_cache.shape == cos_cache.shape, "cos_cache and sin_cache: one shape")
        _tensor("cos_cache", cos_cache, dt, 2, device)
        _tensor("sin_cache", sin_cache, dt, 2, device)
        rows = cos_cache.shape[0]
        _check(cos_cache.shape[1] * 2 == D, "cos_cache: [rows, D/2]")
    if positions is not None:
        _tensor("positions", positions, torch.int32, 1, device)
        _check(positions.shape[0] == tokens, "positions: one for each token")
    ctx, stream = _on(device, stream)
    if query_out is None:
        with torch.cuda.stream(stream):
            query_out = query.new_empty((tokens, H * D))
    else:
        _tensor("query_out", query_out, dt, 2, device)
        _check(query_out.shape == (tokens, H * D), "query_out: [tokens, H * D]")
    dims = _dims(batch, tokens, 1, H, hkv, D, page, num_pages, block_table.shape[1], _DT[dt], rotary_interleaved, rows)
    with ctx:
        st = B.gqa_paged_append(dims, query, key, value, q_norm_weight, k_norm_weight, norm_eps, cos_cache, sin_cache,
                                positions, k_pages, v_pages, block_table, cu_seqlens, seqlens_k,
                                total_sequence_length, query_out, stream)
    _raise(st, "gqa_paged_append")
    return query_out


def _fields(query, k_pages, block_table, batch, max_new_tokens):
    num_pages, hkv, page, D = k_pages.shape
    tokens, width = query.shape
    _check(width % D == 0, "query: a multiple of the head size wide")
    return (batch, tokens, max_new_tokens, width // D, hkv, D, page, num_pages, block_table.shape[1],
            _DT[query.dtype])


def paged_attention(query, k_pages, v_pages, block_table, cu_seqlens, seqlens_k, max_new_tokens,
                    total_sequence_length, scale=0.0, local_window_size=0, output=None, lse=None,
                    workspace: Optional[Workspace] = None, stream=None):
    """Attention of the new tokens (whose rows paged_append has written) over
    their sequences' pages, causal, with an optional window.  Returns the output
    [tokens, H*D]; ``lse`` (float32 [tokens, H]), where given, gets the
    logarithm of the softmax denominators."""
    device, dt = _pools(k_pages, v_pages)
    batch = _lists(device, block_table, cu_seqlens, seqlens_k)
    _tensor("query", query, dt, 2, device)
    fields = _fields(query, k_pages, block_table, batch, max_new_tokens)
    if lse is not None:
        _tensor("lse", lse, torch.float32, 2, device)
        _check(lse.shape == (query.shape[0], fields[3]), "lse: [tokens, H]")
    ctx, stream = _on(device, stream)
    if output is None:
        with torch.cuda.stream(stream):
            output = torch.empty_like(query)
    else:
        _tensor("output", output, dt, 2, device)
        _check(output.shape == query.shape, "output: the shape of query")
    with ctx:
        nbytes = _scratch_bytes(device.index, fields, total_sequence_length, local_window_size)
        ws = _scratch(workspace, nbytes, device, stream)
        st = B.gqa_paged_attention(_dims(*fields), query, k_pages, v_pages, block_table, cu_seqlens, seqlens_k,
                                   total_sequence_length, scale, local_window_size, output, lse, ws, nbytes, stream)
    _raise(st, "gqa_paged_attention")
    return output


def paged_key_weights(query, lse, k_pages, weights, block_table, cu_seqlens, seqlens_k, max_new_tokens,
                      total_sequence_length, scale=0.0, local_window_size=0, weights_in=None,
                      workspace: Optional[Workspace] = None, stream=None):
    """Adds to every cached key's weight the attention weight it receives from
    the new tokens (over the query heads of its KV head): ``weights`` float32
    [pages, Hkv, page_size] becomes ``weights_in`` (default: itself) plus that
    sum for cached keys, the sum alone for new ones.  query and lse as
    paged_attention took and left them.  Returns ``weights``."""
    device, dt = _pools(k_pages)
    batch = _lists(device, block_table, cu_seqlens, seqlens_k)
    _tensor("query", query, dt, 2, device)
    fields = _fields(query, k_pages, block_table, batch, max_new_tokens)
    _tensor("lse", lse, torch.float32, 2, device)
    _check(lse.shape == (query.shape[0], fields[3]), "lse: [tokens, H]")
    weights_in = weights if weights_in is None else weights_in
    for name, t in (("weights", weights), ("weights_in", weights_in)):
        _tensor(name, t, torch.float32, 3, device)
        _check(t.shape == k_pages.shape[:3], f"{name}: [pages, Hkv, page_size]")
    ctx, stream = _on(device, stream)
    with ctx:
        nbytes = _scratch_bytes(device.index, fields, total_sequence_length, local_window_size)
        ws = _scratch(workspace, nbytes, device, stream)
        st = B.gqa_paged_key_weights(_dims(*fields), query, lse, k_pages, block_table, cu_seqlens, seqlens_k,
                                     total_sequence_length, scale, local_window_size, weights_in, weights, ws,
                                     nbytes, stream)
    _raise(st, "gqa_paged_key_weights")
    return weights


def paged_evict(k_pages, v_pages, weights, block_table, seqlens_k, total_sequence_length, budget, recent=0,
                dst_block_table=None, kept=None, new_seqlens=None, workspace: Optional[Workspace] = None, stream=None):
    """Cuts every sequence to at most ``budget`` tokens: of each (sequence, KV
    head) the ``recent`` last ones stay and the heaviest of the others (equal
    weights: the lower slot), in order, moved with their weights to the first
    slots of ``dst_block_table``'s pages (None: in place).  Returns (kept int32
    [B, Hkv, budget], the old slots, -1 behind the last; new_seqlens int32
    [B])."""
    device, dt = _pools(k_pages, v_pages)
    batch = _lists(device, block_table, None, seqlens_k)
    num_pages, hkv, page, D = k_pages.shape
    _tensor("weights", weights, torch.float32, 3, device)
    _check(weights.shape == k_pages.shape[:3], "weights: [pages, Hkv, page_size]")
    columns = 0
    if dst_block_table is not None:
        _tensor("dst_block_table", dst_block_table, torch.int32, 2, device)
        _check(dst_block_table.shape[0] == batch, "dst_block_table: as many rows as block_table")
        columns = dst_block_table.shape[1]
    ctx, stream = _on(device, stream)
    with torch.cuda.stream(stream):
        if kept is None:
            _check(budget >= 1, "budget: at least 1")
            kept = torch.empty((batch, hkv, budget), dtype=torch.int32, device=device)
        if new_seqlens is None:
            new_seqlens = torch.empty_like(seqlens_k)
    _tensor("kept", kept, torch.int32, 3, device)
    _check(kept.shape == (batch, hkv, budget), "kept: [B, Hkv, budget]")
    _tensor("new_seqlens", new_seqlens, torch.int32, 1, device)
    _check(new_seqlens.shape[0] == batch, "new_seqlens: [B]")
    dims = _dims(batch, 1, 1, hkv, hkv, D, page, num_pages, block_table.shape[1], _DT[dt])
    with ctx:
        st = B.gqa_paged_evict(dims, k_pages, v_pages, weights, block_table, dst_block_table, columns, seqlens_k,
                               total_sequence_length, budget, recent, kept, new_seqlens, None, 0, stream)
    _raise(st, "gqa_paged_evict")
    return kept, new_seqlens
