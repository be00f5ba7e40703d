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

import ctypes
import functools
from typing import Optional

import torch

from . import _binding as B
from .api import _DT, Workspace


def _check(cond, what: str):
    if not cond:
        raise ValueError(what)


def _wrong(dev, *specs):
    """Raises for the first of (name, tensor, dtype, shape) that is not a dense
    tensor of that type and shape on device number ``dev`` (None in a shape: any
    extent)."""
    for name, t, dtype, shape in specs:
        fits = t.dim() == len(shape) and all(b is None or a == b for a, b in zip(t.shape, shape))
        if not (fits and t.dtype is dtype and t.get_device() == dev and t.is_contiguous()):
            want = ", ".join("any" if x is None else str(x) for x in shape)
            raise ValueError(f"{name}: expected a contiguous [{want}] {dtype} tensor on cuda:{dev}, got "
                             f"{tuple(t.shape)} {t.dtype} on {t.device}, strides {t.stride()}")
    raise ValueError("a tensor of the call changed while it was checked")


def _dense(t, dtype, dev, shape):
    return t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous()


def _pools(k_pages):
    """Device number, element type and (pages, Hkv, page_size, D)."""
    dt = k_pages.dtype
    dev = k_pages.get_device()
    _check(dev >= 0, "k_pages: a CUDA tensor")
    _check(dt in _DT, "k_pages: float16 or bfloat16")
    _check(k_pages.dim() == 4, "k_pages: [pages, Hkv, page_size, D]")
    return dev, dt, k_pages.shape


@functools.lru_cache(maxsize=1024)
def _plan(dev, *fields):
    """A reference to the dims struct and the scratch bytes of a shape, for any
    length that the block table can hold."""
    dims = B.make_paged_dims(*fields)
    with torch.cuda.device(dev):
        nbytes = B.gqa_paged_workspace_size(dims, max(1, min(dims.max_pages * dims.page_size, 2**31 - 1)), 0)
    return ctypes.byref(dims), nbytes


def _raw(dev, stream):
    """The handle of the stream to launch on."""
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _new(like, shape, stream, dtype=None):
    """A tensor on the device (and of the type) of ``like``, made on the call's
    stream."""
    dtype = dtype or like.dtype
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)  # (new_empty takes 2 us more)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def _capturing(stream):
    if stream is None:
        return torch.cuda.is_current_stream_capturing()
    with torch.cuda.stream(stream):
        return torch.cuda.is_current_stream_capturing()


def _scratch(workspace: Optional[Workspace], nbytes, like, dev, stream, raw):
    """Scratch for one call: the workspace's buffer of this stream, or, without
    one and while the stream is captured into a graph, a buffer of the call's own
    (captured graphs share no scratch with each other or with eager calls)."""
    if nbytes == 0:
        return None
    if workspace is None or _capturing(stream):
        return _new(like, nbytes, stream, torch.uint8)
    buf = workspace.paged.get((dev, raw))
    if buf is None or buf.numel() < nbytes:
        buf = workspace.paged[(dev, raw)] = _new(like, nbytes, stream, torch.uint8)
    return buf


def _ptr(t):
    return None if t is None else t.data_ptr()


def _call(where, dev, *args):
    fn = getattr(_lib or _load(), where)
    if torch._C._cuda_getDevice() == dev:
        status = fn(*args)
    else:
        with torch.cuda.device(dev):
            status = fn(*args)
    if status:
        raise B.GqaError(status, where)


_lib = None


def _load():
    global _lib
    _lib = B.load_library()
    return _lib


def paged_append(query, key, value, k_pages, v_pages, block_table, cu_seqlens, seqlens_k, total_sequence_length,
                 q_norm_weight=None, k_norm_weight=None, norm_eps=1e-6, cos_cache=None, sin_cache=None,
                 positions=None, query_out=None, stream=None, rotary_interleaved=0):
    """The new rows enter the cache: per-head RMS norm (where a weight [D] is
    given) and rotation (where cos/sin [rows, D/2] are given; at ``positions``,
    int32 [tokens], or at the rows' slots) of queries and keys in one pass,
    keys and values written to their pages.  key and value None: packed QKV in
    query.  Returns the queries [tokens, H*D] (``query_out``, which may be
    ``query`` itself unless packed)."""
    dev, dt, shape = _pools(k_pages)
    num_pages, hkv, page, D = shape
    batch, columns = block_table.shape
    tokens, width = query.shape
    packed = key is None and value is None
    _check(packed or (key is not None and value is not None), "key and value: both or neither")
    H = width // D - (2 * hkv if packed else 0)
    i32 = torch.int32
    specs = [("k_pages", k_pages, dt, shape), ("v_pages", v_pages, dt, shape),
             ("block_table", block_table, i32, (batch, columns)), ("cu_seqlens", cu_seqlens, i32, (batch + 1,)),
             ("seqlens_k", seqlens_k, i32, (batch,)),
             ("query", query, dt, (tokens, (H + (2 * hkv if packed else 0)) * D))]
    if not packed:
        specs += [("key", key, dt, (tokens, hkv * D)), ("value", value, dt, (tokens, hkv * D))]
    if q_norm_weight is not None:
        specs.append(("q_norm_weight", q_norm_weight, dt, (D,)))
    if k_norm_weight is not None:
        specs.append(("k_norm_weight", k_norm_weight, dt, (D,)))
    rows = 0
    if cos_cache is not None:
        _check(sin_cache is not None, "cos_cache and sin_cache: both or neither")
        rows = cos_cache.shape[0]
        specs += [("cos_cache", cos_cache, dt, (rows, D // 2)), ("sin_cache", sin_cache, dt, (rows, D // 2))]
    if positions is not None:
        specs.append(("positions", positions, i32, (tokens,)))
    if query_out is None:
        query_out = _new(query, (tokens, H * D), stream)
    else:
        specs.append(("query_out", query_out, dt, (tokens, H * D)))
    for _, t, d, sh in specs:
        if not _dense(t, d, dev, sh):
            _wrong(dev, *specs)
    dims, _ = _plan(dev, batch, tokens, 1, H, hkv, D, page, num_pages, columns, _DT[dt], rotary_interleaved, rows)
    _call("gqa_paged_append", dev, dims, query.data_ptr(), _ptr(key), _ptr(value), _ptr(q_norm_weight),
          _ptr(k_norm_weight), norm_eps, _ptr(cos_cache), _ptr(sin_cache), _ptr(positions), k_pages.data_ptr(),
          v_pages.data_ptr(), block_table.data_ptr(), cu_seqlens.data_ptr(), seqlens_k.data_ptr(),
          total_sequence_length, query_out.data_ptr(), _raw(dev, stream))
    return query_out


def paged_attention(query, k_pages, v_pages, block_table, cu_seqlens, seqlens_k, max_new_tokens,
                    total_sequence_length, scale=0.0, local_window_size=0, output=None, lse=None,
                    workspace: Optional[Workspace] = None, stream=None):
    """Attention of the new tokens (whose rows paged_append has written) over
    their sequences' pages, causal, with an optional window.  Returns the output
    [tokens, H*D]; ``lse`` (float32 [tokens, H]), where given, gets the
    logarithm of the softmax denominators."""
    dev, dt, shape = _pools(k_pages)
    num_pages, hkv, page, D = shape
    batch, columns = block_table.shape
    qshape = query.shape
    tokens, width = qshape
    H = width // D
    i32 = torch.int32
    if output is None:
        output = _new(query, qshape, stream)
    if not (k_pages.is_contiguous() and _dense(v_pages, dt, dev, shape)
            and _dense(block_table, i32, dev, (batch, columns)) and _dense(cu_seqlens, i32, dev, (batch + 1,))
            and _dense(seqlens_k, i32, dev, (batch,)) and _dense(query, dt, dev, (tokens, H * D))
            and _dense(output, dt, dev, qshape)
            and (lse is None or _dense(lse, torch.float32, dev, (tokens, H)))):
        _wrong(dev, ("k_pages", k_pages, dt, shape), ("v_pages", v_pages, dt, shape),
               ("block_table", block_table, i32, (batch, columns)), ("cu_seqlens", cu_seqlens, i32, (batch + 1,)),
               ("seqlens_k", seqlens_k, i32, (batch,)), ("query", query, dt, (tokens, H * D)),
               ("output", output, dt, qshape),
               ("lse", query if lse is None else lse, dt if lse is None else torch.float32,
                qshape if lse is None else (tokens, H)))
    dims, nbytes = _plan(dev, batch, tokens, max_new_tokens, H, hkv, D, page, num_pages, columns, _DT[dt])
    raw = _raw(dev, stream)
    ws = _scratch(workspace, nbytes, query, dev, stream, raw)
    _call("gqa_paged_attention", dev, dims, query.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
          block_table.data_ptr(), cu_seqlens.data_ptr(), seqlens_k.data_ptr(), total_sequence_length, scale,
          local_window_size, output.data_ptr(), _ptr(lse), _ptr(ws), nbytes, raw)
    return output


def paged_key_weights(query, lse, k_pages, weights, block_table, cu_seqlens, seqlens_k, max_new_tokens,
                      total_sequence_length, scale=0.0, local_window_size=0, weights_in=None,
                      workspace: Optional[Workspace] = None, stream=None):
    """Adds to every cached key's weight the attention weight it receives from
    the new tokens (over the query heads of its KV head): ``weights`` float32
    [pages, Hkv, page_size] becomes ``weights_in`` (default: itself) plus that
    sum for cached keys, the sum alone for new ones.  query and lse as
    paged_attention took and left them.  Returns ``weights``.  (No scratch is
    needed: ``workspace`` is taken for uniformity.)"""
    dev, dt, shape = _pools(k_pages)
    num_pages, hkv, page, D = shape
    batch, columns = block_table.shape
    tokens, width = query.shape
    H = width // D
    i32, f32 = torch.int32, torch.float32
    weights_in = weights if weights_in is None else weights_in
    if not (k_pages.is_contiguous() and _dense(block_table, i32, dev, (batch, columns))
            and _dense(cu_seqlens, i32, dev, (batch + 1,)) and _dense(seqlens_k, i32, dev, (batch,))
            and _dense(query, dt, dev, (tokens, H * D)) and _dense(lse, f32, dev, (tokens, H))
            and _dense(weights, f32, dev, shape[:3]) and _dense(weights_in, f32, dev, shape[:3])):
        _wrong(dev, ("k_pages", k_pages, dt, shape), ("block_table", block_table, i32, (batch, columns)),
               ("cu_seqlens", cu_seqlens, i32, (batch + 1,)), ("seqlens_k", seqlens_k, i32, (batch,)),
               ("query", query, dt, (tokens, H * D)), ("lse", lse, f32, (tokens, H)),
               ("weights", weights, f32, shape[:3]), ("weights_in", weights_in, f32, shape[:3]))
    dims, _ = _plan(dev, batch, tokens, max_new_tokens, H, hkv, D, page, num_pages, columns, _DT[dt])
    _call("gqa_paged_key_weights", dev, dims, query.data_ptr(), lse.data_ptr(), k_pages.data_ptr(),
          block_table.data_ptr(), cu_seqlens.data_ptr(), seqlens_k.data_ptr(), total_sequence_length, scale,
          local_window_size, weights_in.data_ptr(), weights.data_ptr(), None, 0, _raw(dev, stream))
    return weights


def paged_evict(k_pages, v_pages, weights, block_table, seqlens_k, total_sequence_length, budget, recent=0,
                dst_block_table=None, kept=None, new_seqlens=None, workspace: Optional[Workspace] = None, stream=None):
    """Cuts every sequence to at most ``budget`` tokens: of each (sequence, KV
    head) the ``recent`` last ones stay and the heaviest of the others (equal
    weights: the lower slot), in order, moved with their weights to the first
    slots of ``dst_block_table``'s pages (None: in place).  Returns (kept int32
    [B, Hkv, budget], the old slots, -1 behind the last; new_seqlens int32
    [B]).  (No scratch is needed: ``workspace`` is taken for uniformity.)"""
    dev, dt, shape = _pools(k_pages)
    num_pages, hkv, page, D = shape
    batch, columns = block_table.shape
    i32, f32 = torch.int32, torch.float32
    _check(budget >= 1, "budget: at least 1")
    dst_columns = 0 if dst_block_table is None else dst_block_table.shape[-1]
    mine = kept is None, new_seqlens is None
    if mine[0]:
        kept = _new(block_table, (batch, hkv, budget), stream)
    if mine[1]:
        new_seqlens = _new(seqlens_k, (batch,), stream)
    if not (k_pages.is_contiguous() and _dense(v_pages, dt, dev, shape) and _dense(weights, f32, dev, shape[:3])
            and _dense(block_table, i32, dev, (batch, columns)) and _dense(seqlens_k, i32, dev, (batch,))
            and (dst_block_table is None or _dense(dst_block_table, i32, dev, (batch, dst_columns)))
            and (mine[0] or _dense(kept, i32, dev, (batch, hkv, budget)))
            and (mine[1] or _dense(new_seqlens, i32, dev, (batch,)))):
        _wrong(dev, ("k_pages", k_pages, dt, shape), ("v_pages", v_pages, dt, shape),
               ("weights", weights, f32, shape[:3]), ("block_table", block_table, i32, (batch, columns)),
               ("seqlens_k", seqlens_k, i32, (batch,)),
               ("dst_block_table", block_table if dst_block_table is None else dst_block_table, i32,
                (batch, columns if dst_block_table is None else dst_columns)),
               ("kept", kept, i32, (batch, hkv, budget)), ("new_seqlens", new_seqlens, i32, (batch,)))
    dims, _ = _plan(dev, batch, 1, 1, hkv, hkv, D, page, num_pages, columns, _DT[dt])
    _call("gqa_paged_evict", dev, dims, k_pages.data_ptr(), v_pages.data_ptr(), weights.data_ptr(),
          block_table.data_ptr(), _ptr(dst_block_table), dst_columns, seqlens_k.data_ptr(), total_sequence_length,
          budget, recent, kept.data_ptr(), new_seqlens.data_ptr(), None, 0, _raw(dev, stream))
    return kept, new_seqlens
