"""Torch marshalling of the operators around the cache (include/pa.h): rotary positions with the cache write,
attention with score modifiers, drafted trees, eviction by attention weight.

Argument checks and pointers only, as in ``_lib``: every step runs in the library's kernels.  All tensors of a call
are on one device; the call runs on that device, on `stream` or its current stream.
"""

from __future__ import annotations

import ctypes
import math

from . import _lib
from ._lib import (PA_ERR_SHAPE, SIZE_MAX, AttendOptions, CacheWriteOptions, PagedAttnError, _check, _ptr, dtype_code,
                   load)

_OPT_SIZE = ctypes.sizeof(AttendOptions)

_torch = _CODES = _raw_stream = _get_device = None
_I32 = _I64 = _F32 = None


def _t():
    """torch and the few names of it that a call looks up (the per-step path), bound once."""
    global _torch, _CODES, _raw_stream, _get_device, _I32, _I64, _F32
    if _torch is None:
        import torch
        _I32, _I64, _F32 = torch.int32, torch.int64, torch.float32
        _raw_stream, _get_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
        dtype_code(torch.empty(0))
        _CODES = _lib._DTYPE_CODES
        _torch = torch
    return _torch


def _code(t):
    c = _CODES.get(t.dtype)
    if c is None:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return c


def _on_one_device(first, *rest):
    """The index of the CUDA device that holds all these tensors (None: an argument left out)."""
    d = first.get_device()
    if d < 0:
        raise ValueError("q/k_cache must be a CUDA tensor")
    for t in rest:
        if t is not None and t.get_device() != d:
            raise ValueError(f"every tensor of a call must be on cuda:{d}, one is on {t.device}")
    return d


def _issue(fn, dev, stream, *args):
    """Calls fn(*args, stream handle) with `dev` current."""
    if stream is None:
        handle = _raw_stream(dev)
    elif stream.device_index == dev:
        handle = stream.cuda_stream
    else:
        raise ValueError(f"stream must be on cuda:{dev}")
    if _get_device() == dev:
        st = fn(*args, handle)
    else:
        with _torch.cuda.device(dev):
            st = fn(*args, handle)
    if st:
        _check(fn.__name__, st)


def _need(name, t, dtype, shape):
    """A contiguous tensor of this dtype and shape."""
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous {dtype} {tuple(shape)}, not {t.dtype} {tuple(t.shape)} with strides "
                         f"{t.stride()}")


def _table(name, t, rows, dtype):
    """A contiguous [rows, any] tensor; returns its width."""
    shape = t.shape
    if t.dtype is not dtype or len(shape) != 2 or shape[0] != rows or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous {dtype} [{rows}, any], not {t.dtype} {tuple(shape)}")
    return shape[1]


def _row_stride(name, t, tokens, heads, dim):
    """[tokens, heads, dim] with contiguous rows; returns the stride between tokens."""
    a, b, c = t.stride()
    if t.shape != (tokens, heads, dim) or c != 1 or (b != dim and heads > 1):
        raise ValueError(f"{name} must be [{tokens}, {heads}, {dim}] with contiguous rows per token, not "
                         f"{tuple(t.shape)} with strides {t.stride()}")
    return a if tokens > 1 else max(a, heads * dim)


def _cache(k_cache, v_cache, block_size):
    """(blocks, KV heads, head size) of the two pools."""
    shape = k_cache.shape
    if len(shape) != 4 or shape[2] != block_size or not k_cache.is_contiguous():
        raise ValueError(f"k_cache must be contiguous [blocks, H_kv, {block_size}, d], not {tuple(shape)}")
    if v_cache.shape != shape or v_cache.dtype is not k_cache.dtype or not v_cache.is_contiguous():
        raise ValueError("v_cache must be contiguous, of the shape and type of k_cache")
    return shape[0], shape[1], shape[3]


def _heads_params(num_kv_heads, scales, zero_points):
    for dtype, named in ((_F32, scales), (_I32, zero_points)):
        for t in named:
            if t is not None:
                _need("a per-KV-head scale" if dtype is _F32 else "a zero point", t, dtype, (num_kv_heads,))


def rope_frequencies(rotary_dim, base=10000.0, *, scaling=None, factor=1.0, original_positions=None, low_factor=1.0,
                     high_factor=4.0):
    """Frequencies [rotary_dim / 2] (float32, CPU) for rope_and_cache: base ** (-2 i / rotary_dim), stretched.

    scaling: None; "linear" (every frequency / factor); "base" (base * factor ** (r / (r - 2)): the slowest
    frequency is divided by factor, the fastest stays); "bands" (a frequency that turns fewer than low_factor times
    over original_positions positions is divided by factor, one that turns more than high_factor times stays, linear
    in the number of turns between them).
    """
    torch = _t()
    r = int(rotary_dim)
    if r < 2 or r % 2:
        raise ValueError("rotary_dim must be even and at least 2")
    if scaling not in (None, "linear", "base", "bands"):
        raise ValueError(f"unknown scaling {scaling!r}")
    if scaling == "base":
        if r == 2:
            raise ValueError("'base' scaling needs rotary_dim > 2")
        base = base * factor ** (r / (r - 2))
    f = base ** (-torch.arange(0, r, 2, dtype=torch.float64) / r)
    if scaling == "linear":
        f = f / factor
    elif scaling == "bands":
        if not original_positions or high_factor <= low_factor:
            raise ValueError("'bands' scaling needs original_positions and high_factor > low_factor")
        turns = f * original_positions / (2.0 * math.pi)
        keep = ((turns - low_factor) / (high_factor - low_factor)).clamp(0.0, 1.0)
        f = f / factor * (1.0 - keep) + f * keep
    return f.float()


def rope_and_cache(q, k, v, k_cache, v_cache, positions, slot_mapping, inv_freq, block_size, *, q_out=None,
                   interleaved=False, rope_scale=1.0, k_inv_scale=None, v_inv_scale=None, k_zero_point=None,
                   v_zero_point=None, pdl=False, stream=None):
    """Rotary positions of q and k, and the cache write of k and v (pa_rope_and_cache).

    q [N, H_q, d], k / v [N, H_kv, d]; positions and slot_mapping int64 [N]; inv_freq float32 [rotary_dim / 2].
    The turned q goes to q_out (default: q itself), the turned k and v into their slots; tokens with a negative slot
    are padding and left alone.  pdl as in reshape_and_cache.  Returns q_out.
    """
    _torch or _t()
    if q_out is None:
        q_out = q
    dev = _on_one_device(q, k, v, k_cache, v_cache, positions, slot_mapping, inv_freq, q_out, k_inv_scale, v_inv_scale,
                         k_zero_point, v_zero_point)
    N, Hq, D = q.shape
    blocks, Hkv, dim = _cache(k_cache, v_cache, block_size)
    if dim != D:
        raise ValueError("q and the caches must have one head size")
    dt = q.dtype
    if k.dtype is not dt or v.dtype is not dt or q_out.dtype is not dt:
        raise ValueError("q, k, v and q_out must have one type")
    qs = _row_stride("q", q, N, Hq, D)
    qos = qs if q_out is q else _row_stride("q_out", q_out, N, Hq, D)
    ks, vs = _row_stride("k", k, N, Hkv, D), _row_stride("v", v, N, Hkv, D)
    tokens = (N,)
    _need("positions", positions, _I64, tokens)
    _need("slot_mapping", slot_mapping, _I64, tokens)
    _need("inv_freq", inv_freq, _F32, inv_freq.shape[:1])
    opt = ki = vi = None
    if k_inv_scale is not None or v_inv_scale is not None:
        _heads_params(Hkv, (k_inv_scale, v_inv_scale), (k_zero_point, v_zero_point))
        ki, vi = _ptr(k_inv_scale), _ptr(v_inv_scale)
    if k_zero_point is not None or v_zero_point is not None or pdl:
        opt = ctypes.byref(CacheWriteOptions(k_zero_point=_ptr(k_zero_point), v_zero_point=_ptr(v_zero_point),
                                             pdl=1 if pdl else 0))
    _issue(load().pa_rope_and_cache, dev, stream, q_out.data_ptr(), qos, q.data_ptr(), qs, Hq, k.data_ptr(), v.data_ptr(),
           _code(q), ks, vs, k_cache.data_ptr(), v_cache.data_ptr(), _code(k_cache), blocks, positions.data_ptr(),
           slot_mapping.data_ptr(), inv_freq.data_ptr(), 2 * inv_freq.shape[0], 1 if interleaved else 0, rope_scale, N,
           Hkv, D, int(block_size), ki, vi, opt)
    return q_out


def attend_workspace_bytes(num_seqs, num_heads, num_kv_heads, head_dim, block_size, max_blocks_per_seq, max_q_len,
                           kv_dtype=_lib.PA_BF16, accumulate=False) -> int:
    """Workspace of attend / attend_tree / attend_accumulate (accumulate=True) for up to these sizes on the current device."""
    n = int(load().pa_attend_workspace_bytes(num_seqs, num_heads, num_kv_heads, head_dim, block_size,
                                             max_blocks_per_seq, max_q_len, kv_dtype, 1 if accumulate else 0))
    if n == SIZE_MAX:
        raise PagedAttnError("pa_attend_workspace_bytes", PA_ERR_SHAPE, "sizes rejected or no usable device")
    return n


def _attend(out, q, k_cache, v_cache, block_tables, seq_lens, q_starts, max_q_len, num_kv_heads, scale, block_size,
            workspace, k_scale, v_scale, k_zero_point, v_zero_point, softcap, slopes, window, prefix_lens, tree_mask,
            mass, pdl, stream):
    _torch or _t()
    dev = _on_one_device(q, out, k_cache, v_cache, block_tables, seq_lens, q_starts, workspace, k_scale, v_scale,
                         k_zero_point, v_zero_point, slopes, prefix_lens, tree_mask, mass)
    N, Hq, D = q.shape
    qs = _row_stride("q", q, N, Hq, D)
    blocks, Hkv, dim = _cache(k_cache, v_cache, block_size)
    if dim != D or Hkv != num_kv_heads:
        raise ValueError("the caches must have q's head size and num_kv_heads heads")
    if out.shape != q.shape or not out.is_contiguous():
        raise ValueError(f"out must be contiguous of shape {tuple(q.shape)}")
    if out.data_ptr() == q.data_ptr() and N:
        raise ValueError("out must not be q: its rows are read by several CTAs")
    S = seq_lens.shape[0]
    width = _table("block_tables", block_tables, S, _I32)
    _need("seq_lens", seq_lens, _I32, (S,))
    starts = None
    if q_starts is not None:
        _need("q_starts", q_starts, _I32, (S + 1,))
        starts = q_starts.data_ptr()
    if k_scale is not None or v_scale is not None:
        _heads_params(Hkv, (k_scale, v_scale), (k_zero_point, v_zero_point))
    ws, wb = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel() * workspace.element_size())
    opt = None
    if softcap or window or pdl or k_zero_point is not None or v_zero_point is not None or slopes is not None or \
            prefix_lens is not None or tree_mask is not None or mass is not None:
        words = mseq = mhead = 0
        if slopes is not None:
            _need("slopes", slopes, _F32, (Hq,))
        if prefix_lens is not None:
            _need("prefix_lens", prefix_lens, _I32, (S,))
        if tree_mask is not None:
            if tree_mask.dtype not in (_I64, getattr(_torch, "uint64", _I64)):
                raise ValueError("tree_mask must be int64 (or uint64) words")
            words = _table("tree_mask", tree_mask, N, tree_mask.dtype)
        if mass is not None:
            mseq, mhead = _mass_strides("mass", mass, S, Hkv)
            if mass.shape[2] < width * block_size:
                raise ValueError("mass rows must hold block_tables.shape[1] * block_size positions")
        opt = ctypes.byref(AttendOptions(_OPT_SIZE, _ptr(k_zero_point), _ptr(v_zero_point), softcap, _ptr(slopes), int(window),
                                         _ptr(prefix_lens), _ptr(tree_mask), words, _ptr(mass), mseq, mhead,
                                         1 if pdl else 0))
    _issue(load().pa_attend, dev, stream, out.data_ptr(), _code(out), q.data_ptr(), _code(q), qs, k_cache.data_ptr(),
           v_cache.data_ptr(), _code(k_cache), blocks, _ptr(k_scale), _ptr(v_scale), block_tables.data_ptr(), width,
           seq_lens.data_ptr(), starts, int(max_q_len), N, S, Hq, Hkv, D, scale, int(block_size), ws, wb, opt)
    return out


def _mass_strides(name, mass, seqs, heads):
    shape, (a, b, c) = mass.shape, mass.stride()
    if mass.dtype is not _F32 or len(shape) != 3 or shape[0] != seqs or shape[1] != heads or (c != 1 and shape[2] > 1):
        raise ValueError(f"{name} must be float32 [{seqs}, {heads}, positions] with contiguous rows, not {mass.dtype} "
                         f"{tuple(shape)} with strides {mass.stride()}")
    h = b if heads > 1 else max(b, shape[2])
    return (a if seqs > 1 else max(a, h * heads)), h


def attend(out, q, k_cache, v_cache, block_tables, seq_lens, q_starts, max_q_len, num_kv_heads, scale, block_size, *,
           workspace=None, k_scale=None, v_scale=None, k_zero_point=None, v_zero_point=None, softcap=0.0, slopes=None,
           window=0, prefix_lens=None, pdl=False, stream=None):
    """Attention of ragged query rows (prompt chunks, decode steps) over the paged cache (pa_attend).

    q, out [N, H_q, d]: sequence s owns rows q_starts[s] .. q_starts[s + 1] - 1 (q_starts int32 [S + 1]; None: one
    query per sequence), its newest positions; max_q_len >= the most queries of one sequence.
    softcap > 0: scores softcap * tanh(score / softcap).  slopes [H_q]: - slopes[h] * distance is added.
    window > 0: the last `window` positions only.  prefix_lens int32 [S]: the first positions are seen by all queries.
    workspace: new_workspace(attend_workspace_bytes(...)), not shared by calls that may overlap.
    """
    return _attend(out, q, k_cache, v_cache, block_tables, seq_lens, q_starts, max_q_len, num_kv_heads, scale,
                   block_size, workspace, k_scale, v_scale, k_zero_point, v_zero_point, softcap, slopes, window,
                   prefix_lens, None, None, pdl, stream)


def attend_tree(out, q, k_cache, v_cache, block_tables, seq_lens, q_starts, max_q_len, tree_mask, num_kv_heads, scale,
                block_size, *, workspace=None, k_scale=None, v_scale=None, k_zero_point=None, v_zero_point=None,
                softcap=0.0, pdl=False, stream=None):
    """Attention of the nodes of drafted trees, whose rows are already in the cache (pa_attend with tree_mask).

    The L queries of a sequence are its tree's nodes, cached at positions T - L .. T - 1.  Node i sees the context
    before T - L and the nodes whose bits are set in its row of tree_mask (int64 words [N, W], bit j % 64 of word
    j // 64 for node j; the node's own bit is not implied).
    """
    if tree_mask is None:
        raise ValueError("attend_tree needs tree_mask")
    return _attend(out, q, k_cache, v_cache, block_tables, seq_lens, q_starts, max_q_len, num_kv_heads, scale,
                   block_size, workspace, k_scale, v_scale, k_zero_point, v_zero_point, softcap, None, 0, None,
                   tree_mask, None, pdl, stream)


def attend_accumulate(out, q, k_cache, v_cache, block_tables, seq_lens, mass, num_kv_heads, scale, block_size, *,
                      workspace=None, k_scale=None, v_scale=None, k_zero_point=None, v_zero_point=None, softcap=0.0,
                      slopes=None, window=0, prefix_lens=None, pdl=False, stream=None):
    """One decode step (q [S, H_q, d]) that also adds each position's attention weight, summed over the KV head's
    query heads, to mass[s, kv_head, position] (float32; pa_attend with the mass option)."""
    if mass is None:
        raise ValueError("attend_accumulate needs mass")
    return _attend(out, q, k_cache, v_cache, block_tables, seq_lens, None, 1, num_kv_heads, scale, block_size,
                   workspace, k_scale, v_scale, k_zero_point, v_zero_point, softcap, slopes, window, prefix_lens, None,
                   mass, pdl, stream)


def commit_tree(k_cache, v_cache, block_tables, seq_lens, q_starts, path, path_lens, new_lens, block_size, *,
                stream=None):
    """Move the accepted path's cache rows (nodes path[s, :path_lens[s]]) to the front of each tree's span and write
    the sequences' new lengths (pa_commit_tree).  Returns new_lens.

    A decode with pdl reads its lengths before the kernels just before it have finished: launch the cache write
    between this call and it without pdl.
    """
    _torch or _t()
    dev = _on_one_device(k_cache, v_cache, block_tables, seq_lens, q_starts, path, path_lens, new_lens)
    blocks, Hkv, D = _cache(k_cache, v_cache, block_size)
    S = seq_lens.shape[0]
    seqs = (S,)
    width, deep = _table("block_tables", block_tables, S, _I32), _table("path", path, S, _I32)
    _need("seq_lens", seq_lens, _I32, seqs)
    _need("q_starts", q_starts, _I32, (S + 1,))
    _need("path_lens", path_lens, _I32, seqs)
    _need("new_lens", new_lens, _I32, seqs)
    _issue(load().pa_commit_tree, dev, stream, k_cache.data_ptr(), v_cache.data_ptr(), _code(k_cache), blocks,
           block_tables.data_ptr(), width, seq_lens.data_ptr(), q_starts.data_ptr(), path.data_ptr(),
           path_lens.data_ptr(), deep, new_lens.data_ptr(), S, Hkv, D, int(block_size))
    return new_lens


def evict(k_cache, v_cache, mass, block_tables, seq_lens, dst_tables, kept, mass_out, new_lens, block_size, *, budget,
          recent=0, sinks=0, stream=None):
    """Cut sequences longer than `budget` back to it: per KV head the first `sinks`, the last `recent` and the heaviest
    other positions move, in order, to the blocks of dst_tables (pa_evict).

    Writes kept int32 / mass_out float32 [S, H_kv, budget] and new_lens int32 [S].  dst_tables must name fresh blocks.
    Returns kept.
    """
    _torch or _t()
    dev = _on_one_device(k_cache, v_cache, mass, block_tables, seq_lens, dst_tables, kept, mass_out, new_lens)
    blocks, Hkv, D = _cache(k_cache, v_cache, block_size)
    S = seq_lens.shape[0]
    seqs, lists = (S,), (S, Hkv, budget)
    width, dst_width = _table("block_tables", block_tables, S, _I32), _table("dst_tables", dst_tables, S, _I32)
    _need("seq_lens", seq_lens, _I32, seqs)
    _need("kept", kept, _I32, lists)
    _need("mass_out", mass_out, _F32, lists)
    _need("new_lens", new_lens, _I32, seqs)
    mseq, mhead = _mass_strides("mass", mass, S, Hkv)
    if mass.shape[2] < width * block_size:
        raise ValueError("mass rows must hold block_tables.shape[1] * block_size positions")
    _issue(load().pa_evict, dev, stream, k_cache.data_ptr(), v_cache.data_ptr(), _code(k_cache), blocks, mass.data_ptr(),
           mseq, mhead, block_tables.data_ptr(), width, seq_lens.data_ptr(), dst_tables.data_ptr(), dst_width,
           kept.data_ptr(), mass_out.data_ptr(), new_lens.data_ptr(), S, Hkv, D, int(block_size), int(budget), int(recent), int(sinks))
    return kept
