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

_torch = None


def _t():
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    return _torch


def _device_of(first, named, stream):
    """The one device of all tensors; a (device guard or None, stream handle) pair for the call."""
    torch = _t()
    if not first.is_cuda:
        raise ValueError("q/k_cache must be a CUDA tensor")
    dev = first.device
    for name, t in named:
        if t is not None and t.device != dev:
            raise ValueError(f"{name} must be on {dev}, the device of the call's other tensors")
    if stream is not None:
        if stream.device != dev:
            raise ValueError(f"stream must be on {dev}")
        handle = stream.cuda_stream
    else:
        handle = torch.cuda.current_stream(dev).cuda_stream
    guard = None if dev.index == torch.cuda.current_device() else torch.cuda.device(dev)
    return guard, handle


def _call(fn, guard, *args):
    if guard is None:
        _check(fn.__name__, fn(*args))
    else:
        with guard:
            _check(fn.__name__, fn(*args))


def _need(name, t, dtype, *shape):
    """A contiguous tensor of this dtype of exactly these sizes (None: any)."""
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
    if t.dim() != len(shape) or any(w is not None and n != w for n, w in zip(t.shape, shape)):
        raise ValueError(f"{name} must have shape {shape}, not {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _rows(name, t, heads, dim):
    """[N, heads, dim] with contiguous rows; returns the stride between tokens."""
    if t.dim() != 3 or t.shape[1] != heads or t.shape[2] != dim:
        raise ValueError(f"{name} must have shape [N, {heads}, {dim}], not {tuple(t.shape)}")
    if t.stride(2) != 1 or t.stride(1) != dim:
        raise ValueError(f"{name} rows must be contiguous per token")
    return t.stride(0) if t.shape[0] > 1 else max(t.stride(0), heads * dim)


def _cache(k_cache, v_cache, num_kv_heads, block_size):
    if (k_cache.dim() != 4 or k_cache.shape[1] != num_kv_heads or k_cache.shape[2] != block_size or
            not k_cache.is_contiguous()):
        raise ValueError(f"k_cache must be contiguous [blocks, {num_kv_heads}, {block_size}, d], not "
                         f"{tuple(k_cache.shape)}")
    if v_cache.shape != k_cache.shape or v_cache.dtype != k_cache.dtype or not v_cache.is_contiguous():
        raise ValueError("v_cache must be contiguous, of the shape and type of k_cache")


def _heads_params(num_kv_heads, **named):
    torch = _t()
    for name, t in named.items():
        if t is not None:
            _need(name, t, torch.int32 if "zero" in name else torch.float32, num_kv_heads)


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
    are padding and left alone.  Returns q_out.
    """
    torch = _t()
    if q_out is None:
        q_out = q
    guard, handle = _device_of(q, (("k", k), ("v", v), ("k_cache", k_cache), ("v_cache", v_cache),
                                   ("positions", positions), ("slot_mapping", slot_mapping), ("inv_freq", inv_freq),
                                   ("q_out", q_out), ("k_inv_scale", k_inv_scale), ("v_inv_scale", v_inv_scale),
                                   ("k_zero_point", k_zero_point), ("v_zero_point", v_zero_point)), stream)
    N, Hq, D = q.shape
    Hkv = k.shape[1]
    _cache(k_cache, v_cache, Hkv, block_size)
    if k_cache.shape[3] != D or k.shape[0] != N or v.shape[0] != N or q_out.shape[0] != N:
        raise ValueError("q, k, v, q_out and the caches must agree in tokens and head size")
    if k.dtype != q.dtype or v.dtype != q.dtype or q_out.dtype != q.dtype:
        raise ValueError("q, k, v and q_out must have one type")
    qs, qos = _rows("q", q, Hq, D), _rows("q_out", q_out, Hq, D)
    ks, vs = _rows("k", k, Hkv, D), _rows("v", v, Hkv, D)
    _need("positions", positions, torch.int64, N)
    _need("slot_mapping", slot_mapping, torch.int64, N)
    _need("inv_freq", inv_freq, torch.float32, None)
    _heads_params(Hkv, k_inv_scale=k_inv_scale, v_inv_scale=v_inv_scale, k_zero_point=k_zero_point,
                  v_zero_point=v_zero_point)
    opt = None
    if k_zero_point is not None or v_zero_point is not None or pdl:
        opt = ctypes.byref(CacheWriteOptions(k_zero_point=_ptr(k_zero_point), v_zero_point=_ptr(v_zero_point),
                                             pdl=1 if pdl else 0))
    _call(load().pa_rope_and_cache, guard, q_out.data_ptr(), qos, q.data_ptr(), qs, Hq, k.data_ptr(), v.data_ptr(),
          dtype_code(q), ks, vs, k_cache.data_ptr(), v_cache.data_ptr(), dtype_code(k_cache), k_cache.shape[0],
          positions.data_ptr(), slot_mapping.data_ptr(), inv_freq.data_ptr(), 2 * inv_freq.shape[0],
          1 if interleaved else 0, float(rope_scale), N, Hkv, D, int(block_size), _ptr(k_inv_scale),
          _ptr(v_inv_scale), opt, handle)
    return q_out


def attend_workspace_bytes(num_seqs, num_heads, num_kv_heads, head_dim, block_size, max_blocks_per_seq, max_q_len,
                           kv_dtype=_lib.PA_BF16, accumulate=False) -> int:
    """Workspace of attend / attend_tree / attend_accumulate (accumulate=True) for these sizes on the current device."""
    n = int(load().pa_attend_workspace_bytes(num_seqs, num_heads, num_kv_heads, head_dim, block_size,
                                             max_blocks_per_seq, max_q_len, kv_dtype, 1 if accumulate else 0))
    if n == SIZE_MAX:
        raise PagedAttnError("pa_attend_workspace_bytes", PA_ERR_SHAPE, "sizes rejected or no usable device")
    return n


def _attend(out, q, k_cache, v_cache, block_tables, seq_lens, q_starts, max_q_len, num_kv_heads, scale, block_size,
            workspace, k_scale, v_scale, k_zero_point, v_zero_point, softcap, slopes, window, prefix_lens, tree_mask,
            mass, pdl, stream):
    torch = _t()
    guard, handle = _device_of(q, (("out", out), ("k_cache", k_cache), ("v_cache", v_cache),
                                   ("block_tables", block_tables), ("seq_lens", seq_lens), ("q_starts", q_starts),
                                   ("workspace", workspace), ("k_scale", k_scale), ("v_scale", v_scale),
                                   ("k_zero_point", k_zero_point), ("v_zero_point", v_zero_point), ("slopes", slopes),
                                   ("prefix_lens", prefix_lens), ("tree_mask", tree_mask), ("mass", mass)), stream)
    N, Hq, D = q.shape
    qs = _rows("q", q, Hq, D)
    _cache(k_cache, v_cache, num_kv_heads, block_size)
    if k_cache.shape[3] != D:
        raise ValueError("q and the caches must have one head size")
    if out.shape != q.shape or not out.is_contiguous():
        raise ValueError(f"out must be contiguous of shape {tuple(q.shape)}")
    S = seq_lens.shape[0]
    _need("block_tables", block_tables, torch.int32, S, None)
    _need("seq_lens", seq_lens, torch.int32, S)
    if q_starts is not None:
        _need("q_starts", q_starts, torch.int32, S + 1)
    _heads_params(num_kv_heads, k_scale=k_scale, v_scale=v_scale, k_zero_point=k_zero_point, v_zero_point=v_zero_point)
    ws, wb = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel() * workspace.element_size())
    words = mseq = mhead = 0
    if slopes is not None:
        _need("slopes", slopes, torch.float32, Hq)
    if prefix_lens is not None:
        _need("prefix_lens", prefix_lens, torch.int32, S)
    if tree_mask is not None:
        if tree_mask.dtype not in (torch.int64, getattr(torch, "uint64", torch.int64)):
            raise ValueError("tree_mask must be int64 (or uint64) words")
        _need("tree_mask", tree_mask, tree_mask.dtype, N, None)
        words = tree_mask.shape[1]
    if mass is not None:
        mseq, mhead = _mass_strides("mass", mass, S, num_kv_heads)
        if mass.shape[2] < block_tables.shape[1] * block_size:
            raise ValueError("mass rows must hold block_tables.shape[1] * block_size positions")
    opt = AttendOptions(k_zero_point=_ptr(k_zero_point), v_zero_point=_ptr(v_zero_point), softcap=float(softcap),
                        slopes=_ptr(slopes), window=int(window), prefix_lens=_ptr(prefix_lens),
                        tree_mask=_ptr(tree_mask), tree_words=words, mass=_ptr(mass), mass_stride_seq=mseq,
                        mass_stride_head=mhead, pdl=1 if pdl else 0)
    _call(load().pa_attend, guard, out.data_ptr(), dtype_code(out), q.data_ptr(), dtype_code(q), qs,
          k_cache.data_ptr(), v_cache.data_ptr(), dtype_code(k_cache), k_cache.shape[0], _ptr(k_scale), _ptr(v_scale),
          block_tables.data_ptr(), block_tables.shape[1], seq_lens.data_ptr(), _ptr(q_starts), int(max_q_len), N, S,
          Hq, int(num_kv_heads), D, float(scale), int(block_size), ws, wb, ctypes.byref(opt), handle)
    return out


def _mass_strides(name, mass, seqs, heads):
    if mass.dtype != _t().float32 or mass.dim() != 3 or mass.shape[0] != seqs or mass.shape[1] != heads:
        raise ValueError(f"{name} must be float32 [{seqs}, {heads}, positions], not {mass.dtype} {tuple(mass.shape)}")
    if mass.stride(2) != 1 and mass.shape[2] > 1:
        raise ValueError(f"{name} rows must be contiguous")
    h = mass.stride(1) if heads > 1 else max(mass.stride(1), mass.shape[2])
    return (mass.stride(0) if seqs > 1 else max(mass.stride(0), h * heads)), h


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
    the sequences' new lengths (pa_commit_tree).  Returns new_lens."""
    torch = _t()
    guard, handle = _device_of(k_cache, (("v_cache", v_cache), ("block_tables", block_tables), ("seq_lens", seq_lens),
                                         ("q_starts", q_starts), ("path", path), ("path_lens", path_lens),
                                         ("new_lens", new_lens)), stream)
    S = seq_lens.shape[0]
    Hkv, D = k_cache.shape[1], k_cache.shape[3]
    _cache(k_cache, v_cache, Hkv, block_size)
    _need("block_tables", block_tables, torch.int32, S, None)
    _need("seq_lens", seq_lens, torch.int32, S)
    _need("q_starts", q_starts, torch.int32, S + 1)
    _need("path", path, torch.int32, S, None)
    _need("path_lens", path_lens, torch.int32, S)
    _need("new_lens", new_lens, torch.int32, S)
    _call(load().pa_commit_tree, guard, k_cache.data_ptr(), v_cache.data_ptr(), dtype_code(k_cache), k_cache.shape[0],
          block_tables.data_ptr(), block_tables.shape[1], seq_lens.data_ptr(), q_starts.data_ptr(), path.data_ptr(),
          path_lens.data_ptr(), path.shape[1], new_lens.data_ptr(), S, Hkv, D, int(block_size), handle)
    return new_lens


def evict(k_cache, v_cache, mass, block_tables, seq_lens, dst_tables, kept, mass_out, new_lens, block_size, *, budget,
          recent=0, sinks=0, stream=None):
    """Cut sequences longer than `budget` back to it: per KV head the first `sinks`, the last `recent` and the heaviest
    other positions move, in order, to the blocks of dst_tables (pa_evict).

    Writes kept int32 / mass_out float32 [S, H_kv, budget] and new_lens int32 [S].  dst_tables must name fresh blocks.
    Returns kept.
    """
    torch = _t()
    guard, handle = _device_of(k_cache, (("v_cache", v_cache), ("mass", mass), ("block_tables", block_tables),
                                         ("seq_lens", seq_lens), ("dst_tables", dst_tables), ("kept", kept),
                                         ("mass_out", mass_out), ("new_lens", new_lens)), stream)
    S = seq_lens.shape[0]
    Hkv, D = k_cache.shape[1], k_cache.shape[3]
    _cache(k_cache, v_cache, Hkv, block_size)
    _need("block_tables", block_tables, torch.int32, S, None)
    _need("seq_lens", seq_lens, torch.int32, S)
    _need("dst_tables", dst_tables, torch.int32, S, None)
    _need("kept", kept, torch.int32, S, Hkv, budget)
    _need("mass_out", mass_out, torch.float32, S, Hkv, budget)
    _need("new_lens", new_lens, torch.int32, S)
    mseq, mhead = _mass_strides("mass", mass, S, Hkv)
    if mass.shape[2] < block_tables.shape[1] * block_size:
        raise ValueError("mass rows must hold block_tables.shape[1] * block_size positions")
    _call(load().pa_evict, guard, k_cache.data_ptr(), v_cache.data_ptr(), dtype_code(k_cache), k_cache.shape[0],
          mass.data_ptr(), mseq, mhead, block_tables.data_ptr(), block_tables.shape[1], seq_lens.data_ptr(),
          dst_tables.data_ptr(), dst_tables.shape[1], kept.data_ptr(), mass_out.data_ptr(), new_lens.data_ptr(), S,
          Hkv, D, int(block_size), int(budget), int(recent), int(sinks), handle)
    return kept
