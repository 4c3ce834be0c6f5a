"""4-bit cache tiles on the host, in plain Python and torch: tile bytes of given codes and pairs, and back.

A tile of B rows of d values: per row d / 2 bytes of codes, then per row (scale, zero) as float16.  Word w of a row's codes
holds values 8 w .. 8 w + 7, value 8 w + 2 j + e in bits 16 e + 4 j.
"""

from __future__ import annotations

import torch

F64 = torch.float64


def _place(d):
    """(byte of the row, shift within the byte) of each value."""
    i = torch.arange(d)
    bit = 16 * (i % 2) + 4 * (i % 8 // 2)
    return 4 * (i // 8) + bit // 8, bit % 8


def pack(codes, scale, zero):
    """uint8 [..., B * (d / 2 + 4)] of codes [..., B, d] and float16 pairs [..., B]."""
    *lead, b, d = codes.shape
    at, shift = _place(d)
    row = torch.zeros((*lead, b, d // 2), dtype=torch.int32)
    row.index_add_(row.dim() - 1, at, codes.to(torch.int32) << shift.to(torch.int32))
    pairs = torch.stack((scale.half(), zero.half()), -1).contiguous().view(torch.uint8)
    return torch.cat((row.to(torch.uint8).reshape(*lead, -1), pairs.reshape(*lead, -1)), -1)


def unpack(tiles, block, d=128):
    """(codes int64 [..., B, d], scale, zero float64 [..., B])."""
    lead = tiles.shape[:-1]
    at, shift = _place(d)
    rows = tiles[..., :block * d // 2].reshape(*lead, block, d // 2)
    codes = (rows[..., at].to(torch.int64) >> shift) & 15
    pairs = tiles[..., block * d // 2:].contiguous().view(torch.float16).reshape(*lead, block, 2).to(F64)
    return codes, pairs[..., 0], pairs[..., 1]


def values(tiles, block, d=128):
    codes, scale, zero = unpack(tiles, block, d)
    return codes.to(F64) * scale[..., None] + zero[..., None]


def make_pool(blocks, heads, block, g, spread=1.0, shift=0.0):
    """(tiles, float64 values) of standard normal rows, quantised by the smallest and largest of each row."""
    x = torch.randn((blocks, heads, block, 128), generator=g) * spread + shift
    zero = x.amin(-1).half()
    scale = ((x.amax(-1) - zero.float()) / 15).half()
    codes = ((x - zero.float()[..., None]) / scale.float()[..., None]).round().clamp(0, 15)
    tiles = pack(codes, scale, zero)
    return tiles, values(tiles, block)


def check_rows(tiles, block, slots, want, slack):
    """Rows at `slots` of a pool [blocks, H, tile] hold `want` [N, H, d] (float64, off by at most `slack` [N, H, 1] where
    they were computed in float32): the pair is the row's bounds rounded to float16, every code the nearest one.

    zero: the smallest value, off by slack, rounded by half a float16 step (2^-11 of it; 2^-25 below the normal numbers).
    scale: (largest - zero) / 15 of the stored zero, off by slack / 15 and two float32 roundings, rounded likewise.  A code is
    the nearest to (x - zero) / scale: off by 1/2, by slack / scale and by three roundings of a quotient of at most 15.
    """
    blk, off = slots // block, slots % block
    codes, scale, zero = unpack(tiles, block)
    codes, scale, zero = codes[blk, :, off].to(F64), scale[blk, :, off], zero[blk, :, off]
    lo, hi, slack1 = want.amin(-1), want.amax(-1), slack[..., 0]
    half = lambda x: 2.0 ** -11 * x.abs() + 2.0 ** -25  # noqa: E731
    assert torch.all((zero - lo).abs() <= slack1 + half(lo))
    ideal = ((hi - zero) / 15).clamp(min=0)
    assert torch.all((scale - ideal).abs() <= slack1 / 15 + 2.0 ** -22 * (hi.abs() + zero.abs()) / 15 + half(ideal))
    flat = scale == 0
    assert torch.all(codes[flat] == 0)
    y = ((want - zero[..., None]) / torch.where(flat, torch.ones_like(scale), scale)[..., None]).clamp(0, 15)
    near = 0.5 + slack / torch.where(flat, torch.ones_like(scale), scale)[..., None] + 15 * 3 * 2.0 ** -23
    near = near + 2.0 ** -23 * (want.abs() + zero.abs()[..., None]) / torch.where(flat, torch.ones_like(scale), scale)[..., None]
    bad = ((codes - y).abs() > near) & ~flat[..., None]
    assert not bad.any(), (codes - y).abs().max()
