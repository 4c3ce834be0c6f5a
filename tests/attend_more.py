"""Attend cases with sinks and with 4-bit caches: AttendCase (operator_cases) with both, and the call that runs them.

A 4-bit value is code * scale + zero.  In calls of few rows (at most 64 rows of queries x query heads per KV head, on the
decode kernel) the codes enter the products exactly, and the weights, times the row's scale, as two float16 values: 22 bits,
as AttendCase.tolerance has it.  But the codes' part and the zeros' part of an output are summed apart and may cancel: each
is at most R = 3 times the largest value (zero is the row's smallest value, code * scale at most the difference to the
largest).  The first is off by 2^-22 R for its weights; either by 2^-23 R for each addition to its accumulator (the tensor
cores cut off, two products per 16 positions; a float32 addition per 8), of which there are at most min(T, 2048) / 8 in a
warp: longer sequences are split over the device, here to shares far below that.  With one query per sequence and a bfloat16
output a scaled weight is one float16 value: 2^-11 R, a quarter of the output's own half step for values near R.

In calls of many rows K and V are rounded to float16 once: half a step, 2^-11 of a value, at most.  A score then is off by
the sum of 128 independent errors q_i k_i 2^-11, uniform: a standard deviation of 2^-11 / sqrt(3) * sqrt(sum q_i^2 k_i^2) /
sqrt(128), about 2.9e-4 for standard normal q and k; six of these in the score, and twice that in a weight, relative to it.
"""

from __future__ import annotations

import torch

import int4_cases
from operator_cases import DT, F64, HALF_STEP, AttendCase, to_gpu


class Case(AttendCase):
    def __init__(self, lens, qlens, *, kv="bf16", q="bf16", heads=8, kv_heads=2, dim=128, block=16, seed=0, window=0, sinks=0,
                 **kw):
        four = kv == "i4"
        super().__init__(lens, qlens, kv="e4m3" if four else kv, q=q, heads=heads, kv_heads=kv_heads, dim=dim, block=block,
                         seed=seed, **kw)
        self.window, self.sinks = window, sinks
        if four:
            self.kv = "i4"
            self.k_scale = self.v_scale = None
            self.k, self.k64 = int4_cases.make_pool(self.blocks, kv_heads, block, self.g)
            self.v, self.v64 = int4_cases.make_pool(self.blocks, kv_heads, block, self.g)

    def visible(self, s, i):
        see = super().visible(s, i)
        if self.window and self.sinks:
            t, pos = torch.arange(self.lens[s]), self.lens[s] - self.qlens[s] + i
            if pos >= 0:
                see = see | ((t < self.sinks) & (t <= pos))
        return see

    def used(self):
        """[blocks, B]: rows that some query of their sequence sees."""
        used = torch.zeros((self.blocks, self.block), dtype=torch.bool)
        for s, t in enumerate(self.lens):
            see = torch.zeros(t, dtype=torch.bool)
            for i in range(self.qlens[s]):
                see |= self.visible(s, i)
            for p in see.nonzero()[:, 0].tolist():
                b, r = self.row_of(s, p)
                used[b, r] = True
        return used

    def spoil(self):
        """Everything that no query sees: NaN (in a 4-bit row's pair; int8 has none); entries of unseen blocks: -1."""
        used = self.used()
        for c in (self.k, self.v):
            if self.kv == "i4":
                pairs = c[..., self.block * 64:].view(torch.float16).view(self.blocks, self.kv_heads, self.block, 2)
                pairs[~used[:, None, :].expand(-1, self.kv_heads, -1)] = float("nan")
            elif self.kv != "i8":
                spoiled = torch.where(used[:, None, :, None], c.float(), torch.full((), float("nan"))).to(c.dtype)
                c.view(torch.uint8).copy_(spoiled.view(torch.uint8))
        self.tables_given = self.tables.clone()
        blocks = used.any(-1)
        for s in range(len(self.lens)):
            for j in range(self.tables.shape[1]):
                if self.tables[s, j] >= 0 and not blocks[self.tables[s, j]]:
                    self.tables_given[s, j] = -1

    def tolerance(self, out_fmt, ref, wabs):
        tol = super().tolerance(out_fmt, ref, wabs)
        if self.kv != "i4":
            return tol
        group = self.heads // self.kv_heads
        mult = max(1.0, float(self.q.float().abs().max()) / 4.5)
        if max(self.qlens) * group <= 16:                  # always on the decode kernel
            steps = 1 + 2 * min(max(self.lens), 2048) // 8
            weight = 2.0 ** -11 if out_fmt == "bf16" and max(self.qlens) == 1 else 2.0 ** -22
            return tol + (weight + steps * 2.0 ** -23) * 3 * float(self.v64.abs().max())
        return tol + (2 * 6 * 2.9e-4 * mult + 2.0 ** -11) * wabs


def run(case, out_fmt="f32", *, mass=None, workspace=None, stream=None, pdl=False, fill=7.0):
    import paged_kv_cache_144_gb300 as pa
    q = case.q_wide.cuda()[:, :case.heads]
    k, v = case.k.cuda(), case.v.cuda()
    out = torch.full((case.rows, case.heads, case.dim), fill, dtype=DT[out_fmt], device="cuda")
    tables, lens = getattr(case, "tables_given", case.tables).cuda(), case.lens_t.cuda()
    max_q = max(case.qlens)
    if workspace is None:
        workspace = pa.new_workspace(pa.attend_workspace_bytes(
            len(case.lens), case.heads, case.kv_heads, case.dim, case.block, case.tables.shape[1], max_q,
            pa.cache_dtype_code(k), accumulate=mass is not None), "cuda")
    kw = dict(workspace=workspace, k_scale=to_gpu(case.k_scale), v_scale=to_gpu(case.v_scale), k_zero_point=to_gpu(case.k_zp),
              v_zero_point=to_gpu(case.v_zp), softcap=case.softcap, pdl=pdl, stream=stream)
    more = dict(slopes=to_gpu(case.slopes), window=case.window, sinks=case.sinks, prefix_lens=to_gpu(case.prefix))
    if mass is not None:
        pa.attend_accumulate(out, q, k, v, tables, lens, mass, case.kv_heads, case.scale, case.block, **kw, **more)
    elif case.tree is not None:
        pa.attend_tree(out, q, k, v, tables, lens, case.starts.cuda(), max_q, case.tree.cuda(), case.kv_heads, case.scale,
                       case.block, **kw)
    else:
        pa.attend(out, q, k, v, tables, lens, case.starts.cuda(), max_q, case.kv_heads, case.scale, case.block, **kw, **more)
    if stream is not None:
        stream.synchronize()
    err = pa.get_device_error()
    return out.cpu().to(F64), err


def check(case, out_fmt="f32", spoil=True, **kw):
    if spoil:
        case.spoil()
    got, err = run(case, out_fmt, **kw)
    ref, wabs, mass = case.reference()
    n = sum(case.qlens)
    assert err == 0, f"device error bits {err}"
    assert torch.all(got[n:] == 7.0), "rows behind the last sequence were written"
    tol = case.tolerance(out_fmt, ref, wabs)
    bad = ~((got[:n] - ref[:n]).abs() <= tol[:n])
    assert not bad.any(), (f"{int(bad.sum())} of {bad.numel()} outputs off, worst {(got[:n] - ref[:n]).abs().max():.3e} "
                           f"(bound there {tol[:n].flatten()[(got[:n] - ref[:n]).abs().argmax()]:.3e}), first at "
                           f"{bad.nonzero()[0].tolist()}")
    return got, ref, mass
