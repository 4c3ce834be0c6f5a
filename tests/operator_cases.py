"""Inputs and plain 64-bit implementations for the tests of the operators around the cache.

Everything here works from the definitions in include/pa.h on host tensors, one query row at a time; it shares no code
with the library.
"""

from __future__ import annotations

import math

import torch

F64 = torch.float64
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn,
      "i8": torch.int8}
HALF_STEP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def tables_for(lens, block, g, spare=3, width=None):
    """Random physical blocks for every sequence; unused entries are -1.  Returns (tables, number of blocks)."""
    need = [-(-t // block) for t in lens]
    n = sum(need) + spare
    perm = torch.randperm(n, generator=g).to(torch.int32)
    width = max(max(need), 1) if width is None else width
    out = torch.full((len(lens), width), -1, dtype=torch.int32)
    at = 0
    for s, m in enumerate(need):
        out[s, :m] = perm[at:at + m]
        at += m
    return out, n


def make_cache(kv, blocks, heads, block, dim, g):
    """(codes in the cache type, float64 values, scale, zero point)."""
    x = torch.randn((blocks, heads, block, dim), generator=g)
    if kv in ("f16", "bf16"):
        c = x.to(DT[kv])
        return c, c.to(F64), None, None
    scale = 0.02 + 0.02 * torch.rand(heads, generator=g)
    if kv == "e4m3":
        c = (x / scale.view(1, -1, 1, 1)).clamp(-448, 448).to(DT[kv])
        return c, c.to(F64) * scale.to(F64).view(1, -1, 1, 1), scale, None
    zp = torch.randint(-30, 31, (heads,), generator=g, dtype=torch.int32)
    c = ((x / scale.view(1, -1, 1, 1)).round() + zp.view(1, -1, 1, 1)).clamp(-128, 127).to(torch.int8)
    return c, (c.to(F64) - zp.to(F64).view(1, -1, 1, 1)) * scale.to(F64).view(1, -1, 1, 1), scale, zp


class AttendCase:
    """One attend call: ragged queries of sequences `lens` with `qlens` queries each."""

    def __init__(self, lens, qlens, *, kv="bf16", q="bf16", heads=8, kv_heads=2, dim=128, block=16, seed=0, pad_rows=2,
                 q_mult=1.0, q_pad=0, width=None):
        g = torch.Generator().manual_seed(seed)
        self.g = g
        if kv in ("f16", "bf16"):
            q = kv
        self.lens, self.qlens, self.kv, self.qt = list(lens), list(qlens), kv, q
        self.heads, self.kv_heads, self.dim, self.block = heads, kv_heads, dim, block
        self.scale = 1.0 / math.sqrt(dim)
        self.tables, self.blocks = tables_for(lens, block, g, width=width)
        self.k, self.k64, self.k_scale, self.k_zp = make_cache(kv, self.blocks, kv_heads, block, dim, g)
        self.v, self.v64, self.v_scale, self.v_zp = make_cache(kv, self.blocks, kv_heads, block, dim, g)
        self.rows = sum(qlens) + pad_rows
        wide = torch.randn((self.rows, heads + q_pad, dim), generator=g) * q_mult
        self.q_wide = wide.to(DT[q])                 # q is a strided view when q_pad > 0
        self.q = self.q_wide[:, :heads]
        self.starts = torch.tensor([0] + list(torch.tensor(qlens).cumsum(0)), dtype=torch.int32)
        self.lens_t = torch.tensor(lens, dtype=torch.int32)
        self.slopes = self.prefix = self.tree = None
        self.window, self.softcap = 0, 0.0

    def spoil_tails(self, value=float("nan")):
        """What lies past every sequence's end, and in blocks of nobody, must not matter (16-bit and FP8 caches)."""
        used = torch.zeros((self.blocks, self.block), dtype=torch.bool)
        for s, t in enumerate(self.lens):
            for p in range(t):
                used[int(self.tables[s, p // self.block]), p % self.block] = True
        for c in (self.k, self.v):
            spoiled = torch.where(used[:, None, :, None], c.float(), torch.full((), value)).to(c.dtype)
            c.view(torch.uint8).copy_(spoiled.view(torch.uint8))

    def row_of(self, s, t):
        return int(self.tables[s, t // self.block]), t % self.block

    def with_tree(self, words=None, parents=8, selfless=False):
        words = words or max(1, -(-max(self.qlens) // 64))
        bits = torch.zeros((self.rows, words), dtype=torch.int64)
        self.ancestors = []
        n = 0
        for L in self.qlens:
            anc = []
            for i in range(L):
                par = -1 if i == 0 else int(torch.randint(max(-1, i - parents), i, (1,), generator=self.g))
                anc.append(([] if par < 0 else anc[par]) + ([] if selfless else [i]))
                for j in anc[i]:
                    w = int(bits[n, j // 64]) & ((1 << 64) - 1) | 1 << (j % 64)
                    bits[n, j // 64] = w - (1 << 64) if w >= 1 << 63 else w
                n += 1
            self.ancestors.append(anc)
        self.tree = bits
        return self

    def visible(self, s, i):
        """Boolean [T]: what query i of sequence s sees."""
        T, L = self.lens[s], self.qlens[s]
        pos, t = T - L + i, torch.arange(self.lens[s])
        if pos < 0:
            return torch.zeros(T, dtype=torch.bool)
        if self.tree is not None:
            see = t < T - L
            for j in self.ancestors[s][i]:
                if T - L + j >= 0:
                    see[T - L + j] = True
            return see
        see = t <= pos
        if self.window:
            see &= t > pos - self.window
        if self.prefix is not None:
            see |= t < int(self.prefix[s])
        return see

    def reference(self):
        """(out, sum of p |v|, weights mass [S, H_kv, width*block]) in float64."""
        G = self.heads // self.kv_heads
        out = torch.zeros((self.rows, self.heads, self.dim), dtype=F64)
        wabs = torch.zeros_like(out)
        mass = torch.zeros((len(self.lens), self.kv_heads, self.tables.shape[1] * self.block), dtype=F64)
        n = 0
        for s, (T, L) in enumerate(zip(self.lens, self.qlens)):
            blk = torch.tensor([self.row_of(s, t) for t in range(T)], dtype=torch.long).view(-1, 2)
            K = self.k64[blk[:, 0], :, blk[:, 1]]            # [T, H_kv, d]
            V = self.v64[blk[:, 0], :, blk[:, 1]]
            for i in range(L):
                see = self.visible(s, i)
                if see.any():
                    idx = see.nonzero()[:, 0]
                    pos = T - L + i
                    for h in range(self.heads):
                        z = K[idx, h // G] @ self.q[n, h].to(F64) * self.scale
                        if self.softcap:
                            z = self.softcap * torch.tanh(z / self.softcap)
                        if self.slopes is not None:
                            z = z - float(self.slopes[h]) * (idx - pos).abs().to(F64)
                        p = torch.softmax(z, 0)
                        out[n, h] = p @ V[idx, h // G]
                        wabs[n, h] = p @ V[idx, h // G].abs()
                        mass[s, h // G, idx] += p
                n += 1
        return out, wabs, mass

    def tolerance(self, out_fmt, ref, wabs):
        """Bound on the error of one output.

        Scores are float32 sums of d <= 128 products: each is off by at most 128 steps of 2^-23 of the sum of the
        products' magnitudes, about 8 for the standard normal inputs here (8 * q_mult): an absolute error of 1.3e-4
        in the score, a relative one of e in its weight, and of 2e after the division by their sum.  A weight enters
        its product rounded to 16 bits (its half step), or as two such parts when the output is float32.  The output
        is rounded to its type once.
        """
        mult = max(1.0, float(self.q.float().abs().max()) / 4.5)
        e = 2 * 1.3e-4 * mult
        w = 2.0 ** -11 if self.kv != "bf16" else 2.0 ** -8
        if out_fmt == "f32":
            w = w * w
        return (e + w) * wabs + HALF_STEP[out_fmt] * ref.abs() + 1e-7


def to_gpu(t):
    return None if t is None else t.cuda()


def run_attend(case, out_fmt="f32", *, mass=None, workspace=None, stream=None, use_starts=True, pdl=False, fill=7.0):
    """The library's answer for a case: (out float64 on the host, device error bits)."""
    import paged_kv_cache_144_gb300 as pa
    q = case.q_wide.cuda()[:, :case.heads]
    k, v = case.k.cuda(), case.v.cuda()
    out = torch.full((case.rows, case.heads, case.dim), fill, dtype=DT[out_fmt], device="cuda")
    tables, lens = case.tables.cuda(), case.lens_t.cuda()
    max_q = max(case.qlens)
    if workspace is None:
        workspace = pa.new_workspace(pa.attend_workspace_bytes(
            len(case.lens), case.heads, case.kv_heads, case.dim, case.block, case.tables.shape[1], max_q,
            pa.dtype_code(k), accumulate=mass is not None), "cuda")
    kw = dict(workspace=workspace, k_scale=to_gpu(case.k_scale), v_scale=to_gpu(case.v_scale),
              k_zero_point=to_gpu(case.k_zp), v_zero_point=to_gpu(case.v_zp), softcap=case.softcap, pdl=pdl,
              stream=stream)
    if mass is not None:
        pa.attend_accumulate(out, q, k, v, tables, lens, mass, case.kv_heads, case.scale, case.block,
                             slopes=to_gpu(case.slopes), window=case.window, prefix_lens=to_gpu(case.prefix), **kw)
    elif case.tree is not None:
        pa.attend_tree(out, q, k, v, tables, lens, case.starts.cuda(), max_q, case.tree.cuda(), case.kv_heads,
                       case.scale, case.block, **kw)
    else:
        pa.attend(out, q, k, v, tables, lens, case.starts.cuda() if use_starts else None, max_q, case.kv_heads,
                  case.scale, case.block, slopes=to_gpu(case.slopes), window=case.window,
                  prefix_lens=to_gpu(case.prefix), **kw)
    err = pa.get_device_error()
    return out.cpu().to(F64), err


def check_attend(case, out_fmt="f32", spoil=True, **kw):
    if spoil and case.kv != "i8":
        case.spoil_tails()
    got, err = run_attend(case, out_fmt, **kw)
    ref, wabs, mass = case.reference()
    n = sum(case.qlens)
    assert err == 0, f"device error bits {err}"
    assert torch.all(got[n:] == 7.0), "rows behind the last sequence were written"
    tol = case.tolerance(out_fmt, ref, wabs)
    bad = ~((got[:n] - ref[:n]).abs() <= tol[:n])
    assert not bad.any(), (f"{int(bad.sum())} of {bad.numel()} outputs off, worst "
                           f"{(got[:n] - ref[:n]).abs().max():.3e}, first at {bad.nonzero()[0].tolist()}")
    return got, ref, mass


# ------------------------------------------------------------------------------------------------ rotary positions

def rope_reference(x, positions, inv_freq, interleaved, scale):
    """[N, H, d] float64: columns turned pair by pair."""
    r2 = inv_freq.numel()
    y = x.to(F64).clone()
    a = positions.to(F64)[:, None] * inv_freq.to(F64)[None]
    c, s = (torch.cos(a) * scale)[:, None], (torch.sin(a) * scale)[:, None]
    i = torch.arange(r2)
    lo, hi = (2 * i, 2 * i + 1) if interleaved else (i, i + r2)
    p, q = x.to(F64)[..., lo], x.to(F64)[..., hi]
    y[..., lo] = p * c - q * s
    y[..., hi] = q * c + p * s
    return y


# ------------------------------------------------------------------------------------------------ eviction

def kept_positions(mass, T, budget, recent, sinks):
    """Ascending kept positions of one (sequence, head) from the definition."""
    if T <= budget:
        return list(range(T))
    always = set(range(sinks)) | set(range(T - recent, T))
    middle = [t for t in range(T) if t not in always]
    weight = [(-math.inf if math.isnan(float(mass[t])) else float(mass[t]), math.isnan(float(mass[t]))) for t in range(T)]
    middle.sort(key=lambda t: (weight[t][1], -weight[t][0], t))
    return sorted(always | set(middle[:budget - sinks - recent]))
