"""Timing cases of a cache held in 4 bits and of what fills, bounds and reads it: queries and keys normalised for each
head and turned to their positions in the pass that writes the cache, attention over a 4-bit cache, attention with a
sliding window whose first tokens stay visible, and reading cached rows back as values.

`run(state)` is one pass through an operator.  With `own` false it is the operator's plain form: elementary torch
operations in 32 bits, rounded once at the end.  With `own` true it is the calls a user makes of the library.
`exact(case, seed)` is the same answer from the definition in 64 bits.

A 4-bit row of d values is d / 2 bytes of codes and a float16 pair (scale, zero); a value is code * scale + zero.  A
cache tile of one block and KV head holds the codes of its rows, then their pairs.  Word w of a row (32 bits, little
end first) holds values 8 w .. 8 w + 7: value 8 w + 2 j + e in bits 16 e + 4 j and up.
"""

import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn, "i8": torch.int8,
          "i4": torch.uint8, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "e4m3": 1, "i8": 1, "f32": 4}


# ------------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # --- norms of queries and keys, their positions and the cache write
        # one decode step of a 32-sequence batch (the latency that every layer of every step pays)
        dict(name="norm_step_32", kind="norm", q="bf16", kv="bf16", heads=32, kv_heads=8, dim=128, block=16, tokens=32,
             pos_max=4096, rotary=128, interleaved=False, weights="both"),
        # the prompts of several sequences written to a 4-bit cache at once, and their rows read back for the prompt's
        # own layers
        dict(name="norm_prompt_8k_int4", kind="norm", q="bf16", kv="i4", heads=32, kv_heads=8, dim=128, block=16,
             tokens=8192, pos_max=131072, rotary=128, interleaved=False, weights="both"),
        # an odd number of prompt tokens into an FP8 cache, half of each head turned, adjacent pairs, keys alone normed
        dict(name="norm_partial_fp8", kind="norm", q="f16", kv="e4m3", heads=32, kv_heads=8, dim=128, block=32,
             tokens=2049, pos_max=32768, rotary=64, interleaved=True, weights="k"),
        # --- attention over a 4-bit cache
        # a small batch of short contexts (the latency of a lightly loaded server)
        dict(name="int4_small", kind="attend", q="f16", kv="i4", heads=4, kv_heads=4, dim=128, block=16, seqs=4,
             len_lo=20, len_hi=300, q_lo=1, q_hi=1, window=0, sinks=0, lens_seed=51),
        # one decode step of a 32-sequence batch
        dict(name="int4_step_32x4k", kind="attend", q="bf16", kv="i4", heads=32, kv_heads=8, dim=128, block=16,
             seqs=32, len_lo=1, len_hi=4096, q_lo=1, q_hi=1, window=0, sinks=0, lens_seed=11),
        # long contexts, eight query heads per KV head: what a cache is cut to 4 bits for
        dict(name="int4_long_8x32k", kind="attend", q="bf16", kv="i4", heads=64, kv_heads=8, dim=128, block=16, seqs=8,
             len_lo=32768, len_hi=32768, q_lo=1, q_hi=1, window=0, sinks=0, lens_seed=32),
        # chunks of prompts over a cached context
        dict(name="int4_chunk", kind="attend", q="bf16", kv="i4", heads=32, kv_heads=8, dim=128, block=16, seqs=4,
             len_lo=4096, len_hi=8192, q_lo=1024, q_hi=2048, window=0, sinks=0, lens_seed=12),
        # --- attention with a window and first tokens that stay visible
        # one decode step at the end of long streams: of 32K cached positions 4 + 4096 are seen
        dict(name="sinks_step_8x32k", kind="attend", q="bf16", kv="bf16", heads=64, kv_heads=8, dim=128, block=16,
             seqs=8, len_lo=32768, len_hi=32768, q_lo=1, q_hi=1, window=4096, sinks=4, lens_seed=32),
        # a decode step of a large batch over a 4-bit cache: short windows, a first block's worth of sinks
        dict(name="sinks_step_64_int4", kind="attend", q="bf16", kv="i4", heads=32, kv_heads=8, dim=128, block=32,
             seqs=64, len_lo=16, len_hi=8192, q_lo=1, q_hi=1, window=1024, sinks=32, lens_seed=13),
        # chunks of prompts whose queries see the last 1024 positions and the first 4
        dict(name="sinks_chunk", kind="attend", q="bf16", kv="bf16", heads=32, kv_heads=8, dim=128, block=16, seqs=4,
             len_lo=4096, len_hi=8192, q_lo=1024, q_hi=2048, window=1024, sinks=4, lens_seed=12),
        # --- cached rows read back as values
        # a few hundred rows of a shared prefix from an FP8 cache
        dict(name="read_small_fp8", kind="read", kv="e4m3", out="bf16", kv_heads=8, dim=128, block=16, tokens=333),
        # the rows of several 4-bit sequences, to be moved to a 16-bit cache
        dict(name="read_32k_int4", kind="read", kv="i4", out="bf16", kv_heads=8, dim=128, block=16, tokens=32768),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the same ranges, no larger than the largest listed one."""
    most = [max(work(c)[k] for c in listed()) for k in ("bytes", "flops")]
    while True:
        c = _draw(rng)
        w = work(c)
        if w["bytes"] <= most[0] and w["flops"] <= most[1]:
            return c


def _draw(rng):
    kind = rng.choice(["norm", "int4", "int4", "sinks", "sinks", "read"])
    kv = "i4" if kind == "int4" else rng.choice(["bf16", "f16", "e4m3", "i8", "i4", "i4"])
    q = kv if kv in ("bf16", "f16") else rng.choice(["bf16", "f16"])
    dim = rng.choice([64, 128]) if kv in ("bf16", "f16") else 128
    kv_heads = rng.choice([1, 2, 4, 5, 8])
    c = dict(kind=kind, kv=kv, kv_heads=kv_heads, dim=dim, block=rng.choice([8, 16, 32, 64, 128, 256]))
    if kind == "read":
        c.update(out=rng.choice(["bf16", "f16", "f32"]), tokens=_log_int(rng, 1, 32768))
        return c
    c.update(q=q, heads=kv_heads * rng.choice([1, 2, 3, 4, 5, 7, 8]))
    if kind == "norm":
        c.update(tokens=_log_int(rng, 1, 8192), pos_max=_log_int(rng, 64, 1000000),
                 rotary=rng.choice([dim, dim, dim // 2, 32, 24, 10, 0]), interleaved=rng.random() < 0.5,
                 weights=rng.choice(["both", "both", "k", "none"]))
        return c
    c.update(kind="attend", lens_seed=rng.randrange(1 << 30), window=0, sinks=0)
    if rng.random() < 0.4:  # chunks of prompts
        hi = _log_int(rng, 16, 8192)
        q_hi = _log_int(rng, 2, min(2048, hi))
        c.update(seqs=_log_int(rng, 1, 4), len_lo=rng.randint(1, hi), len_hi=hi, q_lo=rng.randint(1, q_hi), q_hi=q_hi)
    else:  # decode steps, of one token or a few drafted ones
        hi = _log_int(rng, 1, 32768)
        c.update(seqs=_log_int(rng, 1, max(1, min(64, 262144 // hi))), len_lo=rng.randint(1, hi), len_hi=hi, q_lo=1,
                 q_hi=rng.choice([1, 1, 4]))
    if kind == "sinks":
        c.update(window=_log_int(rng, 1, hi), sinks=rng.choice([1, 4, 16, 33, 128, 200]))
    return c


# ------------------------------------------------------------------------------------------------ shapes of a case

def _lengths(case):
    """Sequence lengths and query counts (fixed by the case, not by the seed)."""
    r = random.Random(case["lens_seed"])
    lens = [r.randint(case["len_lo"], case["len_hi"]) for _ in range(case["seqs"])]
    lens[r.randrange(len(lens))] = case["len_hi"]
    q = [min(t, r.randint(case["q_lo"], case["q_hi"])) for t in lens]
    return lens, q


def _visible(case, lens, qlens):
    """(query, key) pairs one head attends, and the cache rows that any query of each sequence sees."""
    pairs, rows = 0, 0
    for t, n in zip(lens, qlens):
        first = t - n
        w = case["window"] or t
        for i in range(n):
            lo = max(0, first + i + 1 - w)
            pairs += first + i + 1 - lo + min(case["sinks"], lo)
        lo = max(0, first + 1 - w)
        rows += t - lo + min(case["sinks"], lo)
    return pairs, rows


def _row_bytes(case):
    """K and V of one token."""
    d = case["dim"]
    return 2 * case["kv_heads"] * (d // 2 + 4 if case["kv"] == "i4" else d * BYTES[case["kv"]])


def work(case):
    d, hk, row = case["dim"], case["kv_heads"], _row_bytes(case)
    if case["kind"] == "read":
        n = case["tokens"]
        return {"bytes": n * (row + 2 * hk * d * BYTES[case["out"]] + 8), "flops": n * 2 * hk * d * 2}
    hq = case["heads"]
    if case["kind"] == "norm":
        n = case["tokens"]
        back = row + 2 * hk * d * BYTES[case["q"]] + 8 if case["kv"] in ("i4", "i8") else 0
        return {"bytes": n * (2 * hq * d * 2 + 2 * hk * d * 2 + row + 16 + back),
                "flops": n * (hq + hk) * (3 * case["rotary"] + 4 * d)}
    lens, qlens = _lengths(case)
    pairs, rows = _visible(case, lens, qlens)
    tables = -(-rows // case["block"]) * 4
    return {"bytes": rows * row + sum(qlens) * hq * d * 4 + tables, "flops": pairs * hq * 4 * d}


# ------------------------------------------------------------------------------------------------ 4-bit rows

def _quantise4(x):
    """Rows of x [..., d] as (codes uint8 [..., d], scale float16, zero float16 [...])."""
    x = x.float().clamp(-32768.0, 32768.0)
    zero = x.amin(-1).half()
    scale = ((x.amax(-1) - zero.float()) / 15.0).clamp(min=0.0).half()
    # (a true quotient: halves are common between 16-bit values, and go to the even code)
    step = torch.where(scale > 0, scale.float(), torch.full((), math.inf, device=x.device))
    code = ((x - zero.float()[..., None]) / step[..., None]).round().clamp(0.0, 15.0).to(torch.uint8)
    return code, scale, zero


def _pack4(code, scale, zero):
    """Cache tiles [..., B * (d / 2 + 4)] of rows [..., B, d]."""
    b, d = code.shape[-2:]
    c = code.view(*code.shape[:-1], d // 8, 2, 2, 2)  # word, pair of nibbles, nibble, half of the word
    octets = (c[..., 0, :] | (c[..., 1, :] << 4)).transpose(-1, -2)
    pairs = torch.stack((scale, zero), -1).contiguous().view(torch.uint8)
    return torch.cat((octets.reshape(*code.shape[:-2], b * d // 2), pairs.reshape(*code.shape[:-2], b * 4)), -1)


def _codes(octets):
    """Codes [..., d] of rows of d / 2 bytes."""
    o = octets.view(*octets.shape[:-1], octets.shape[-1] // 4, 2, 2)  # word, half of the word, byte
    c = torch.stack((o & 15, o >> 4), -1)  # word, half, byte, nibble
    return c.permute(*range(c.dim() - 3), -2, -1, -3).reshape(*octets.shape[:-1], octets.shape[-1] * 2)


def _rows4(cache, blk, off, block, dim, real):
    """Values of rows (blk, off) of every KV head: [..., H_kv, d]."""
    tiles = block * dim // 2
    octets = cache[..., :tiles].view(cache.shape[0], cache.shape[1], block, dim // 2)[blk, :, off]
    pairs = cache[..., tiles:].reshape(cache.shape[0], cache.shape[1], block, 4)[blk, :, off].view(torch.float16)
    return _codes(octets).to(real) * pairs[..., :1].to(real) + pairs[..., 1:].to(real)


# ------------------------------------------------------------------------------------------------ inputs

def _normal(g, *shape, dtype):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)


def _pool(g, case, blocks):
    """One cache pool in its storage type, with per-head scale and zero point for 8-bit types."""
    h, b, d = case["kv_heads"], case["block"], case["dim"]
    if case["kv"] == "i4":
        out = torch.empty((blocks, h, b * (d // 2 + 4)), device=DEV, dtype=torch.uint8)
        scale = zp = None
    else:
        out = torch.empty((blocks, h, b, d), device=DEV, dtype=DTYPES[case["kv"]])
        scale = None if case["kv"] in ("bf16", "f16") else 0.02 + 0.01 * torch.rand(h, generator=g, device=DEV)
        zp = torch.randint(-20, 21, (h,), generator=g, device=DEV, dtype=torch.int32) if case["kv"] == "i8" else None
    for piece in out.split(max(1, (1 << 26) // (h * b * d))):
        x = torch.randn((piece.shape[0], h, b, d), generator=g, device=DEV)
        if case["kv"] == "i4":
            piece.copy_(_pack4(*_quantise4(x)))
            continue
        if scale is not None:
            x = x / scale.view(1, h, 1, 1)
        if zp is not None:
            x = (x.round() + zp.view(1, h, 1, 1)).clamp_(-128, 127)
        piece.copy_(x)
    return out, scale, zp


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    hk, d, b = case["kv_heads"], case["dim"], case["block"]
    st = dict(case=case)
    if own:
        import paged_kv_cache_144_gb300 as pa
        pa.load()
    if case["kind"] == "read":
        n = case["tokens"]
        blocks = -(-n // b) + 4
        for w in ("k", "v"):
            st[w + "_cache"], st[w + "_scale"], st[w + "_zp"] = _pool(g, case, blocks)
            st[w + "_out"] = torch.empty((n, hk, d), device=DEV, dtype=DTYPES[case["out"]])
        # whole blocks in any order, as a sequence's table names them
        perm = torch.randperm(blocks, generator=g, device=DEV)
        t = torch.arange(n, device=DEV)
        st["slots"] = perm[t // b] * b + t % b
        return st
    hq = case["heads"]
    qt = DTYPES[case["q"]]
    if case["kind"] == "norm":
        n = case["tokens"]
        blocks = -(-n // b) + 4
        st["q"] = _normal(g, n, hq, d, dtype=qt)
        st["k"] = _normal(g, n, hk, d, dtype=qt)
        st["v"] = _normal(g, n, hk, d, dtype=qt)
        st["q_out"] = torch.empty_like(st["q"])
        st["q_weight"] = st["k_weight"] = None
        if case["weights"] == "both":
            st["q_weight"] = (1.0 + 0.2 * torch.randn(d, generator=g, device=DEV)).to(qt)
        if case["weights"] != "none":
            st["k_weight"] = (1.0 + 0.2 * torch.randn(d, generator=g, device=DEV)).to(qt)
        st["slots"] = torch.randperm(blocks * b, generator=g, device=DEV)[:n].contiguous()
        st["positions"] = torch.randint(0, case["pos_max"], (n,), generator=g, device=DEV)
        r = case["rotary"]
        i = torch.arange(0, r, 2, dtype=torch.float64)
        st["inv_freq"] = (1.0 / (10000.0 ** (i / max(r, 1)))).float().to(DEV)
        if case["kv"] == "i4":
            st["k_cache"] = torch.zeros((blocks, hk, b * (d // 2 + 4)), device=DEV, dtype=torch.uint8)
        else:
            st["k_cache"] = torch.zeros((blocks, hk, b, d), device=DEV, dtype=DTYPES[case["kv"]])
        st["v_cache"] = torch.zeros_like(st["k_cache"])
        for w in ("k", "v"):
            eight = case["kv"] in ("e4m3", "i8")
            st[w + "_inv"] = 20.0 + 20.0 * torch.rand(hk, generator=g, device=DEV) if eight else None
            st[w + "_scale"] = 1.0 / st[w + "_inv"] if eight else None
            st[w + "_zp"] = None
            if case["kv"] == "i8":
                st[w + "_zp"] = torch.randint(-20, 21, (hk,), generator=g, device=DEV, dtype=torch.int32)
            if case["kv"] in ("i4", "i8"):
                st[w + "_out"] = torch.empty_like(st["k"])
        return st
    lens, qlens = _lengths(case)
    need = [-(-t // b) for t in lens]
    blocks = sum(need) + max(1, sum(need) // 16)
    st["scale"] = 1.0 / math.sqrt(d)
    for w in ("k", "v"):
        st[w + "_cache"], st[w + "_scale"], st[w + "_zp"] = _pool(g, case, blocks)
    perm = torch.randperm(blocks, generator=g, device=DEV).to(torch.int32)
    st["tables"] = torch.full((len(lens), max(need)), -1, dtype=torch.int32, device=DEV)
    at = 0
    for s, m in enumerate(need):
        st["tables"][s, :m] = perm[at:at + m]
        at += m
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    starts = [0]
    for x in qlens:
        starts.append(starts[-1] + x)
    st["starts"] = torch.tensor(starts, dtype=torch.int32, device=DEV)
    st["max_q"] = max(qlens)
    st["q"] = _normal(g, sum(qlens), hq, d, dtype=qt)
    st["out"] = torch.empty_like(st["q"])
    if own:
        nbytes = pa.attend_workspace_bytes(len(lens), hq, hk, d, b, max(need), st["max_q"],
                                           pa.cache_dtype_code(st["k_cache"]))
        st["workspace"] = pa.new_workspace(nbytes, DEV)
    return st


# ------------------------------------------------------------------------------------------------ one pass

def run(st):
    kind = st["case"]["kind"]
    if own:
        return _OWN[kind](st)
    return _PLAIN[kind](st)


def _own_read(st):
    import paged_kv_cache_144_gb300 as pa
    pa.read_cache(st["k_out"], st["v_out"], st["k_cache"], st["v_cache"], st["slots"], st["case"]["block"],
                  k_scale=st["k_scale"], v_scale=st["v_scale"], k_zero_point=st["k_zp"], v_zero_point=st["v_zp"])
    return {"k": st["k_out"], "v": st["v_out"]}


def _own_norm(st):
    import paged_kv_cache_144_gb300 as pa
    c = st["case"]
    pa.norm_rope_and_cache(st["q"], st["k"], st["v"], st["k_cache"], st["v_cache"], st["positions"], st["slots"],
                           st["inv_freq"], c["block"], q_weight=st["q_weight"], k_weight=st["k_weight"], eps=1e-6,
                           q_out=st["q_out"], interleaved=c["interleaved"], k_inv_scale=st["k_inv"],
                           v_inv_scale=st["v_inv"], k_zero_point=st["k_zp"], v_zero_point=st["v_zp"])
    if c["kv"] in ("i4", "i8"):
        return dict(_own_read(st), q=st["q_out"])
    return {"q": st["q_out"], "k": st["k_cache"], "v": st["v_cache"]}


def _own_attend(st):
    import paged_kv_cache_144_gb300 as pa
    c = st["case"]
    return pa.attend(st["out"], st["q"], st["k_cache"], st["v_cache"], st["tables"], st["lens"], st["starts"],
                     st["max_q"], c["kv_heads"], st["scale"], c["block"], workspace=st["workspace"],
                     k_scale=st["k_scale"], v_scale=st["v_scale"], k_zero_point=st["k_zp"], v_zero_point=st["v_zp"],
                     window=c["window"], sinks=c["sinks"])


_OWN = {"norm": _own_norm, "attend": _own_attend, "read": _own_read}


# ---- plain forms

def _at(st, which, blk, off, real):
    """Values of cache rows (blk, off), any shape: [..., H_kv, d]."""
    c = st["case"]
    cache = st[which + "_cache"]
    if c["kv"] == "i4":
        return _rows4(cache, blk, off, c["block"], c["dim"], real)
    raw = cache.view(torch.uint8) if c["kv"] == "e4m3" else cache
    x = raw[blk, :, off].view(DTYPES[c["kv"]]).to(real)
    if st[which + "_zp"] is not None:
        x = x - st[which + "_zp"].view(-1, 1)
    if st[which + "_scale"] is not None:
        x = x * st[which + "_scale"].view(-1, 1).to(real)
    return x


def _plain_read(st):
    b = st["case"]["block"]
    st["k_out"].copy_(_at(st, "k", st["slots"] // b, st["slots"] % b, torch.float32))
    st["v_out"].copy_(_at(st, "v", st["slots"] // b, st["slots"] % b, torch.float32))
    return {"k": st["k_out"], "v": st["v_out"]}


def _plain_norm(st):
    c = st["case"]
    r = c["rotary"]
    angle = st["positions"].double()[:, None] * st["inv_freq"].double()[None, :]
    cos, sin = torch.cos(angle).float()[:, None, :], torch.sin(angle).float()[:, None, :]

    def rotate(x, weight):
        x = x.float()
        if weight is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * weight.float()
        y = x.clone()
        if c["interleaved"]:
            a, b = x[..., 0:r:2], x[..., 1:r:2]
            y[..., 0:r:2] = a * cos - b * sin
            y[..., 1:r:2] = b * cos + a * sin
        else:
            a, b = x[..., :r // 2], x[..., r // 2:r]
            y[..., :r // 2] = a * cos - b * sin
            y[..., r // 2:r] = b * cos + a * sin
        return y

    st["q_out"].copy_(rotate(st["q"], st["q_weight"]))
    k, v = rotate(st["k"], st["k_weight"]), st["v"].float()
    at = (st["slots"] // c["block"])[:, None], torch.arange(c["kv_heads"], device=DEV)[None], (st["slots"] % c["block"])[:, None]
    if c["kv"] == "i4":
        _store4(st["k_cache"], at, *_quantise4(k))
        _store4(st["v_cache"], at, *_quantise4(v))
    elif c["kv"] == "e4m3":
        kt = DTYPES["e4m3"]
        st["k_cache"].view(torch.uint8)[at] = (k * st["k_inv"][:, None]).clamp(-448.0, 448.0).to(kt).view(torch.uint8)
        st["v_cache"].view(torch.uint8)[at] = (v * st["v_inv"][:, None]).clamp(-448.0, 448.0).to(kt).view(torch.uint8)
    elif c["kv"] == "i8":
        st["k_cache"][at] = ((k * st["k_inv"][:, None]).round() + st["k_zp"][:, None]).clamp(-128, 127).to(torch.int8)
        st["v_cache"][at] = ((v * st["v_inv"][:, None]).round() + st["v_zp"][:, None]).clamp(-128, 127).to(torch.int8)
    else:
        st["k_cache"][at] = k.to(DTYPES[c["kv"]])
        st["v_cache"][at] = v.to(DTYPES[c["kv"]])
    if c["kv"] in ("i4", "i8"):
        return dict(_plain_read(st), q=st["q_out"])
    return {"q": st["q_out"], "k": st["k_cache"], "v": st["v_cache"]}


def _store4(cache, at, code, scale, zero):
    """Rows [N, H_kv, d] to (block, head, row) of a 4-bit cache."""
    d, b = code.shape[-1], cache.shape[-1] // (code.shape[-1] // 2 + 4)
    row = _pack4(code[..., None, :], scale[..., None], zero[..., None])
    lead = cache.shape[:-1]
    cache[..., :b * d // 2].view(*lead, b, d // 2)[at] = row[..., :d // 2]
    cache[..., b * d // 2:].view(*lead, b, 4)[at] = row[..., d // 2:]


def _plain_attend(st):
    c = st["case"]
    hq, hk, d, S = c["heads"], c["kv_heads"], c["dim"], c["seqs"]
    # ragged rows as [S, L], with each row's index into q and whether it exists
    i = torch.arange(st["max_q"], device=DEV)
    starts = st["starts"].long()
    count = starts[1:] - starts[:-1]
    there = i[None, :] < count[:, None]
    index = torch.where(there, starts[:-1, None] + i[None, :], torch.zeros_like(starts[:-1, None]))
    q = st["q"][index].float().view(S, -1, hk, hq // hk, d).permute(0, 2, 3, 1, 4).reshape(S, hk, -1, d)
    # the sequences' rows through the block table
    t = torch.arange(st["tables"].shape[1] * c["block"], device=DEV)
    blk, off = st["tables"].clamp(min=0).long()[:, t // c["block"]], (t % c["block"])[None, :].expand(S, -1)
    s = torch.matmul(q, _at(st, "k", blk, off, torch.float32).permute(0, 2, 3, 1)) * st["scale"]
    lens = st["lens"].long()[:, None, None]
    pos = lens - count[:, None, None] + i[None, :, None]
    seen = (t <= pos) & (t < lens)
    if c["window"]:
        seen = seen & ((t > pos - c["window"]) | (t < c["sinks"]))
    seen = seen & there[:, :, None]
    s = s.view(S, hk, hq // hk, st["max_q"], -1).masked_fill(~seen[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total == 0, torch.ones_like(total), total)
    o = torch.matmul(p.view(S, hk, -1, p.shape[-1]), _at(st, "v", blk, off, torch.float32).transpose(1, 2))
    o = o.view(S, hk, hq // hk, -1, d).permute(0, 3, 1, 2, 4).reshape(S, -1, hq, d)
    st["out"][index[there]] = o[there].to(st["out"].dtype)
    return st["out"]


_PLAIN = {"norm": _plain_norm, "attend": _plain_attend, "read": _plain_read}


# ------------------------------------------------------------------------------------------------ from the definition

def exact(case, seed):
    st = prepare(case, seed)
    if case["kind"] == "read":
        return {w: _exact_rows(st, w, st["slots"]) for w in ("k", "v")}
    if case["kind"] == "norm":
        return _exact_norm(st)
    out = torch.zeros(st["q"].shape, device=DEV, dtype=torch.float64)
    starts = st["starts"].tolist()
    hk, g, b = case["kv_heads"], case["heads"] // case["kv_heads"], case["block"]
    for s, t in enumerate(st["lens"].tolist()):
        n = starts[s + 1] - starts[s]
        # only the rows that some query of the sequence sees
        lo = max(0, t - n + 1 - (case["window"] or t))
        p = torch.cat((torch.arange(min(case["sinks"], lo)), torch.arange(lo, t))).to(DEV)
        slots = st["tables"][s].long()[p // b] * b + p % b
        at = torch.arange(t - n, t, device=DEV)[:, None]
        hidden = p > at
        if case["window"]:
            hidden = hidden | ((at - p >= case["window"]) & (p >= case["sinks"]))
        for h in range(hk):
            kk, vv = (_exact_rows(st, w, slots, h) for w in ("k", "v"))
            for j in range(h * g, (h + 1) * g):
                x = st["q"][starts[s]:starts[s + 1], j].double() @ kk.T / math.sqrt(case["dim"])
                w = torch.softmax(x.masked_fill(hidden, -math.inf), -1)
                out[starts[s]:starts[s + 1], j] = w @ vv
    return out


def _exact_rows(st, which, slots, head=None):
    """Values in 64 bits of cache rows by slot: [N, H_kv, d], or [N, d] of one head."""
    c = st["case"]
    b, d = c["block"], c["dim"]
    cache = st[which + "_cache"]
    heads = range(c["kv_heads"]) if head is None else [head]
    got = []
    for h in heads:
        if c["kv"] == "i4":
            tile = cache[:, h]
            words = tile[:, :b * d // 2].contiguous().view(torch.int32).view(-1, d // 8)[slots].long()
            sz = tile[:, b * d // 2:].contiguous().view(torch.float16).view(-1, 2)[slots].double()
            i = torch.arange(d, device=DEV)
            code = (words[:, i // 8] >> (16 * (i % 2) + 4 * (i % 8 // 2))) & 15
            got.append(code.double() * sz[:, :1] + sz[:, 1:])
            continue
        x = cache[:, h].contiguous().view(torch.uint8).view(-1, d * cache.element_size())[slots].view(cache.dtype).double()
        if st[which + "_zp"] is not None:
            x = x - float(st[which + "_zp"][h])
        if st[which + "_scale"] is not None:
            x = x * float(st[which + "_scale"][h])
        got.append(x)
    return torch.stack(got, 1) if head is None else got[0]


def _exact_norm(st):
    c = st["case"]
    half = c["rotary"] // 2
    theta = torch.outer(st["positions"].double(), st["inv_freq"].double())
    turn = torch.polar(torch.ones_like(theta), theta)[:, None, :]

    def placed(x, weight):
        x = x.double()
        if weight is not None:
            x = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / c["dim"] + 1e-6) * weight.double()
        pairs = x[..., :c["rotary"]]
        if c["interleaved"]:
            z = torch.complex(pairs[..., 0::2].contiguous(), pairs[..., 1::2].contiguous()) * turn
            y = torch.stack((z.real, z.imag), -1).flatten(-2)
        else:
            z = torch.complex(pairs[..., :half].contiguous(), pairs[..., half:].contiguous()) * turn
            y = torch.cat((z.real, z.imag), -1)
        return torch.cat((y, x[..., c["rotary"]:]), -1)

    out = {"q": placed(st["q"], st["q_weight"])}
    for w, x in (("k", placed(st["k"], st["k_weight"])), ("v", st["v"].double())):
        if c["kv"] == "i4":
            low = x.amin(-1, keepdim=True).half().double()
            step = ((x.amax(-1, keepdim=True) - low) / 15).half().double()
            x = torch.round((x - low) / step).clamp(0, 15) * step + low
        elif c["kv"] == "i8":
            x = x * st[w + "_inv"].double()[:, None]
            x = (torch.round(x) + st[w + "_zp"].double()[:, None]).clamp(-128, 127)
            x = (x - st[w + "_zp"].double()[:, None]) * st[w + "_scale"].double()[:, None]
        else:
            if c["kv"] == "e4m3":
                x = (x * st[w + "_inv"].double()[:, None]).clamp(-448, 448)
            pool = torch.zeros(st["k_cache"].shape, device=DEV, dtype=torch.float64).transpose(1, 2).contiguous()
            pool.view(-1, c["kv_heads"], c["dim"])[st["slots"]] = x
            x = pool.transpose(1, 2).contiguous()
        out[w] = x
    return out
