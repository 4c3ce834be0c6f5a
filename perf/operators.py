"""Timing cases of the operators around the paged cache: rotary positions written with the cache rows, attention
with score modifiers, attention for a tree of drafted tokens with the commit of the accepted path, attention that
accumulates each cached token's weight, and the eviction that reads those weights.

`run(state)` is one pass through an operator.  With `own` false it is the operator's plain form: elementary torch
operations in 32 bits, rounded once at the end.  With `own` true it is the calls a user makes of the library.
`exact(case, seed)` is the same answer from the definition in 64 bits.
"""

import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn, "i8": torch.int8}
KV_BYTES = {"bf16": 2, "f16": 2, "e4m3": 1, "i8": 1}
Q_BYTES = 2


# ------------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # --- rotary positions with the cache write
        # one decode step of a 32-sequence batch (the latency that every layer of every step pays)
        dict(name="rope_step_32", kind="rope", q="bf16", kv="bf16", heads=32, kv_heads=8, dim=128, block=16, tokens=32,
             pos_max=4096, rotary=128, interleaved=False, base=10000.0, rope_scale=1.0, stretch=1.0),
        # prompts of several sequences written at once, far positions with a stretched frequency table
        dict(name="rope_prompt_8k", kind="rope", q="bf16", kv="bf16", heads=32, kv_heads=8, dim=128, block=16,
             tokens=8192, pos_max=131072, rotary=128, interleaved=False, base=500000.0, rope_scale=1.0, stretch=8.0),
        # an odd number of prompt tokens into an FP8 cache, half of each head rotated, adjacent pairs
        dict(name="rope_partial_fp8", kind="rope", q="bf16", kv="e4m3", heads=32, kv_heads=8, dim=128, block=32,
             tokens=2049, pos_max=32768, rotary=64, interleaved=True, base=10000.0, rope_scale=1.1, stretch=1.0),
        # --- attention with capped scores, a distance bias, a window, a prefix mask
        # one decode step of a 32-sequence batch with capped scores
        dict(name="attend_step_capped", kind="attend", q="bf16", kv="bf16", heads=32, kv_heads=8, dim=128, block=16,
             seqs=32, len_lo=1, len_hi=4096, q_lo=1, q_hi=1, cap=30.0, bias=False, window=0, prefix=0, lens_seed=11),
        # chunks of prompts over a cached context, the first part of each sequence seen by every query
        dict(name="attend_chunk_prefix", kind="attend", q="bf16", kv="bf16", heads=32, kv_heads=8, dim=128, block=16,
             seqs=4, len_lo=4096, len_hi=8192, q_lo=1024, q_hi=2048, cap=0.0, bias=False, window=0, prefix=512,
             lens_seed=12),
        # a decode step over an FP8 cache with a bias by distance
        dict(name="attend_step_bias_fp8", kind="attend", q="bf16", kv="e4m3", heads=32, kv_heads=8, dim=128, block=16,
             seqs=64, len_lo=16, len_hi=8192, q_lo=1, q_hi=1, cap=0.0, bias=True, window=0, prefix=0, lens_seed=13),
        # --- verification of drafted trees: attention of the nodes, then the accepted path moves to the front
        # a few small trees over short contexts (the latency of a small serving batch)
        dict(name="verify_small", kind="verify", q="f16", kv="f16", heads=4, kv_heads=4, dim=64, block=16, seqs=4,
             len_lo=20, len_hi=300, q_lo=5, q_hi=16, cap=0.0, lens_seed=21),
        # 64-node trees over 32K tokens of context, eight query heads per KV head
        dict(name="verify_long_64", kind="verify", q="bf16", kv="bf16", heads=64, kv_heads=8, dim=128, block=16, seqs=8,
             len_lo=32768, len_hi=32768, q_lo=64, q_hi=64, cap=0.0, lens_seed=22),
        # --- a decode step that adds each cached token's attention weight to its running total
        dict(name="accumulate_step", kind="accumulate", q="bf16", kv="bf16", heads=32, kv_heads=8, dim=128, block=16,
             seqs=32, len_lo=1, len_hi=4096, cap=0.0, lens_seed=31),
        dict(name="accumulate_long", kind="accumulate", q="bf16", kv="bf16", heads=64, kv_heads=8, dim=128, block=16,
             seqs=8, len_lo=32768, len_hi=32768, cap=0.0, lens_seed=32),
        # --- eviction by those totals: the kept rows of each KV head move to the sequence's new blocks
        # a small batch that has just passed its budget
        dict(name="evict_small", kind="evict", q="bf16", kv="bf16", heads=32, kv_heads=8, dim=128, block=16, seqs=4,
             len_lo=300, len_hi=1100, budget=256, recent=32, sinks=4, lens_seed=41),
        # long sequences cut back to an eighth
        dict(name="evict_long", kind="evict", q="bf16", kv="bf16", heads=64, kv_heads=8, dim=128, block=16, seqs=8,
             len_lo=16384, len_hi=32768, budget=4096, recent=256, sinks=4, lens_seed=42),
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
    kind = rng.choice(["rope", "attend", "verify", "accumulate", "evict"])
    kv = rng.choice(["bf16", "f16", "e4m3"] if kind == "rope" else ["bf16", "f16", "e4m3", "i8"])
    q = kv if kv in ("bf16", "f16") else rng.choice(["bf16", "f16"])
    dim = rng.choice([64, 128]) if kv in ("bf16", "f16") else 128
    kv_heads = rng.choice([1, 2, 4, 5, 8])
    group = rng.choice([1, 2, 3, 4, 5, 7, 8])
    c = dict(kind=kind, q=q, kv=kv, heads=kv_heads * group, kv_heads=kv_heads, dim=dim,
             block=rng.choice([8, 16, 32, 64, 128, 256]))
    if kind == "rope":
        c.update(tokens=_log_int(rng, 1, 8192), pos_max=_log_int(rng, 64, 1000000),
                 rotary=rng.choice([dim, dim, dim // 2, 32, 24, 10]), interleaved=rng.random() < 0.5,
                 base=rng.choice([10000.0, 500000.0]), rope_scale=rng.choice([1.0, 1.0, 1.2]),
                 stretch=rng.choice([1.0, 4.0]))
        return c
    c["lens_seed"] = rng.randrange(1 << 30)
    if kind == "evict":
        hi = _log_int(rng, 64, 32768)
        budget = _log_int(rng, 16, max(17, hi // 2))
        c.update(seqs=_log_int(rng, 1, 8), len_lo=rng.randint(1, hi), len_hi=hi, budget=budget,
                 recent=rng.randint(0, budget // 2), sinks=rng.choice([0, 1, 4]))
        return c
    if kind == "attend" and rng.random() < 0.5:  # chunks of prompts
        hi = _log_int(rng, 16, 8192)
        q_hi = _log_int(rng, 2, min(2048, hi))
        c.update(seqs=_log_int(rng, 1, 4), len_lo=rng.randint(1, hi), len_hi=hi, q_lo=rng.randint(1, q_hi), q_hi=q_hi)
    else:
        hi = _log_int(rng, 1, 32768)
        seqs = _log_int(rng, 1, max(1, min(64, 262144 // hi)))
        c.update(seqs=seqs, len_lo=rng.randint(1, hi), len_hi=hi)
        if kind == "attend":
            c.update(q_lo=1, q_hi=rng.choice([1, 1, 4]))
        if kind == "verify":
            q_hi = _log_int(rng, 1, min(64, hi))
            c.update(q_lo=rng.randint(1, q_hi), q_hi=q_hi, seqs=min(seqs, 8))
    c["cap"] = rng.choice([0.0, 0.0, 20.0, 50.0])
    if kind == "attend":
        form = rng.choice(["plain", "bias", "window", "prefix"])
        c.update(bias=form == "bias", window=_log_int(rng, 1, hi) if form == "window" else 0,
                 prefix=rng.randint(1, hi) if form == "prefix" else 0)
    return c


# ------------------------------------------------------------------------------------------------ shapes of a case

def _lengths(case):
    """Sequence lengths and query counts (fixed by the case, not by the seed)."""
    r = random.Random(case["lens_seed"])
    lens = [r.randint(case["len_lo"], case["len_hi"]) for _ in range(case["seqs"])]
    lens[r.randrange(len(lens))] = case["len_hi"]
    q = [min(t, r.randint(case.get("q_lo", 1), case.get("q_hi", 1))) for t in lens]
    return lens, q


def _visible_pairs(case, lens, qlens):
    """(query, key) pairs one head attends, and the cache rows that any query of each sequence sees."""
    pairs, rows = 0, 0
    w, pre = case.get("window", 0), case.get("prefix", 0)
    for t, n in zip(lens, qlens):
        first = t - n
        if case["kind"] == "verify":
            pairs += n * first + sum(len(p) for p in _tree(case, n))
            rows += t
        elif w:
            pairs += sum(min(w, first + i + 1) for i in range(n))
            rows += t - max(0, first + 1 - w)
        elif pre:
            pairs += sum(max(min(pre, t), first + i + 1) for i in range(n))
            rows += t
        else:
            pairs += sum(first + i + 1 for i in range(n))
            rows += t
    return pairs, rows


def _tree(case, n):
    """Ancestor lists (self included) of an n-node tree whose nodes come in topological order."""
    r = random.Random(case["lens_seed"] * 1000003 + n)
    anc = []
    for i in range(n):
        parent = -1 if i == 0 else r.randint(max(-1, i - 8), i - 1)
        anc.append(([] if parent < 0 else anc[parent]) + [i])
    return anc


def work(case):
    d, hq, hk = case["dim"], case["heads"], case["kv_heads"]
    row = hk * d * KV_BYTES[case["kv"]] * 2  # K and V of one token
    if case["kind"] == "rope":
        n = case["tokens"]
        return {"bytes": n * (2 * hq * d * Q_BYTES + 2 * hk * d * Q_BYTES + row + 16),
                "flops": n * (hq + hk) * case["rotary"] * 3}
    lens, qlens = _lengths(case)
    tables = sum(-(-t // case["block"]) for t in lens) * 4
    if case["kind"] == "evict":
        kept = sum(min(t, case["budget"]) for t in lens)
        return {"bytes": sum(lens) * hk * 4 + kept * (2 * row + hk * 8) + 2 * tables, "flops": sum(lens) * hk}
    pairs, rows = _visible_pairs(case, lens, qlens)
    nbytes = rows * row + sum(qlens) * hq * d * Q_BYTES * 2 + tables
    if case["kind"] == "accumulate":
        nbytes += rows * hk * 8
    if case["kind"] == "verify":
        nbytes += sum(len(_path(case, n)) for n in qlens) * row * 2 + sum(n * -(-n // 64) * 8 for n in qlens)
    return {"bytes": nbytes, "flops": pairs * hq * 4 * d}


def _path(case, n):
    """The accepted path: the nodes from a root to one of the deepest leaves."""
    return max(_tree(case, n), key=len)


# ------------------------------------------------------------------------------------------------ inputs

def _normal(g, *shape, dtype):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)


def _pool(g, case, blocks):
    """One cache pool [blocks, H_kv, B, d] in its storage type, with per-head scale and zero point for 8-bit types."""
    shape = (blocks, case["kv_heads"], case["block"], case["dim"])
    h = case["kv_heads"]
    if case["kv"] in ("bf16", "f16"):
        out = torch.empty(shape, device=DEV, dtype=DTYPES[case["kv"]])
        for piece in out.split(max(1, (1 << 26) // max(1, out[0].numel()))):
            piece.normal_(generator=g)
        return out, None, None
    scale = 0.02 + 0.01 * torch.rand(h, generator=g, device=DEV)
    zp = None
    out = torch.empty(shape, device=DEV, dtype=DTYPES[case["kv"]])
    if case["kv"] == "i8":
        zp = torch.randint(-20, 21, (h,), generator=g, device=DEV, dtype=torch.int32)
    for piece in out.split(max(1, (1 << 26) // max(1, out[0].numel()))):
        x = torch.randn(piece.shape, generator=g, device=DEV) / scale.view(1, h, 1, 1)
        if zp is not None:
            x = (x.round() + zp.view(1, h, 1, 1)).clamp_(-128, 127)
        piece.copy_(x)
    return out, scale, zp


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    hq, hk, d, b = case["heads"], case["kv_heads"], case["dim"], case["block"]
    qt = DTYPES[case["q"]]
    st = dict(case=case, scale=1.0 / math.sqrt(d))
    if case["kind"] == "rope":
        n = case["tokens"]
        blocks = -(-n // b) + 4
        st["q"] = _normal(g, n, hq, d, dtype=qt)
        st["k"] = _normal(g, n, hk, d, dtype=qt)
        st["v"] = _normal(g, n, hk, d, dtype=qt)
        st["q_out"] = torch.empty_like(st["q"])
        st["k_cache"] = torch.zeros((blocks, hk, b, d), device=DEV, dtype=DTYPES[case["kv"]])
        st["v_cache"] = torch.zeros_like(st["k_cache"])
        st["slots"] = torch.randperm(blocks * b, generator=g, device=DEV)[:n].contiguous()
        st["positions"] = torch.randint(0, case["pos_max"], (n,), generator=g, device=DEV)
        r = case["rotary"]
        i = torch.arange(0, r, 2, dtype=torch.float64)
        st["inv_freq"] = (1.0 / (case["base"] ** (i / r) * case["stretch"])).float().to(DEV)
        st["k_inv"] = st["v_inv"] = None
        if case["kv"] == "e4m3":
            st["k_inv"] = 20.0 + 20.0 * torch.rand(hk, generator=g, device=DEV)
            st["v_inv"] = 20.0 + 20.0 * torch.rand(hk, generator=g, device=DEV)
        return st
    lens, qlens = _lengths(case)
    need = [-(-t // b) for t in lens]
    extra = -(-min(case["budget"], max(lens)) // b) * len(lens) if case["kind"] == "evict" else 0
    blocks = sum(need) + extra + max(1, sum(need) // 16)
    st["k_cache"], st["k_scale"], st["k_zp"] = _pool(g, case, blocks)
    st["v_cache"], st["v_scale"], st["v_zp"] = _pool(g, case, blocks)
    perm = torch.randperm(blocks, generator=g, device=DEV).to(torch.int32)
    width = max(need)

    def tables_of(counts, at):
        t = torch.full((len(lens), max(counts)), -1, dtype=torch.int32, device=DEV)
        for s, m in enumerate(counts):
            t[s, :m] = perm[at:at + m]
            at += m
        return t, at

    st["tables"], at = tables_of(need, 0)
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    if case["kind"] in ("accumulate", "evict"):
        # running totals as decode steps leave them: a few heavy tokens, many light ones
        m = torch.rand((len(lens), hk, width * b), generator=g, device=DEV)
        st["mass"] = m.pow_(8).mul_(50.0)
    if case["kind"] == "evict":
        st["dst_tables"], _ = tables_of([-(-min(t, case["budget"]) // b) for t in lens], at)
        st["mass_out"] = torch.zeros((len(lens), hk, case["budget"]), device=DEV)
        st["kept"] = torch.full((len(lens), hk, case["budget"]), -1, dtype=torch.int32, device=DEV)
        st["new_lens"] = torch.zeros(len(lens), dtype=torch.int32, device=DEV)
        if own:
            import paged_kv_cache_144_gb300 as pa
            pa.load()
        return st
    n = sum(qlens)
    st["q"] = _normal(g, n, hq, d, dtype=qt)
    st["out"] = torch.empty_like(st["q"])
    starts = [0]
    for x in qlens:
        starts.append(starts[-1] + x)
    st["starts"] = torch.tensor(starts, dtype=torch.int32, device=DEV)
    st["max_q"] = max(qlens)
    st["slopes"] = st["prefix"] = None
    if case.get("bias"):
        st["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / hq) for h in range(hq)], device=DEV)
    if case.get("prefix"):
        st["prefix"] = torch.tensor([min(case["prefix"], t) for t in lens], dtype=torch.int32, device=DEV)
    if case["kind"] == "verify":
        words = -(-st["max_q"] // 64)
        bits = [[0] * words for _ in range(n)]
        paths, k = [], 0
        for x in qlens:
            for a in _tree(case, x):
                for j in a:
                    bits[k][j // 64] |= 1 << (j % 64)
                k += 1
            paths.append(_path(case, x))
        signed = [[w - (1 << 64) if w >= 1 << 63 else w for w in ws] for ws in bits]
        st["tree"] = torch.tensor(signed, dtype=torch.int64, device=DEV)
        deep = max(len(p) for p in paths)
        st["path"] = torch.tensor([p + [0] * (deep - len(p)) for p in paths], dtype=torch.int32, device=DEV)
        st["path_lens"] = torch.tensor([len(p) for p in paths], dtype=torch.int32, device=DEV)
        st["new_lens"] = torch.zeros(len(lens), dtype=torch.int32, device=DEV)
    if own:
        import paged_kv_cache_144_gb300 as pa
        nbytes = pa.attend_workspace_bytes(len(lens), hq, hk, d, b, width, st["max_q"], pa.dtype_code(st["k_cache"]),
                                           accumulate=case["kind"] == "accumulate")
        st["workspace"] = pa.new_workspace(nbytes, DEV)
    return st


# ------------------------------------------------------------------------------------------------ one pass

def run(st):
    kind = st["case"]["kind"]
    if own:
        return _OWN[kind](st)
    return _PLAIN[kind](st)


def _own_rope(st):
    import paged_kv_cache_144_gb300 as pa
    c = st["case"]
    pa.rope_and_cache(st["q"], st["k"], st["v"], st["k_cache"], st["v_cache"], st["positions"], st["slots"],
                      st["inv_freq"], c["block"], q_out=st["q_out"], interleaved=c["interleaved"],
                      rope_scale=c["rope_scale"], k_inv_scale=st["k_inv"], v_inv_scale=st["v_inv"])
    return {"q": st["q_out"], "k_cache": st["k_cache"], "v_cache": st["v_cache"]}


def _own_attend(st):
    import paged_kv_cache_144_gb300 as pa
    c = st["case"]
    return pa.attend(st["out"], st["q"], st["k_cache"], st["v_cache"], st["tables"], st["lens"], st["starts"],
                     st["max_q"], c["kv_heads"], st["scale"], c["block"], workspace=st["workspace"],
                     k_scale=st["k_scale"], v_scale=st["v_scale"], k_zero_point=st["k_zp"], v_zero_point=st["v_zp"],
                     softcap=c["cap"], slopes=st["slopes"], window=c["window"], prefix_lens=st["prefix"])


def _own_verify(st):
    import paged_kv_cache_144_gb300 as pa
    c = st["case"]
    pa.attend_tree(st["out"], st["q"], st["k_cache"], st["v_cache"], st["tables"], st["lens"], st["starts"],
                   st["max_q"], st["tree"], c["kv_heads"], st["scale"], c["block"], workspace=st["workspace"],
                   k_scale=st["k_scale"], v_scale=st["v_scale"], k_zero_point=st["k_zp"], v_zero_point=st["v_zp"],
                   softcap=c["cap"])
    pa.commit_tree(st["k_cache"], st["v_cache"], st["tables"], st["lens"], st["starts"], st["path"], st["path_lens"],
                   st["new_lens"], c["block"])
    return {"out": st["out"], "new_lens": st["new_lens"], "k_cache": _values(st["k_cache"]),
            "v_cache": _values(st["v_cache"])}


def _own_accumulate(st):
    import paged_kv_cache_144_gb300 as pa
    c = st["case"]
    pa.attend_accumulate(st["out"], st["q"], st["k_cache"], st["v_cache"], st["tables"], st["lens"], st["mass"],
                         c["kv_heads"], st["scale"], c["block"], workspace=st["workspace"], k_scale=st["k_scale"],
                         v_scale=st["v_scale"], k_zero_point=st["k_zp"], v_zero_point=st["v_zp"], softcap=c["cap"])
    return {"out": st["out"], "mass": st["mass"]}


def _own_evict(st):
    import paged_kv_cache_144_gb300 as pa
    c = st["case"]
    pa.evict(st["k_cache"], st["v_cache"], st["mass"], st["tables"], st["lens"], st["dst_tables"], st["kept"],
             st["mass_out"], st["new_lens"], c["block"], budget=c["budget"], recent=c["recent"], sinks=c["sinks"])
    return {"kept": st["kept"], "mass": st["mass_out"], "new_lens": st["new_lens"], "k_cache": _values(st["k_cache"]),
            "v_cache": _values(st["v_cache"])}


_OWN = {"rope": _own_rope, "attend": _own_attend, "verify": _own_verify, "accumulate": _own_accumulate,
        "evict": _own_evict}


def _values(cache):
    """A pool whose rows are only moved: its bytes tell the rows apart whatever they stand for."""
    return cache.view(torch.uint8) if cache.dtype == torch.float8_e4m3fn else cache


# ---- plain forms

def _plain_rope(st):
    c = st["case"]
    r, d = c["rotary"], c["dim"]
    angle = st["positions"].double()[:, None] * st["inv_freq"].double()[None, :]
    cos = (torch.cos(angle) * c["rope_scale"]).float()[:, None, :]
    sin = (torch.sin(angle) * c["rope_scale"]).float()[:, None, :]

    def rotate(x):
        x = x.float()
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

    st["q_out"].copy_(rotate(st["q"]))
    k, v = rotate(st["k"]), st["v"].float()
    if c["kv"] == "e4m3":
        k = (k * st["k_inv"][None, :, None]).clamp(-448.0, 448.0)
        v = (v * st["v_inv"][None, :, None]).clamp(-448.0, 448.0)
    blk, off = st["slots"] // c["block"], st["slots"] % c["block"]
    heads = torch.arange(c["kv_heads"], device=DEV)
    at = (blk[:, None], heads[None, :], off[:, None])
    kt = DTYPES[c["kv"]]
    if c["kv"] == "e4m3":
        st["k_cache"].view(torch.uint8)[at] = k.to(kt).view(torch.uint8)
        st["v_cache"].view(torch.uint8)[at] = v.to(kt).view(torch.uint8)
    else:
        st["k_cache"][at] = k.to(kt)
        st["v_cache"][at] = v.to(kt)
    return {"q": st["q_out"], "k_cache": st["k_cache"], "v_cache": st["v_cache"]}


def _rows(st, which, real=torch.float32):
    """K or V of every sequence through the block table: [S, H_kv, T_max, d], rows past the end zero."""
    c = st["case"]
    cache, scale, zp = st[which + "_cache"], st[which + "_scale"], st[which + "_zp"]
    t = torch.arange(st["tables"].shape[1] * c["block"], device=DEV)
    blk = st["tables"].clamp(min=0).long()[:, t // c["block"]]
    raw = cache.view(torch.uint8) if c["kv"] == "e4m3" else cache
    x = raw[blk, :, (t % c["block"])[None, :]]  # [S, T, H_kv, d]
    x = x.view(DTYPES[c["kv"]]).to(real)
    if zp is not None:
        x = x - zp.view(1, 1, -1, 1)
    if scale is not None:
        x = x * scale.view(1, 1, -1, 1)
    x = torch.where((t[None, :] < st["lens"][:, None])[:, :, None, None], x, torch.zeros((), device=DEV, dtype=real))
    return x.transpose(1, 2)


def _queries(st):
    """Ragged rows as [S, L_max], with each row's index into q and whether it exists."""
    i = torch.arange(st["max_q"], device=DEV)
    starts = st["starts"].long()
    count = starts[1:] - starts[:-1]
    there = i[None, :] < count[:, None]
    index = torch.where(there, starts[:-1, None] + i[None, :], torch.zeros_like(starts[:-1, None]))
    return index, there, count


def _mask(st, index, there, count):
    """visible [S, L, T]: which cached positions each query attends."""
    c = st["case"]
    width = st["tables"].shape[1] * c["block"]
    t = torch.arange(width, device=DEV)[None, None, :]
    lens = st["lens"].long()[:, None, None]
    i = torch.arange(st["max_q"], device=DEV)[None, :, None]
    first = lens - count[:, None, None]
    pos = first + i
    if c["kind"] == "verify":
        node = (t - first).clamp(0, 64 * st["tree"].shape[1] - 1)
        words = torch.gather(st["tree"][index], 2, (node // 64).expand(-1, st["max_q"], -1))
        seen = (t < first) | ((t >= first) & (t < lens) & (((words >> (node % 64)) & 1) != 0))
    else:
        seen = t <= pos
        if c.get("window"):
            seen = seen & (t > pos - c["window"])
        if c.get("prefix"):
            seen = seen | (t < st["prefix"].long()[:, None, None])
        seen = seen & (t < lens)
    return seen & there[:, :, None], pos


def _weights(st):
    """Softmax weights [S, H_kv, G, L, T] of the padded batch, with the index of its query rows."""
    c = st["case"]
    hq, hk = c["heads"], c["kv_heads"]
    index, there, count = _queries(st)
    q = st["q"][index].float()  # [S, L, Hq, d]
    S, L = index.shape
    q = q.view(S, L, hk, hq // hk, c["dim"]).permute(0, 2, 3, 1, 4).reshape(S, hk, hq // hk * L, c["dim"])
    s = torch.matmul(q, _rows(st, "k").transpose(2, 3)).view(S, hk, hq // hk, L, -1) * st["scale"]
    if c["cap"]:
        s = c["cap"] * torch.tanh(s / c["cap"])
    seen, pos = _mask(st, index, there, count)
    if c.get("bias"):
        t = torch.arange(s.shape[-1], device=DEV)[None, None, :]
        s = s - st["slopes"].view(1, hk, hq // hk, 1, 1) * (pos - t).abs()[:, None, None].float()
    s = s.masked_fill(~seen[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    return p / torch.where(total == 0, torch.ones_like(total), total), index, there


def _plain_attend(st):
    c = st["case"]
    p, index, there = _weights(st)
    S, hk, G, L, T = p.shape
    o = torch.matmul(p.view(S, hk, G * L, T), _rows(st, "v")).view(S, hk, G, L, c["dim"])
    o = o.permute(0, 3, 1, 2, 4).reshape(S, L, hk * G, c["dim"])
    st["out"][index[there]] = o[there].to(st["out"].dtype)
    return st["out"]


def _plain_verify(st):
    c = st["case"]
    _plain_attend(st)
    lens, starts = st["lens"].long(), st["starts"].long()
    first = lens - (starts[1:] - starts[:-1])
    i = torch.arange(st["path"].shape[1], device=DEV)
    moved = i[None, :] < st["path_lens"][:, None]
    src = (first[:, None] + st["path"].long())[moved]
    dst = (first[:, None] + i[None, :])[moved]
    seq = torch.arange(lens.shape[0], device=DEV)[:, None].expand_as(moved)[moved]
    heads = torch.arange(c["kv_heads"], device=DEV)[None, :]
    tables = st["tables"].long()
    for cache in (_values(st["k_cache"]), _values(st["v_cache"])):
        rows = cache[tables[seq, src // c["block"]][:, None], heads, (src % c["block"])[:, None]]
        cache[tables[seq, dst // c["block"]][:, None], heads, (dst % c["block"])[:, None]] = rows
    st["new_lens"].copy_((first + st["path_lens"]).to(torch.int32))
    return {"out": st["out"], "new_lens": st["new_lens"], "k_cache": _values(st["k_cache"]),
            "v_cache": _values(st["v_cache"])}


def _plain_accumulate(st):
    c = st["case"]
    p, index, there = _weights(st)
    S, hk, G, L, T = p.shape
    o = torch.matmul(p.view(S, hk, G, T), _rows(st, "v"))
    st["out"].copy_(o.reshape(S, hk * G, c["dim"]))
    st["mass"][:, :, :T] += p.sum((2, 3))
    return {"out": st["out"], "mass": st["mass"]}


def _plain_evict(st):
    c = st["case"]
    lens = st["lens"].long()[:, None, None]
    S, hk, width = st["mass"].shape
    t = torch.arange(width, device=DEV)[None, None, :]
    # every kept token has a rank below the budget: the always-kept ones first, then by weight, then by position
    always = (t < c["sinks"]) | (t >= lens - c["recent"])
    key = torch.where(always, torch.full_like(st["mass"], math.inf), st["mass"])
    key = torch.where(t < lens, key, torch.full_like(key, -math.inf))
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(order)
    rank.scatter_(2, order, torch.arange(width, device=DEV).expand_as(order))
    keep = (rank < c["budget"]) & (t < lens)
    s, h, src = keep.nonzero(as_tuple=True)
    dst = (keep.cumsum(-1) - 1)[s, h, src]
    st["kept"][s, h, dst] = src.to(torch.int32)
    st["mass_out"][s, h, dst] = st["mass"][s, h, src]
    st["new_lens"].copy_(lens.view(-1).clamp(max=c["budget"]).to(torch.int32))
    from_block, to_block = st["tables"].long()[s, src // c["block"]], st["dst_tables"].long()[s, dst // c["block"]]
    for cache in (_values(st["k_cache"]), _values(st["v_cache"])):
        cache[to_block, h, dst % c["block"]] = cache[from_block, h, src % c["block"]]
    return {"kept": st["kept"], "mass": st["mass_out"], "new_lens": st["new_lens"], "k_cache": _values(st["k_cache"]),
            "v_cache": _values(st["v_cache"])}


_PLAIN = {"rope": _plain_rope, "attend": _plain_attend, "verify": _plain_verify, "accumulate": _plain_accumulate,
          "evict": _plain_evict}


# ------------------------------------------------------------------------------------------------ from the definition

def exact(case, seed):
    st = prepare(case, seed)
    if case["kind"] == "rope":
        return _exact_rope(st)
    if case["kind"] == "evict":
        return None  # whole numbers and moved rows: nothing is computed
    out = torch.zeros(st["q"].shape, device=DEV, dtype=torch.float64)
    mass = st["mass"].double() if case["kind"] == "accumulate" else None
    lens, starts = st["lens"].tolist(), st["starts"].tolist()
    hk, g = case["kv_heads"], case["heads"] // case["kv_heads"]
    for s, t in enumerate(lens):
        blocks = st["tables"][s, :-(-t // case["block"])].long()
        n = starts[s + 1] - starts[s]
        seen = torch.zeros((n, t), dtype=torch.bool)
        if case["kind"] == "verify":
            seen[:, :t - n] = True
            for i, anc in enumerate(_tree(case, n)):
                seen[i, [t - n + a for a in anc]] = True
        else:
            p = torch.arange(t)
            for i in range(n):
                at = t - n + i
                row = p <= at
                if case.get("window"):
                    row &= p >= at - case["window"] + 1
                if case.get("prefix"):
                    row |= p < case["prefix"]
                seen[i] = row
        seen = seen.to(DEV)
        for h in range(hk):
            kk, vv = (_head64(st, w, blocks, h, t) for w in ("k", "v"))
            for j in range(g):
                qq = st["q"][starts[s]:starts[s + 1], h * g + j].double()
                x = (qq @ kk.T) / math.sqrt(case["dim"])
                if case["cap"]:
                    x = torch.tanh(x / case["cap"]) * case["cap"]
                if case.get("bias"):
                    at = torch.arange(t - n, t, device=DEV)[:, None]
                    x = x - st["slopes"][h * g + j].double() * (at - torch.arange(t, device=DEV)[None]).abs()
                x = torch.where(seen, x, torch.full_like(x, -math.inf))
                w = torch.softmax(x, -1)
                out[starts[s]:starts[s + 1], h * g + j] = w @ vv
                if mass is not None:
                    mass[s, h, :t] += w[0]
    if case["kind"] == "verify":
        return {"out": out, "new_lens": None, "k_cache": None, "v_cache": None}
    return out if mass is None else {"out": out, "mass": mass}


def _head64(st, which, blocks, head, t):
    x = st[which + "_cache"][:, head].view(torch.uint8)[blocks].view(st[which + "_cache"].dtype).double()
    x = x.reshape(-1, st["case"]["dim"])[:t]
    if st[which + "_zp"] is not None:
        x = x - float(st[which + "_zp"][head])
    if st[which + "_scale"] is not None:
        x = x * st[which + "_scale"][head].double()
    return x


def _exact_rope(st):
    c = st["case"]
    half = c["rotary"] // 2
    q, k, v = st["q"].double(), st["k"].double(), st["v"].double()
    theta = torch.outer(st["positions"].double(), st["inv_freq"].double())
    turn = torch.polar(torch.full_like(theta, c["rope_scale"]), theta)[:, None, :]

    def rotated(x):
        pairs = x[..., :c["rotary"]]
        if c["interleaved"]:
            z = torch.complex(pairs[..., 0::2].contiguous(), pairs[..., 1::2].contiguous()) * turn
            y = torch.stack((z.real, z.imag), -1).flatten(-2)
        else:
            z = torch.complex(pairs[..., :half].contiguous(), pairs[..., half:].contiguous()) * turn
            y = torch.cat((z.real, z.imag), -1)
        return torch.cat((y, x[..., c["rotary"]:]), -1)

    k = rotated(k)
    if c["kv"] == "e4m3":
        k, v = k * st["k_inv"].double()[:, None], v * st["v_inv"].double()[:, None]
    caches = []
    for x in (k, v):
        pool = torch.zeros(st["k_cache"].shape, device=DEV, dtype=torch.float64).transpose(1, 2).contiguous()
        pool.view(-1, c["kv_heads"], c["dim"])[st["slots"]] = x
        caches.append(pool.transpose(1, 2).contiguous())
    return {"q": rotated(q), "k_cache": caches[0], "v_cache": caches[1]}
