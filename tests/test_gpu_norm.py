"""pa_norm_rope_and_cache, and the writes into a 4-bit cache, against the definition in 64 bits.

A normed value is x * inv * w in float32: the sum of at most 128 squares is off by at most 24 roundings of its partial sums
(16 in a thread, 3 exchanges, the mean), rsqrtf by 2 steps, two products by one each: below 2^-19 of the value.  Turned, it
is off by 1e-6 (|x| + |y|) more (test_gpu_rope.py).  Both are below 4e-6 of the row's largest value.
"""

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import int4_cases  # noqa: E402
import paged_kv_cache_144_gb300 as pa  # noqa: E402
from operator_cases import DT, F64, HALF_STEP, rope_reference  # noqa: E402


def normed(x, w, eps, offset):
    x = x.to(F64)
    if w is None:
        return x
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * (w.to(F64) + offset)


def run(n, hq, hk, dim=128, rotary=128, *, src="bf16", kv=None, interleaved=False, block=16, seed=0, scale=1.0, offset=0.0,
        eps=1e-6, weights="both", wt=None, in_place=False, pad=0, skip=(), call="norm", rows=None, pos_max=5000, stream=None):
    kv = kv or src
    g = torch.Generator().manual_seed(seed)
    blocks = -(-n // block) + 2

    def make(h):
        x = torch.randn((n, h + pad, dim), generator=g) * torch.exp2(torch.randint(-6, 7, (n, h + pad, 1), generator=g))
        return x.to(DT[src])[:, :h]

    q, k, v = make(hq), make(hk), make(hk)
    if rows is not None:
        rows(q, k, v)
    pos = torch.randint(-pos_max, pos_max, (n,), generator=g)
    slots = torch.randperm(blocks * block, generator=g)[:n].contiguous()
    for i in skip:
        slots[i] = -1
    inv = pa.rope_frequencies(rotary) if rotary else None
    wt = DT[wt or src]
    qw = (1 + 0.3 * torch.randn(dim, generator=g)).to(wt) if weights == "both" else None
    kw = (1 + 0.3 * torch.randn(dim, generator=g)).to(wt) if weights in ("both", "k") else None
    if kv == "i4":
        kc = torch.full(pa.int4_cache_shape(blocks, hk, block), 0x33, dtype=torch.uint8, device="cuda")
    else:
        kc = torch.full((blocks, hk, block, dim), 3.0).to(DT[kv]).cuda()
    vc = kc.clone()
    kis = vis = kz = vz = None
    if kv in ("e4m3", "i8"):
        kis, vis = 20 + 10 * torch.rand(hk, generator=g), 20 + 10 * torch.rand(hk, generator=g)
        if kv == "i8":
            kz = torch.randint(-20, 21, (hk,), generator=g, dtype=torch.int32)
            vz = torch.randint(-20, 21, (hk,), generator=g, dtype=torch.int32)
    up = lambda t: None if t is None else t.cuda()  # noqa: E731

    def strided(x):
        wide = torch.zeros((n, x.shape[1] + pad, dim), dtype=DT[src], device="cuda")
        wide[:, :x.shape[1]] = x.cuda()
        return wide[:, :x.shape[1]]

    qd, kd, vd = strided(q), strided(k), strided(v)
    q_out = None if in_place else torch.full((n, hq, dim), 5.0, dtype=DT[src], device="cuda")
    kws = dict(k_inv_scale=up(kis), v_inv_scale=up(vis), k_zero_point=up(kz), v_zero_point=up(vz), stream=stream)
    if call == "norm":
        got = pa.norm_rope_and_cache(qd, kd, vd, kc, vc, up(pos) if rotary else None, slots.cuda(), up(inv), block,
                                     q_weight=up(qw), k_weight=up(kw), eps=eps, weight_offset=offset, q_out=q_out,
                                     interleaved=interleaved, rope_scale=scale, **kws)
    elif call == "rope":
        got = pa.rope_and_cache(qd, kd, vd, kc, vc, up(pos), slots.cuda(), up(inv), block, q_out=q_out,
                                interleaved=interleaved, rope_scale=scale, **kws)
    else:
        pa.reshape_and_cache(kd, vd, kc, vc, slots.cuda(), block)
        got = None
    if stream is not None:
        stream.synchronize()
    assert pa.get_device_error() == 0
    live = [i for i in range(n) if slots[i] >= 0]
    place = (lambda x: rope_reference(x, pos, inv, interleaved, scale)) if rotary and call != "plain" else (lambda x: x)
    want_k = place(normed(k, kw if call == "norm" else None, eps, offset))
    if got is not None:
        want = place(normed(q, qw if call == "norm" else None, eps, offset))
        got = got.cpu().to(F64)
        slack = 4e-6 * want.abs().amax(-1, keepdim=True)
        assert torch.all((got[live] - want[live]).abs() <= (HALF_STEP[src] * want.abs() + slack + 1e-7)[live])
        for i in skip:
            assert torch.all(got[i] == (q[i].to(F64) if in_place else 5.0))
    for name, cache, want, inv_s, zp in (("k", kc, want_k, kis, kz), ("v", vc, v.to(F64), vis, vz)):
        slack = 4e-6 * want.abs().amax(-1, keepdim=True) + 1e-9 if name == "k" else torch.zeros_like(want[..., :1])
        untouched = torch.ones(blocks * block, dtype=torch.bool)
        untouched[slots[live]] = False
        if kv == "i4":
            tiles = cache.cpu()
            int4_cases.check_rows(tiles, block, slots[live], want[live], slack[live])
            codes, sc, _ = int4_cases.unpack(tiles, block)
            assert torch.all(codes.transpose(1, 2).reshape(-1, hk, dim)[untouched] == 3)
            assert torch.all(sc.transpose(1, 2).reshape(-1, hk)[untouched] == 0.2249755859375)  # 0x3333
            continue
        flat = cache.cpu().to(torch.float32).to(F64) if kv != "i8" else cache.cpu().to(F64)
        flat = flat.transpose(1, 2).reshape(blocks * block, hk, dim)
        rows_got, w = flat[slots[live]], want[live]
        if kv in ("f16", "bf16"):
            assert torch.all((rows_got - w).abs() <= HALF_STEP[kv] * w.abs() + slack[live] + 2.0 ** -25)
        else:
            y = w * inv_s.to(F64)[None, :, None]
            if kv == "e4m3":
                y = y.clamp(-448, 448)
                step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
            else:
                y = (y + zp.to(F64)[None, :, None]).clamp(-128, 127)
                step = torch.ones_like(y)
            near = slack[live] * inv_s.to(F64)[None, :, None] + 2.0 ** -23 * (y.abs() + 128)
            assert torch.all((rows_got - y).abs() <= step / 2 + near)
        assert torch.all(flat[untouched] == 3.0)


@pytest.mark.parametrize("kv", ["bf16", "f16", "e4m3", "i8", "i4"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n,hq,hk", [(1, 1, 1), (3, 4, 2), (65, 8, 8), (7, 14, 2)])
def test_norms_types_and_heads(kv, interleaved, n, hq, hk):
    run(n, hq, hk, src=kv if kv in ("bf16", "f16") else "bf16", kv=kv, interleaved=interleaved, seed=n)


@pytest.mark.parametrize("rotary", [0, 2, 10, 24, 32, 64, 126, 128])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("kv", ["f16", "i4"])
def test_part_of_the_head_turned(rotary, interleaved, kv):
    run(21, 4, 2, rotary=rotary, src="f16", kv=kv, interleaved=interleaved, seed=rotary)


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "i8"])
@pytest.mark.parametrize("rotary", [0, 10, 64])
def test_head_size_64(kv, rotary):
    run(19, 6, 3, dim=64, rotary=rotary, kv=kv, seed=2)
    run(19, 6, 3, dim=64, rotary=rotary, kv=kv, seed=2, interleaved=True)


@pytest.mark.parametrize("weights", ["none", "k", "both"])
@pytest.mark.parametrize("wt", ["f32", "f16", "bf16"])
def test_weights(weights, wt):
    run(9, 4, 2, weights=weights, wt=wt, offset=1.0, eps=1e-5, scale=1.2, seed=3)
    run(9, 4, 2, weights=weights, wt=wt, kv="i4", seed=4)


@pytest.mark.parametrize("kv", ["bf16", "i4"])
def test_in_place_strided_and_padded(kv):
    run(40, 8, 2, kv=kv, in_place=True, pad=3, skip=(0, 7, 39), seed=5)
    run(40, 8, 2, kv=kv, pad=1, skip=tuple(range(40)), seed=6)


@pytest.mark.parametrize("block", [8, 64, 1024])
def test_int4_blocks_through_every_write(block):
    for call in ("norm", "rope", "plain"):
        run(150, 4, 3, kv="i4", block=block, call=call, seed=7, interleaved=block == 64)
        run(33, 4, 3, src="f16", kv="i4", block=block, call=call, seed=8)


def test_many_tokens_fill_every_slice():
    run(2050, 32, 8, kv="i4", seed=9)
    run(1025, 5, 5, kv="bf16", seed=10)


def test_another_stream():
    run(33, 4, 2, kv="i4", seed=11, stream=torch.cuda.Stream())


def _write_rows(x):
    """The 4-bit rows of x [N, d] (as V of one head) through reshape_and_cache."""
    n = x.shape[0]
    c = torch.zeros(pa.int4_cache_shape(-(-n // 8), 1, 8), dtype=torch.uint8, device="cuda")
    d = x.reshape(n, 1, 128).contiguous().cuda()
    pa.reshape_and_cache(d, d, torch.zeros_like(c), c, torch.arange(n, device="cuda"), 8)
    assert pa.get_device_error() == 0
    codes, scale, zero = int4_cases.unpack(c.cpu(), 8)
    return codes[:, 0].reshape(-1, 128)[:n], scale.reshape(-1)[:n], zero.reshape(-1)[:n]


def test_int4_rows_at_the_borders():
    """Rows of one value, exact halves, infinities and NaN, bounds beyond the clip, tiny rows."""
    x = torch.zeros((9, 128))
    x[1] = 0.1                                            # one value: scale 0, code 0, the value rounded to float16
    x[2] = torch.arange(128) % 31 * 0.5                   # zero 0, scale 1: halves go to the even code
    x[3] = torch.linspace(-1, 1, 128)
    x[3, 5], x[3, 9] = float("inf"), float("-inf")
    x[4] = torch.linspace(0, 15, 128)
    x[4, 7] = float("nan")
    x[5] = float("nan")
    x[6] = torch.linspace(-1e5, 1e5, 128)
    x[7] = torch.linspace(0, 1e-7, 128)
    x[8] = -torch.arange(128) % 16 * 2.0 ** -24
    x = x.to(torch.bfloat16)
    codes, scale, zero = _write_rows(x)
    assert scale[0] == 0 and zero[0] == 0 and torch.all(codes[0] == 0)
    assert scale[1] == 0 and zero[1] == x[1, 0].half().to(F64) and torch.all(codes[1] == 0)
    assert scale[2] == 1 and zero[2] == 0
    assert torch.equal(codes[2], torch.round(x[2].to(F64)).to(torch.int64))
    assert zero[3] == -32768 and codes[3, 5] == 15 and codes[3, 9] == 0 and scale[3] == torch.tensor(65536 / 15).half()
    assert zero[4] == 0 and scale[4] == 1 and codes[4, 7] == 0 and codes[4, 127] == 15
    assert scale[5] == 0 and zero[5] == 0 and torch.all(codes[5] == 0)
    assert zero[6] == -32768 and torch.isfinite(codes[6] * scale[6] + zero[6]).all()
    assert (codes[6] * scale[6] + zero[6]).abs().max() < 65504
    for i in (7, 8):                                      # below float16's normal numbers: within a step of its smallest
        y = codes[i] * scale[i] + zero[i]
        assert torch.all((y - x[i].to(F64)).abs() <= scale[i] / 2 + 15 * 2.0 ** -25 + 2.0 ** -25)


def test_rows_with_infinity_follow_the_formula():
    """An infinite value makes the row's norm infinite: 0 where the row is finite, NaN where it is not."""
    q = torch.randn((2, 1, 128)).to(torch.bfloat16)
    q[1, 0, 3] = float("inf")
    c = torch.zeros((1, 1, 16, 128), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(128, device="cuda")
    out = pa.norm_rope_and_cache(q.cuda(), q.cuda(), q.cuda(), c, c.clone(), None, torch.arange(2, device="cuda"), None, 16,
                                 q_weight=w, k_weight=w).cpu()
    assert torch.isfinite(out[0]).all() and torch.isnan(out[1, 0, 3])
    rest = torch.cat((out[1, 0, :3], out[1, 0, 4:]))
    assert torch.all(rest == 0)


def test_slot_outside_the_pool_is_skipped():
    q = torch.ones((2, 1, 128), dtype=torch.bfloat16, device="cuda")
    c = torch.zeros(pa.int4_cache_shape(1, 1, 16), dtype=torch.uint8, device="cuda")
    slots = torch.tensor([16, 3], device="cuda")
    out = torch.zeros_like(q)
    pa.norm_rope_and_cache(q, q, q, c, c.clone(), None, slots, None, 16, q_out=out)
    assert pa.get_device_error() == pa.PA_DEVERR_SLOT
    assert torch.all(out[0] == 0) and torch.all(out[1] == 1)


def test_captured_and_replayed():
    n, block = 37, 16
    g = torch.Generator().manual_seed(12)
    q, k, v = (torch.randn((n, h, 128), generator=g).to(torch.bfloat16).cuda() for h in (4, 2, 2))
    caches = [torch.zeros(pa.int4_cache_shape(5, 2, block), dtype=torch.uint8, device="cuda") for _ in range(4)]
    pos, slots = torch.arange(n, device="cuda"), torch.randperm(80, generator=g)[:n].cuda()
    inv, w = pa.rope_frequencies(128).cuda(), torch.ones(128, device="cuda")
    outs = [torch.zeros_like(q) for _ in range(2)]

    def step(i):
        pa.norm_rope_and_cache(q, k, v, caches[2 * i], caches[2 * i + 1], pos, slots, inv, block, q_weight=w, k_weight=w,
                               q_out=outs[i], pdl=True)

    step(0)
    graph = pa.StepGraph(lambda: step(1))
    for t in (outs[1], caches[2], caches[3]):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1]) and torch.equal(caches[0], caches[2]) and torch.equal(caches[1], caches[3])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("where", ["far", "far_negative", "edges", "large_frequencies"])
def test_far_positions_and_large_frequencies(interleaved, where):
    """Angles against exact ones: at most 2^-26 turns for the float32 nearest to the fraction, 2^-32 for the bits below it, and
    2^-62 for the step, times |p| <= 2^31.  The rest as in test_gpu_rope_far.py, whose exact angles these are: p = 2^16 h + l,
    both times a float32 of at most 24 bits exact in 64."""
    import math
    from test_gpu_rope_far import exact_cos_sin
    g = torch.Generator().manual_seed(60)
    n = 64
    near = torch.randint(0, 5000, (n,), generator=g)
    pos = {"far": (1 << 31) - 1 - near, "far_negative": near - (1 << 31), "large_frequencies": near - 2500,
           "edges": torch.tensor([0, 1, -1, (1 << 31) - 1, -(1 << 31), 1 << 30, -(1 << 30), 65535] * 8)}[where]
    inv = pa.rope_frequencies(128)
    if where == "large_frequencies":                       # 2^-140 .. 2^20 and both signs (exact in 64 bits with such positions)
        inv = torch.exp2(torch.linspace(-140, 20, 64, dtype=F64)).float() * torch.where(torch.arange(64) % 2 == 0, 1.0, -1.0)
    q = torch.randn((n, 3, 128), generator=g).to(torch.float16)
    c = torch.zeros((n // 16, 3, 16, 128), dtype=torch.float16, device="cuda")
    got = pa.norm_rope_and_cache(q.cuda(), q.cuda(), q.cuda(), c, c.clone(), pos.cuda(), torch.arange(n, device="cuda"), inv.cuda(),
                                 16, q_out=torch.empty_like(q, device="cuda"), interleaved=interleaved).cpu().to(F64)
    assert pa.get_device_error() == 0
    cos, sin = exact_cos_sin(pos, inv)
    i = torch.arange(64)
    lo, hi = (2 * i, 2 * i + 1) if interleaved else (i, i + 64)
    x = q.to(F64)
    a, b = x[..., lo], x[..., hi]
    turns = 2.0 ** -26 + 2.0 ** -32 + 2.0 ** -31
    size = (2 * math.pi * turns + 2.0 ** -21) * (a.abs() + b.abs())
    for column, want in ((lo, a * cos[:, None] - b * sin[:, None]), (hi, b * cos[:, None] + a * sin[:, None])):
        assert torch.all((got[..., column] - want).abs() <= HALF_STEP["f16"] * (want.abs() + size) + size)


def test_halves_between_16_bit_values_go_to_the_even_code():
    """Rows whose quotients are whole numbers and halves of a scale that is no power of two: (x - zero) / scale is exact."""
    scale = torch.tensor([3.0, 5.0, 7.0, 0.375, 1.25])
    rows = []
    for s in scale.tolist():
        y = torch.arange(128) % 31 * 0.5                   # 0, 0.5 .. 15
        rows.append(y * s)
    x = torch.stack(rows).to(torch.float16)                # exact: 5 bits times 3
    codes, sc, zero = _write_rows(x)
    assert torch.equal(sc, scale.to(F64)) and torch.all(zero == 0)
    want = torch.round(torch.arange(128) % 31 * 0.5).to(torch.int64)
    assert torch.equal(codes, want.expand(5, -1))
