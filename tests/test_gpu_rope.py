"""pa_rope_and_cache against the definition in 64 bits.

A turned value is x cos a - y sin a in float32 from angles exact to about 2^-31 turns: its error is below 1e-6 (|x| +
|y|) before the one rounding to its type (half a step).  An 8-bit code may differ from the exact one where that error
crosses a rounding border: it is then a neighbouring code, so the value it stands for is within one step.
"""

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import paged_kv_cache_144_gb300 as pa  # noqa: E402
from operator_cases import DT, F64, HALF_STEP, rope_reference  # noqa: E402


def _run(n, hq, hk, dim, rotary, *, src="bf16", kv=None, interleaved=False, block=16, seed=0, scale=1.0, pos_max=5000,
         in_place=False, pad=0, skip=(), inv=None, pdl=False):
    kv = kv or src
    g = torch.Generator().manual_seed(seed)
    blocks = -(-n // block) + 2

    def rows(h):
        return torch.randn((n, h + pad, dim), generator=g).to(DT[src])[:, :h]

    q, k, v = rows(hq), rows(hk), rows(hk)
    pos = torch.randint(0, pos_max, (n,), generator=g)
    slots = torch.randperm(blocks * block, generator=g)[:n].contiguous()
    for i in skip:
        slots[i] = -1
    inv = pa.rope_frequencies(rotary) if inv is None else inv
    fill = {"f16": 3.0, "bf16": 3.0, "e4m3": 3.0, "i8": 3}[kv]
    kc = torch.full((blocks, hk, block, dim), fill).to(DT[kv]).cuda()
    vc = kc.clone()
    kis = vis = kz = vz = None
    if kv in ("e4m3", "i8"):
        kis, vis = 20 + 10 * torch.rand(hk, generator=g), 20 + 10 * torch.rand(hk, generator=g)
        if kv == "i8":
            kz = torch.randint(-20, 21, (hk,), generator=g, dtype=torch.int32)
            vz = torch.randint(-20, 21, (hk,), generator=g, dtype=torch.int32)
    wide = torch.zeros((n, hq + pad, dim), dtype=DT[src], device="cuda")
    wide[:, :hq] = q.cuda()
    qd = wide[:, :hq]
    q_out = None if in_place else torch.full((n, hq, dim), 5.0, dtype=DT[src], device="cuda")
    up = lambda t: None if t is None else t.cuda()  # noqa: E731
    kw, vw = (torch.zeros((n, hk + pad, dim), dtype=DT[src], device="cuda") for _ in range(2))
    kw[:, :hk], vw[:, :hk] = k.cuda(), v.cuda()
    got = pa.rope_and_cache(qd, kw[:, :hk], vw[:, :hk], kc, vc, pos.cuda(), slots.cuda(), inv.cuda(), block,
                            q_out=q_out, interleaved=interleaved, rope_scale=scale, k_inv_scale=up(kis),
                            v_inv_scale=up(vis), k_zero_point=up(kz), v_zero_point=up(vz), pdl=pdl)
    err = pa.get_device_error()
    live = [i for i in range(n) if slots[i] >= 0]
    want_q, want_k = rope_reference(q, pos, inv, interleaved, scale), rope_reference(k, pos, inv, interleaved, scale)
    slack = lambda x: 2e-6 * (x.abs().amax(-1, keepdim=True).to(F64) + 1) * 2 * scale  # noqa: E731
    got = got.cpu().to(F64)
    assert torch.all((got[live] - want_q[live]).abs() <= (HALF_STEP[src] * want_q.abs() + slack(q))[live])
    for i in skip:
        assert torch.all(got[i] == (q[i].to(F64) if in_place else 5.0))
    for cache, want, src_rows, inv_s, zp in ((kc, want_k, k, kis, kz), (vc, v.to(F64), v, vis, vz)):
        flat = cache.cpu().to(torch.float32).to(F64) if kv != "i8" else cache.cpu().to(F64)
        flat = flat.transpose(1, 2).reshape(blocks * block, hk, dim)
        rows_got = flat[slots[live]]
        w = want[live]
        if kv in ("f16", "bf16"):
            assert torch.all((rows_got - w).abs() <= HALF_STEP[kv] * w.abs() + slack(src_rows)[live])
            if cache is vc:
                assert torch.equal(rows_got, w)                     # copied bits
        else:
            y = w * inv_s.to(F64)[None, :, None]
            if kv == "e4m3":
                y = y.clamp(-448, 448)
                step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
                off = (rows_got - y).abs()
            else:
                y = (y + zp.to(F64)[None, :, None]).clamp(-128, 127)
                step = torch.ones_like(y)
                off = (rows_got - y).abs()
            near = slack(src_rows)[live] * inv_s.to(F64)[None, :, None] + 2.0 ** -23 * y.abs()
            assert torch.all(off <= step / 2 + near), off.max()
        untouched = torch.ones(blocks * block, dtype=torch.bool)
        untouched[slots[live]] = False
        assert torch.all(flat[untouched] == 3.0)
    assert err == 0
    return got


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("src,kv,dim", [("bf16", "bf16", 128), ("f16", "f16", 64), ("bf16", "e4m3", 128),
                                        ("f16", "i8", 128), ("f16", "e4m3", 64), ("bf16", "i8", 64)])
@pytest.mark.parametrize("part", ["all", "half", 2, 10, 24, 32])
def test_rope_layouts_and_types(interleaved, src, kv, dim, part):
    r = dim if part == "all" else dim // 2 if part == "half" else part
    _run(19, 6, 2, dim, r, src=src, kv=kv, interleaved=interleaved, seed=1)


@pytest.mark.parametrize("n", [1, 2, 3, 129, 1000])
@pytest.mark.parametrize("in_place", [False, True])
def test_rope_token_counts(n, in_place):
    _run(n, 8, 8, 128, 128, in_place=in_place, seed=2)
    _run(n, 3, 1, 64, 24, src="f16", in_place=in_place, seed=2)


def test_rope_padding_tokens_are_left_alone():
    for in_place in (False, True):
        _run(10, 4, 2, 128, 64, skip=(0, 4, 9), in_place=in_place, seed=3)
        _run(10, 4, 2, 128, 20, skip=(0, 4, 9), in_place=in_place, seed=3)


def test_rope_strided_rows_and_scale():
    _run(33, 5, 3, 128, 96, pad=2, scale=1.3, seed=4)
    _run(33, 5, 3, 128, 96, pad=2, scale=1.3, seed=4, interleaved=True, in_place=True)


def test_rope_far_positions():
    """Positions up to 2^31: the reduced angle stays exact to 2^-30 turns of the float32 frequency's product.

    The product with 1 / (2 pi) in 53 bits is off by at most 2^-56 turns a position, 2^-25 at 2^31."""
    _run(64, 2, 1, 128, 128, pos_max=1 << 20, seed=5, src="f16")
    g = torch.Generator().manual_seed(6)
    pos = (1 << 31) - 1 - torch.randint(0, 1000, (16,), generator=g)
    q = torch.ones((16, 1, 64), dtype=torch.float16)
    inv = pa.rope_frequencies(64)
    kc = torch.zeros((2, 1, 16, 64), dtype=torch.float16, device="cuda")
    got = pa.rope_and_cache(q.cuda(), q.cuda(), q.cuda(), kc, kc.clone(), pos.cuda(),
                            torch.arange(16, device="cuda"), inv.cuda(), 16, q_out=torch.empty_like(q, device="cuda"))
    want = rope_reference(q, pos, inv, False, 1.0)
    # 64-bit reference angles of 2^31 radians are themselves off by 2^-22
    assert torch.all((got.cpu().to(F64) - want).abs() <= 2 * (2.0 ** -11 + 2.0 ** -21))


def test_rope_stretched_frequencies():
    for kw in (dict(scaling="linear", factor=4.0), dict(scaling="base", factor=8.0),
               dict(scaling="bands", factor=8.0, original_positions=8192)):
        _run(40, 2, 2, 128, 128, inv=pa.rope_frequencies(128, 500000.0, **kw), pos_max=100000, src="f16", seed=7)


def test_rope_dependent_launch_gives_the_same():
    a = _run(50, 4, 2, 128, 128, seed=8)
    b = _run(50, 4, 2, 128, 128, seed=8, pdl=True)
    assert torch.equal(a, b)


def test_rope_equals_cache_write_without_turn():
    """Position 0 turns nothing: the caches hold the bytes of the plain cache write, quantised ones too."""
    g = torch.Generator().manual_seed(9)
    q = torch.randn((30, 4, 128), generator=g).bfloat16().cuda()
    k, v = (torch.randn((30, 2, 128), generator=g).bfloat16().cuda() for _ in range(2))
    slots = torch.randperm(64, generator=g)[:30].cuda()
    inv = torch.full((2,), 25.0, device="cuda")
    for t in ("bf16", "e4m3"):
        a, b, c, d = (torch.zeros((4, 2, 16, 128), device="cuda").to(DT[t]) for _ in range(4))
        kw = {} if t == "bf16" else dict(k_inv_scale=inv, v_inv_scale=inv)
        pa.reshape_and_cache(k, v, a, b, slots, 16, **kw)
        qo = pa.rope_and_cache(q, k, v, c, d, torch.zeros(30, dtype=torch.int64, device="cuda"), slots,
                               pa.rope_frequencies(128).cuda(), 16, q_out=torch.empty_like(q), **kw)
        assert torch.equal(qo, q)
        assert torch.equal(a.view(torch.uint8), c.view(torch.uint8)) and torch.equal(b.view(torch.uint8), d.view(torch.uint8))


def test_rope_slot_out_of_range_is_reported():
    q = torch.ones((2, 1, 64), dtype=torch.float16, device="cuda")
    kc = torch.zeros((2, 1, 16, 64), dtype=torch.float16, device="cuda")
    out = torch.full_like(q, 5.0)
    pa.rope_and_cache(q, q, q, kc, kc.clone(), torch.zeros(2, dtype=torch.int64, device="cuda"),
                      torch.tensor([3, 32], device="cuda"), pa.rope_frequencies(64).cuda(), 16, q_out=out)
    assert pa.get_device_error() == pa.PA_DEVERR_SLOT
    assert torch.all(out[0] == 1) and torch.all(out[1] == 5)
