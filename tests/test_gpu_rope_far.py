"""pa_rope_and_cache at positions near +-2^31 and below zero, against angles that are exact in 64 bits.

Bound on the angle, in turns: the float32 nearest to the position's fraction of a turn, 2^-26, and 2^-32 for the bits below it;
and for a frequency of at most 1 its part of a turn, 1 / (2 pi) of it, is a product in 53 bits with a constant of 53 bits, off by
at most 2 * 2^-53 of 0.16, which the position multiplies: |p| 2^-54.6.  Then (x, y) -> x cos a - y sin a in float32: sincospif is
within 2 units in the last place, the factor, the two products and the sum round: at most 2^-21 (|x| + |y|) together.  The
result is rounded to its type once.

The reference splits p = 2^16 h + l: both parts times a float32 are exact in 64 bits, the library's cosine of a 64-bit argument
reduces it exactly, and the sum's cosine follows from theirs."""

import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import paged_kv_cache_144_gb300 as pa  # noqa: E402
from operator_cases import DT, F64, HALF_STEP  # noqa: E402


def exact_cos_sin(pos, inv):
    hi, lo = torch.div(pos, 1 << 16, rounding_mode="floor"), torch.remainder(pos, 1 << 16)
    a = (hi * (1 << 16)).to(F64)[:, None] * inv.to(F64)[None]
    b = lo.to(F64)[:, None] * inv.to(F64)[None]
    return torch.cos(a) * torch.cos(b) - torch.sin(a) * torch.sin(b), torch.sin(a) * torch.cos(b) + torch.cos(a) * torch.sin(b)


@pytest.mark.parametrize("src,dim,rotary", [("bf16", 128, 128), ("f16", 64, 64), ("f16", 128, 20)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("where", ["far", "far_negative", "negative", "edges"])
def test_far_and_negative_positions(src, dim, rotary, interleaved, where):
    g = torch.Generator().manual_seed(50)
    n = 64
    near = torch.randint(0, 5000, (n,), generator=g)
    pos = {"far": (1 << 31) - 1 - near, "far_negative": near - (1 << 31), "negative": -1 - near,
           "edges": torch.tensor([0, 1, -1, (1 << 31) - 1, -(1 << 31), 1 << 30, -(1 << 30), 65535] * 8)}[where]
    q, k, v = (torch.randn((n, h, dim), generator=g).to(DT[src]) for h in (3, 2, 2))
    inv = pa.rope_frequencies(rotary)
    kc = torch.zeros((n // 16, 2, 16, dim), dtype=DT[src], device="cuda")
    vc = torch.zeros_like(kc)
    got_q = pa.rope_and_cache(q.cuda(), k.cuda(), v.cuda(), kc, vc, pos.cuda(), torch.arange(n, device="cuda"), inv.cuda(), 16,
                              q_out=torch.empty_like(q, device="cuda"), interleaved=interleaved)
    assert pa.get_device_error() == 0
    c, s = exact_cos_sin(pos, inv)
    i = torch.arange(rotary // 2)
    lo, hi = (2 * i, 2 * i + 1) if interleaved else (i, i + rotary // 2)
    turns = 2.0 ** -26 + 2.0 ** -32 + pos.abs().to(F64) * 2.0 ** -54.6
    off = (2 * math.pi * turns + 2.0 ** -21)[:, None, None]
    for x, got in ((q, got_q), (k, kc.transpose(1, 2).reshape(n, 2, dim))):
        x, got = x.to(F64), got.cpu().to(F64)
        a, b = x[..., lo], x[..., hi]
        size = off * (a.abs() + b.abs())
        for column, want in ((lo, a * c[:, None] - b * s[:, None]), (hi, b * c[:, None] + a * s[:, None])):
            assert torch.all((got[..., column] - want).abs() <= HALF_STEP[src] * (want.abs() + size) + size)
        assert torch.equal(got[..., rotary:], x[..., rotary:])
    assert torch.equal(vc.transpose(1, 2).reshape(n, 2, dim).cpu(), v)
