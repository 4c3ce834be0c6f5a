"""pa_read_cache against the definition.  code * scale + zero is exact in 64 bits and rounded to float32 once by the kernel,
(code - zero point) * scale and e4m3 * scale are one product: the values are equal, and rounded once more to 16 bits."""

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import int4_cases  # noqa: E402
import paged_kv_cache_144_gb300 as pa  # noqa: E402
from operator_cases import DT, F64, make_cache  # noqa: E402


def pools(kv, blocks, heads, block, dim, g):
    if kv == "i4":
        return (*int4_cases.make_pool(blocks, heads, block, g), None, None)
    return make_cache(kv, blocks, heads, block, dim, g)


def up(t):
    return None if t is None else t.cuda()


def run(n, heads, kv, out, *, dim=128, block=16, seed=0, wide=0, skip=(), repeat=False, stream=None, blocks=None):
    g = torch.Generator().manual_seed(seed)
    blocks = blocks or -(-n // block) + 1
    k, k64, ks, kz = pools(kv, blocks, heads, block, dim, g)
    v, v64, vs, vz = pools(kv, blocks, heads, block, dim, g)
    slots = torch.randint(0, blocks * block, (n,), generator=g) if repeat else torch.randperm(blocks * block, generator=g)[:n]
    slots = slots.contiguous()
    for i in skip:
        slots[i] = -1
    ko = torch.full((n, heads + wide, dim), 9.0, dtype=DT[out], device="cuda")
    vo = torch.full_like(ko, 8.0)
    got = pa.read_cache(ko[:, :heads], vo[:, :heads], k.cuda(), v.cuda(), slots.cuda(), block, k_scale=up(ks), v_scale=up(vs),
                        k_zero_point=up(kz), v_zero_point=up(vz), stream=stream)
    if stream is not None:
        stream.synchronize()
    assert pa.get_device_error() == 0
    for x, whole, x64, fill in ((got[0], ko, k64, 9.0), (got[1], vo, v64, 8.0)):
        want = x64.transpose(1, 2).reshape(-1, heads, dim)[slots.clamp(min=0)].to(torch.float32).to(DT[out])
        want[list(skip)] = fill
        assert torch.equal(x.cpu(), want)
        assert torch.all(whole[:, heads:] == fill)


@pytest.mark.parametrize("kv", ["bf16", "f16", "e4m3", "i8", "i4"])
@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n,heads", [(1, 1), (5, 3), (33, 8), (700, 2)])
def test_types(kv, out, n, heads):
    run(n, heads, kv, out, seed=n)


@pytest.mark.parametrize("kv", ["bf16", "f16", "e4m3", "i8"])
def test_head_size_64(kv):
    run(37, 5, kv, "bf16", dim=64, seed=1)


@pytest.mark.parametrize("block", [8, 32, 256, 1024])
@pytest.mark.parametrize("kv", ["i4", "e4m3"])
def test_block_sizes(block, kv):
    run(300, 3, kv, "f32", block=block, seed=2)


def test_strides_padding_and_repeated_slots():
    for kv in ("i4", "bf16"):
        run(50, 2, kv, "bf16", wide=2, skip=(0, 3, 49), seed=3)
        run(50, 2, kv, "f32", wide=1, skip=tuple(range(50)), seed=4)
        run(200, 2, kv, "f16", repeat=True, blocks=2, seed=5)


def test_k_and_v_side_by_side_in_one_buffer():
    g = torch.Generator().manual_seed(6)
    k, k64, _, _ = pools("i4", 3, 2, 16, 128, g)
    both = torch.zeros((10, 4, 128), device="cuda")
    slots = torch.arange(20, 30)
    pa.read_cache(both[:, :2], both[:, 2:], k.cuda(), k.cuda(), slots.cuda(), 16)
    want = k64.transpose(1, 2).reshape(-1, 2, 128)[slots].float()
    assert torch.equal(both[:, :2].cpu(), want) and torch.equal(both[:, 2:].cpu(), want)


def test_another_stream():
    run(100, 4, "i4", "bf16", seed=7, stream=torch.cuda.Stream())


def test_slot_outside_the_pool_is_skipped():
    c = torch.zeros(pa.int4_cache_shape(1, 1, 16), dtype=torch.uint8, device="cuda")
    out = torch.full((3, 1, 128), 4.0, device="cuda")
    pa.read_cache(out, out.clone(), c, c, torch.tensor([15, 16, 1 << 40], device="cuda"), 16)
    assert pa.get_device_error() == pa.PA_DEVERR_SLOT
    assert torch.all(out[0] == 0) and torch.all(out[1:] == 4)


def test_a_pool_beyond_32_bit_offsets():
    """Rows on both sides of 4 GB, of tiles written through the library."""
    block, heads = 64, 8
    shape = pa.int4_cache_shape(140000, heads, block)       # 140000 * 8 * 64 * 68 bytes = 4.9 GB
    k, v = (torch.zeros(shape, dtype=torch.uint8, device="cuda") for _ in range(2))
    slots = torch.tensor([0, 63, 124000 * block + 5, 139999 * block + 63], device="cuda")
    x = torch.randn((4, heads, 128), generator=torch.Generator().manual_seed(8)).to(torch.bfloat16).cuda()
    pa.reshape_and_cache(x, -x, k, v, slots, block)
    out = torch.zeros((4, heads, 128), device="cuda")
    pa.read_cache(out, out2 := torch.zeros_like(out), k, v, slots, block)
    assert pa.get_device_error() == 0
    for got, want in ((out, x), (out2, -x)):
        w = want.float()
        step = (w.amax(-1, keepdim=True) - w.amin(-1, keepdim=True)) / 15
        # half a code, the pair's roundings to float16 (2^-11 of the bound; of the scale, 15 times), two float32 roundings
        assert torch.all((got - w).abs() <= step * (0.5 + 15 * 2.0 ** -11) + 2.0 ** -10 * w.abs().amax(-1, keepdim=True))
    assert int((k != 0).any(-1).sum()) == 3 * heads  # the first two rows share their tiles


def test_written_then_read_with_queries_of_another_type_captured():
    k = torch.randn((20, 2, 128), generator=torch.Generator().manual_seed(9)).to(torch.float16).cuda()
    kc, vc = (torch.zeros(pa.int4_cache_shape(2, 2, 16), dtype=torch.uint8, device="cuda") for _ in range(2))
    slots = torch.arange(20, device="cuda")
    outs = [torch.zeros((20, 2, 128), device="cuda") for _ in range(4)]

    def step(a, b):
        pa.reshape_and_cache(k, k, kc, vc, slots, 16, pdl=True)
        pa.read_cache(a, b, kc, vc, slots, 16, pdl=True)

    step(outs[0], outs[1])
    graph = pa.StepGraph(lambda: step(outs[2], outs[3]))
    outs[2].zero_(), outs[3].zero_(), kc.zero_(), vc.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[2]) and torch.equal(outs[0], outs[3]) and outs[0].abs().max() > 0
