"""pa_attend over a 4-bit cache, on the decode kernel and on the tensor cores, against a plain 64-bit implementation over the
values that the cache stands for (bounds: attend_more).  Pairs of rows that no query sees are NaN, table entries of unseen
blocks -1."""

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import int4_cases  # noqa: E402
import paged_kv_cache_144_gb300 as pa  # noqa: E402
from attend_more import Case, check, run  # noqa: E402
from operator_cases import F64  # noqa: E402


@pytest.mark.parametrize("q", ["bf16", "f16"])
@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
def test_decode_step(q, out):
    check(Case([1, 7, 16, 17, 63, 64, 65, 127, 128, 129, 300, 0], [1] * 11 + [0], kv="i4", q=q, seed=1), out)


@pytest.mark.parametrize("q", ["bf16", "f16"])
def test_few_queries(q):
    check(Case([5, 40, 133, 260, 33], [2, 4, 1, 3, 0], kv="i4", q=q, seed=2))


@pytest.mark.parametrize("q", ["bf16", "f16"])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_chunks(q, out):
    check(Case([5, 40, 133, 260, 700], [5, 33, 64, 1, 300], kv="i4", q=q, seed=3), out)


@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (3, 3), (8, 1), (6, 2), (7, 1), (40, 8), (32, 1), (64, 1)])
def test_head_groups(heads, kv_heads):
    check(Case([1, 30, 140, 33], [1, 3, 9, 33], kv="i4", heads=heads, kv_heads=kv_heads, seed=4))
    check(Case([1, 30, 140, 33], [1, 1, 1, 1], kv="i4", heads=heads, kv_heads=kv_heads, seed=5))


@pytest.mark.parametrize("block", [8, 16, 32, 64, 128, 256, 1024])
def test_block_sizes(block):
    check(Case([3, 130, 257, 1030], [1, 1, 1, 1], block=block, kv="i4", heads=4, kv_heads=2, seed=6))
    check(Case([3, 130, 257, 1030], [3, 4, 1, 2], block=block, kv="i4", heads=4, kv_heads=2, seed=7))
    check(Case([3, 130, 257, 1030], [3, 70, 1, 5], block=block, kv="i4", heads=4, kv_heads=2, seed=8))


@pytest.mark.parametrize("window,sinks", [(1, 0), (17, 0), (1, 1), (33, 33), (100, 129), (64, 5000), (130, 4)])
def test_windows_and_sinks(window, sinks):
    check(Case([1, 16, 40, 129, 300, 777], [1] * 6, kv="i4", seed=9, window=window, sinks=sinks))
    check(Case([3, 50, 400, 260], [3, 4, 2, 4], kv="i4", seed=10, window=window, sinks=sinks))
    check(Case([5, 140, 700, 520], [5, 133, 64, 300], kv="i4", seed=11, window=window, sinks=sinks))


@pytest.mark.parametrize("block", [8, 64, 256, 1024])
def test_windows_and_sinks_in_blocks(block):
    for window, sinks in ((70, 5), (900, 40), (200, 300)):
        check(Case([3, 257, 1400, 2100], [3, 70, 1, 5], block=block, kv="i4", heads=4, kv_heads=2, seed=12, window=window,
                   sinks=sinks))
        check(Case([3, 257, 1400, 2100], [1] * 4, block=block, kv="i4", heads=4, kv_heads=2, seed=13, window=window, sinks=sinks))


def test_long_context_split_over_the_device():
    check(Case([20001, 9000], [1, 1], kv="i4", heads=4, kv_heads=1, seed=14))
    check(Case([9001, 4100], [1, 20], kv="i4", heads=4, kv_heads=1, seed=15))
    check(Case([900, 517], [600, 517], kv="i4", heads=4, kv_heads=1, seed=16), "bf16")


def test_many_sequences():
    g = torch.Generator().manual_seed(17)
    lens = torch.randint(0, 90, (300,), generator=g).tolist()
    check(Case(lens, [min(t, 1 + i % 3) for i, t in enumerate(lens)], kv="i4", heads=2, kv_heads=1, seed=17))
    check(Case(lens, [min(t, 40) for t in lens], kv="i4", heads=4, kv_heads=1, seed=18))


@pytest.mark.parametrize("qlens", [[1, 1, 1], [1, 3, 4], [1, 40, 200]])
def test_cap_and_distance_bias(qlens):
    c = Case([5, 200, 300], qlens, kv="i4", seed=19)
    c.slopes = torch.tensor([2.0 ** (-(h + 1)) for h in range(8)])
    check(c)
    c.softcap = 20.0
    check(c)


def test_prefix():
    c = Case([10, 300, 270, 64], [10, 40, 270, 1], kv="i4", seed=20)
    c.prefix = torch.tensor([0, 290, 1000, 64], dtype=torch.int32)
    check(c, spoil=False)


@pytest.mark.parametrize("lens,qlens", [([20, 70, 31, 64], [4, 3, 2, 4]), ([20, 200, 131, 64], [7, 16, 5, 64])])
def test_trees(lens, qlens):
    check(Case(lens, qlens, kv="i4", seed=21).with_tree(), spoil=False)


def test_more_queries_than_tokens():
    got, _, _ = check(Case([3, 1, 40], [5, 9, 2], kv="i4", seed=22))
    assert torch.all(got[:2] == 0) and torch.all(got[5:13] == 0)


def test_weights_added_up():
    for window, sinks in ((0, 0), (65, 6)):
        c = Case([1, 40, 300, 700], [1] * 4, kv="i4", seed=23, window=window, sinks=sinks)
        mass = torch.full((4, 2, c.tables.shape[1] * c.block), 0.5, device="cuda")
        _, _, ref = check(c, mass=mass)
        got = mass.cpu().to(F64) - 0.5
        assert torch.all((got - ref).abs() <= 9e-4 * ref + 2.0 ** -23)
        assert torch.all(got[ref == 0] == 0)


@pytest.mark.parametrize("mult", [2.0 ** 17, 2.0 ** -20])
def test_queries_beyond_the_range_of_float16(mult):
    """bf16 queries enter f16 products times a power of two (as over 8-bit caches): the scale makes up for mult."""
    for qlens in ([1, 1], [3, 40]):
        c = Case([300, 77], qlens, kv="i4", seed=24)
        plain, _, _ = check(c)
        c.q_wide = (c.q_wide.float() * mult).to(torch.bfloat16)
        c.q = c.q_wide[:, :c.heads]
        c.scale /= mult
        got, err = run(c)
        assert err == 0
        assert torch.equal(got, plain)


@pytest.mark.parametrize("value", [2.0 ** 60, float("inf"), float("nan")])
@pytest.mark.parametrize("qlens", [[1, 1], [3, 2], [40, 64]])
def test_a_head_out_of_range_does_not_disturb_the_others(qlens, value):
    """Each query row enters the f16 products times a power of two of its own."""
    c = Case([300, 77], qlens, kv="i4", seed=29)
    ref, wabs, _ = c.reference()
    tol = c.tolerance("f32", ref, wabs)
    c.q_wide = c.q_wide.clone()
    c.q_wide[:, 1, 5] = value
    c.q = c.q_wide[:, :c.heads]
    got, err = run(c)
    assert err == 0
    rest = [0] + list(range(2, c.heads))
    n = sum(qlens)
    assert torch.all((got - ref).abs()[:n, rest] <= tol[:n, rest])


@pytest.mark.parametrize("spread,shift", [(2.0 ** -12, 0.0), (0.05, 40.0), (300.0, -1000.0)])
def test_rows_of_other_sizes(spread, shift):
    """Small values, rows far from zero, large ones.  Queries and scale are chosen so that the scores stay near one; K's size
    enters the bound of the scores (attend_more.Case.tolerance is written for values near one), V's the output."""
    for qlens in ([1, 1], [3, 4], [30, 60]):
        c = Case([300, 77], qlens, kv="i4", seed=25)
        c.k, c.k64 = int4_cases.make_pool(c.blocks, c.kv_heads, c.block, c.g, spread, shift)
        c.v, c.v64 = int4_cases.make_pool(c.blocks, c.kv_heads, c.block, c.g, spread, shift)
        size = (spread ** 2 + shift ** 2) ** 0.5
        c.scale /= size
        check(c)


def test_nan_shows_where_it_is_seen():
    for qlens in ([1], [3], [70]):
        c = Case([300], qlens, kv="i4", seed=26)
        b, r = c.row_of(0, 270)
        pairs = c.v[..., c.block * 64:].view(torch.float16).view(c.blocks, c.kv_heads, c.block, 2)
        pairs[b, 0, r, 1] = float("nan")                     # the zero of one row of KV head 0
        got, err = run(c)
        assert err == 0
        for i in range(qlens[0]):
            seen = bool(c.visible(0, i)[270])
            assert bool(torch.isnan(got[i, :4]).all()) == seen and bool(torch.isnan(got[i, :4]).any()) == seen, i
            assert not torch.isnan(got[i, 4:]).any()


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("which", ["k", "v"])
def test_not_finite_in_a_segment_split_over_many_warps(value, which):
    """One pair of 9000 positions that is not finite: KV head 0's rows show it, through the join of their records; the others
    do not."""
    c = Case([9000], [1], kv="i4", seed=31)
    plain, _ = run(c)
    b, r = c.row_of(0, 4321)
    pool = getattr(c, which)
    pool[..., c.block * 64:].view(torch.float16).view(c.blocks, c.kv_heads, c.block, 2)[b, 0, r, 1] = value
    got, err = run(c)
    assert err == 0
    if which == "v" and value == float("inf"):
        assert torch.all(got[0, :4] == value)                # every column of that row is infinite
    elif which == "v":
        assert torch.isnan(got[0, :4]).all()
    else:                                                    # a score of either infinity, by the sign of sum(q), or NaN
        q = c.q[0, :4].to(F64).sum(-1)
        for h in range(4):
            if value == float("inf") and q[h] < 0:
                assert torch.isfinite(got[0, h]).all()       # that position has no weight
            else:
                assert torch.isnan(got[0, h]).all()
    assert torch.equal(got[0, 4:], plain[0, 4:])


def test_many_segments_joined_by_few_blocks():
    """More segments than CTAs, each cut in two or three: CTAs that join several of them."""
    g = torch.Generator().manual_seed(32)
    lens = torch.randint(900, 1300, (90,), generator=g).tolist()
    check(Case(lens, [1] * 90, kv="i4", heads=16, kv_heads=4, seed=32), spoil=False)
    check(Case(lens, [1] * 90, kv="i4", heads=16, kv_heads=4, seed=33, window=700, sinks=70), "bf16", spoil=False)


def test_bad_block_is_reported():
    c = Case([40], [1], kv="i4", seed=27)
    c.tables[0, 1] = c.blocks + 3
    _, err = run(c)
    assert err == pa.PA_DEVERR_BLOCK_ID


def test_same_answer_every_time_and_captured():
    for qlens in ([1, 1, 1], [4, 1, 2], [30, 64, 9]):
        c = Case([3000, 140, 9], qlens, kv="i4", seed=28)
        first, _ = run(c)
        q, k, v, t, n, st = (x.cuda() for x in (c.q, c.k, c.v, c.tables, c.lens_t, c.starts))
        ws = pa.new_workspace(pa.attend_workspace_bytes(3, 8, 2, 128, 16, c.tables.shape[1], 64, pa.PA_INT4), "cuda")
        out = torch.zeros((c.rows, 8, 128), device="cuda")
        graph = pa.StepGraph(lambda: pa.attend(out, q, k, v, t, n, st, max(qlens), 2, c.scale, 16, workspace=ws, pdl=True))
        for _ in range(3):
            out.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out.cpu().to(F64)[:sum(qlens)], first[:sum(qlens)])


def test_pools_beyond_32_bit_offsets():
    """Blocks on both sides of 4 GB."""
    block, heads, blocks = 64, 8, 140000                    # 4.9 GB a pool
    k, v = (torch.zeros(pa.int4_cache_shape(blocks, heads, block), dtype=torch.uint8, device="cuda") for _ in range(2))
    g = torch.Generator().manual_seed(29)
    tables = torch.tensor([[139999, 5, 130001, 124000]], dtype=torch.int32)
    T = 250
    pos = torch.arange(T)
    slots = tables[0].long()[pos // block] * block + pos % block
    x, y = (torch.randn((T, heads, 128), generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    pa.reshape_and_cache(x, y, k, v, slots.cuda(), block)
    kf, vf = (torch.zeros((T, heads, 128), device="cuda") for _ in range(2))
    pa.read_cache(kf, vf, k, v, slots.cuda(), block)
    for L in (1, 60):
        q = torch.randn((L, heads, 128), generator=g).to(torch.bfloat16)
        out = torch.zeros((L, heads, 128), device="cuda")
        ws = pa.new_workspace(pa.attend_workspace_bytes(1, heads, heads, 128, block, 4, L, pa.PA_INT4), "cuda")
        pa.attend(out, q.cuda(), k, v, tables.cuda(), torch.tensor([T], dtype=torch.int32).cuda(),
                  torch.tensor([0, L], dtype=torch.int32).cuda(), L, heads, 128 ** -0.5, block, workspace=ws)
        assert pa.get_device_error() == 0
        z = torch.einsum("lhd,thd->hlt", q.to(F64), kf.cpu().to(F64)) * 128 ** -0.5
        hidden = pos[None] > torch.arange(T - L, T)[:, None]
        ref = torch.einsum("hlt,thd->lhd", torch.softmax(z.masked_fill(hidden, -torch.inf), -1), vf.cpu().to(F64))
        # the bounds of attend_more.Case.tolerance, of values of at most 6
        assert torch.all((out.cpu().to(F64) - ref).abs() <= 6 * (2.6e-4 + 12 * 2.9e-4 + 2.0 ** -11 + 2.0 ** -11))


def test_copied_blocks():
    """pa_copy_blocks moves whole tiles: a copied block attends as its source."""
    c = Case([40, 40], [1, 1], kv="i4", seed=30)
    c.tables[1] = c.tables[0]
    k, v = c.k.cuda(), c.v.cuda()
    used = set(c.tables[0].tolist())
    spare = [b for b in range(c.blocks) if b not in used][0]
    pa.copy_blocks(k, v, torch.tensor([[int(c.tables[0, 1]), spare]], dtype=torch.int32, device="cuda"))
    c.tables[1, 1] = spare
    c.q_wide[1] = c.q_wide[0]
    c.k, c.v = k.cpu(), v.cpu()
    got, err = run(c)
    assert err == 0 and torch.equal(got[0], got[1])
