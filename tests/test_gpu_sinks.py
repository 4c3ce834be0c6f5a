"""pa_attend with a window whose first tokens stay visible, every cache type, against a plain 64-bit implementation.  Whatever
no query sees is NaN, and the table entries of blocks without a seen row are -1 (attend_more.Case.spoil)."""

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import paged_kv_cache_144_gb300 as pa  # noqa: E402
from attend_more import Case, check, run  # noqa: E402
from operator_cases import F64, HALF_STEP  # noqa: E402

KINDS = [("bf16", "bf16", 128), ("f16", "f16", 64), ("e4m3", "f16", 128), ("i8", "bf16", 128)]


@pytest.mark.parametrize("kv,q,dim", KINDS)
@pytest.mark.parametrize("window,sinks", [(1, 1), (16, 4), (33, 33), (100, 129), (500, 7), (64, 5000)])
def test_decode_step(kv, q, dim, window, sinks):
    c = Case([1, 7, 16, 40, 129, 300, 777, 0], [1] * 7 + [0], kv=kv, q=q, dim=dim, seed=1, window=window, sinks=sinks)
    check(c)


@pytest.mark.parametrize("kv,q,dim", KINDS)
@pytest.mark.parametrize("window,sinks", [(1, 4), (40, 3), (130, 20), (64, 200), (300, 1)])
def test_few_queries(kv, q, dim, window, sinks):
    c = Case([3, 50, 400, 260], [3, 4, 2, 16], kv=kv, q=q, dim=dim, seed=2, window=window, sinks=sinks)
    check(c, c.qt)


@pytest.mark.parametrize("kv,q,dim", KINDS)
@pytest.mark.parametrize("window,sinks", [(1, 1), (64, 4), (128, 128), (130, 150), (1000, 9)])
def test_chunks(kv, q, dim, window, sinks):
    c = Case([5, 140, 700, 520], [5, 133, 64, 300], kv=kv, q=q, dim=dim, seed=3, window=window, sinks=sinks)
    check(c)


@pytest.mark.parametrize("block", [8, 32, 64, 256, 1024])
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_block_sizes(block, kv):
    """Sinks that end inside a block, a gap that starts inside one and ends inside another, or none."""
    for window, sinks in ((70, 5), (900, 40), (200, 300)):
        c = Case([3, 257, 1400, 2100], [3, 70, 1, 5], block=block, kv=kv, heads=4, kv_heads=2, seed=4, window=window, sinks=sinks)
        check(c)


@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (8, 1), (7, 1), (40, 8), (32, 1)])
def test_head_groups(heads, kv_heads):
    c = Case([1, 90, 440, 133], [1, 3, 9, 33], heads=heads, kv_heads=kv_heads, seed=5, window=60, sinks=6)
    check(c)


def test_long_context_split_over_the_device():
    check(Case([20001, 16500], [1, 1], heads=4, kv_heads=1, seed=6, window=9000, sinks=300))
    check(Case([12001, 9500], [1, 20], heads=4, kv_heads=1, seed=7, window=5000, sinks=300))
    check(Case([3000], [1200], heads=4, kv_heads=1, seed=8, window=700, sinks=260), "bf16")


def test_many_short_sequences():
    g = torch.Generator().manual_seed(9)
    lens = torch.randint(0, 90, (300,), generator=g).tolist()
    check(Case(lens, [min(t, 1 + i % 3) for i, t in enumerate(lens)], heads=2, kv_heads=1, seed=9, window=20, sinks=4))
    check(Case(lens, [min(t, 40) for t in lens], heads=4, kv_heads=1, seed=10, window=20, sinks=4))


@pytest.mark.parametrize("kv", ["f16", "i8"])
def test_with_cap_and_distance_bias(kv):
    for lens, q in (([5, 200, 300], [1, 1, 1]), ([5, 200, 300], [1, 40, 200])):
        c = Case(lens, q, kv=kv, q="f16", seed=11, window=50, sinks=10)
        c.slopes = torch.tensor([2.0 ** (-(h + 1)) for h in range(8)])
        c.softcap = 20.0
        check(c)


def test_more_queries_than_tokens():
    c = Case([3, 1, 40], [5, 9, 2], seed=12, window=2, sinks=1)
    got, _, _ = check(c)
    assert torch.all(got[:2] == 0) and torch.all(got[5:13] == 0)


@pytest.mark.parametrize("qlens", [[1, 1], [40, 64]])
def test_sinks_without_a_window_change_nothing(qlens):
    c = Case([300, 140], qlens, seed=13, sinks=9)
    a, _ = run(c)
    c.sinks = 0
    b, _ = run(c)
    assert torch.equal(a, b)


@pytest.mark.parametrize("qlens", [[1, 1], [40, 64]])
def test_sinks_that_close_the_gap_see_everything(qlens):
    """A window and sinks that together cover every position: the rows of the call without a window."""
    c = Case([300, 140], qlens, seed=14, window=200, sinks=150)
    a, err = run(c)
    c.window = c.sinks = 0
    b, err2 = run(c)
    ref, wabs, _ = c.reference()
    n = sum(qlens)
    assert err == 0 and err2 == 0
    assert torch.all((a[:n] - b[:n]).abs() <= 2 * c.tolerance("f32", ref, wabs)[:n])


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_weights_added_up(kv):
    """Sinks and window receive their weights, the gap keeps what it held."""
    c = Case([1, 40, 300, 700], [1] * 4, kv=kv, seed=15, window=65, sinks=6)
    mass = torch.full((4, 2, c.tables.shape[1] * c.block), 0.5, device="cuda")
    _, _, ref = check(c, mass=mass)
    got = mass.cpu().to(F64) - 0.5
    assert torch.all((got - ref).abs() <= 3e-4 * ref * 3 + 2.0 ** -23)
    seen = ref > 0
    assert torch.all(got[~seen] == 0)


@pytest.mark.parametrize("where", [2, 100, 290])
def test_nan_shows_where_it_is_seen(where):
    """A NaN V row: in the sinks and the window it shows in the rows that see it, in the gap in none."""
    for qlens in ([1], [3], [70]):
        c = Case([300], qlens, seed=16, window=100, sinks=4)
        b, r = c.row_of(0, where)
        c.v[b, :, r] = float("nan")
        got, err = run(c)
        assert err == 0
        for i in range(qlens[0]):
            assert bool(torch.isnan(got[i]).all()) == bool(c.visible(0, i)[where]), i
            assert bool(torch.isnan(got[i]).any()) == bool(c.visible(0, i)[where]), i


def test_captured_and_replayed_on_shared_workspaces():
    cases = [Case([300, 140, 9], [1, 1, 1], seed=17, window=40, sinks=5), Case([300, 140, 9], [30, 64, 9], seed=18, window=40, sinks=5)]
    outs, want, args = [], [], []
    ws = pa.new_workspace(pa.attend_workspace_bytes(3, 8, 2, 128, 16, cases[0].tables.shape[1], 64), "cuda")
    for c in cases:
        outs.append(torch.zeros((c.rows, 8, 128), device="cuda"))
        args.append((c.q.cuda(), c.k.cuda(), c.v.cuda(), c.tables.cuda(), c.lens_t.cuda(), c.starts.cuda(), max(c.qlens)))
        want.append(c.reference())

    def step():
        for c, o, (q, k, v, t, n, st, mq) in zip(cases, outs, args):
            pa.attend(o, q, k, v, t, n, st, mq, 2, c.scale, 16, workspace=ws, window=c.window, sinks=c.sinks, pdl=True)

    graph = pa.StepGraph(step)
    for o in outs:
        o.zero_()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    for c, o, (ref, wabs, _) in zip(cases, outs, want):
        n = sum(c.qlens)
        assert torch.all((o.cpu().to(F64)[:n] - ref[:n]).abs() <= c.tolerance("f32", ref, wabs)[:n])
