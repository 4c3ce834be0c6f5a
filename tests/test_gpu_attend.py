"""pa_attend (score modifiers, ragged queries, drafted trees, accumulated weights) against a plain 64-bit
implementation, with bounds derived in operator_cases.AttendCase.tolerance."""

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import paged_kv_cache_144_gb300 as pa  # noqa: E402
from operator_cases import AttendCase, check_attend, run_attend  # noqa: E402

KINDS = [("bf16", "bf16", 128), ("f16", "f16", 128), ("f16", "f16", 64), ("bf16", "bf16", 64), ("e4m3", "bf16", 128),
         ("i8", "bf16", 128), ("e4m3", "f16", 128), ("i8", "f16", 128)]


@pytest.mark.parametrize("kv,q,dim", KINDS)
@pytest.mark.parametrize("out_fmt", ["f32", "q"])
def test_decode_step(kv, q, dim, out_fmt):
    c = AttendCase([1, 7, 16, 17, 127, 128, 129, 300, 0], [1] * 8 + [0], kv=kv, q=q, dim=dim, seed=1)
    check_attend(c, c.qt if out_fmt == "q" else "f32")


@pytest.mark.parametrize("kv,q,dim", KINDS)
def test_chunks(kv, q, dim):
    c = AttendCase([5, 40, 133, 260], [5, 33, 64, 1], kv=kv, q=q, dim=dim, seed=2)
    check_attend(c)


@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (3, 3), (8, 1), (6, 2), (7, 1), (40, 8), (32, 1), (64, 1)])
def test_head_groups(heads, kv_heads):
    c = AttendCase([1, 30, 140, 33], [1, 3, 9, 33], heads=heads, kv_heads=kv_heads, seed=3)
    check_attend(c)


@pytest.mark.parametrize("block", [8, 16, 32, 64, 128, 256, 1024])
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_block_sizes(block, kv):
    c = AttendCase([3, 130, 257, 1030], [3, 70, 1, 5], block=block, kv=kv, heads=4, kv_heads=2, seed=4)
    check_attend(c)


def test_long_chunk_many_row_tiles():
    c = AttendCase([700, 517], [400, 517], heads=4, kv_heads=1, seed=5)
    check_attend(c, "bf16")


def test_long_context_split_over_the_device():
    c = AttendCase([9001, 4100], [1, 20], heads=4, kv_heads=1, seed=6)
    check_attend(c)


def test_many_sequences():
    g = torch.Generator().manual_seed(7)
    lens = torch.randint(0, 90, (300,), generator=g).tolist()
    c = AttendCase(lens, [min(t, 1 + i % 3) for i, t in enumerate(lens)], heads=2, kv_heads=1, seed=7)
    check_attend(c)


@pytest.mark.parametrize("cap", [1.0, 30.0])
@pytest.mark.parametrize("kv", ["bf16", "i8"])
def test_softcap(cap, kv):
    c = AttendCase([5, 200, 131], [1, 40, 131], kv=kv, seed=8, q_mult=4.0)
    c.softcap = cap
    check_attend(c)


@pytest.mark.parametrize("kv", ["f16", "e4m3"])
@pytest.mark.parametrize("softcap", [0.0, 20.0])
def test_distance_bias(kv, softcap):
    c = AttendCase([5, 200, 300], [1, 40, 200], kv=kv, seed=9)
    c.slopes = torch.tensor([2.0 ** (-(h + 1)) for h in range(8)])
    c.softcap = softcap
    check_attend(c)


def test_distance_bias_of_either_sign_with_prefix():
    c = AttendCase([50, 150], [50, 40], seed=10)
    c.slopes = torch.tensor([0.5, -0.25, 0.0, 0.125, -0.01, 1.0, 0.3, 0.0])
    c.prefix = torch.tensor([50, 120], dtype=torch.int32)
    check_attend(c)


@pytest.mark.parametrize("window", [1, 2, 17, 128, 129, 4000])
@pytest.mark.parametrize("kv", ["bf16", "i8"])
def test_window(window, kv):
    c = AttendCase([1, 300, 450, 140], [1, 40, 1, 140], kv=kv, seed=11)
    c.window = window
    check_attend(c)


def test_prefix():
    c = AttendCase([10, 300, 270, 64], [10, 40, 270, 1], seed=12)
    c.prefix = torch.tensor([0, 290, 1000, 64], dtype=torch.int32)   # 1000: above the length, the whole sequence
    check_attend(c)


def test_more_queries_than_tokens_gives_zero_rows():
    c = AttendCase([3, 1, 40], [5, 9, 2], seed=13)
    got, ref, _ = check_attend(c)
    assert torch.all(got[:2] == 0) and torch.all(got[5:13] == 0)


@pytest.mark.parametrize("kv,q,dim", KINDS)
def test_tree(kv, q, dim):
    c = AttendCase([20, 200, 131, 64], [7, 16, 5, 64], kv=kv, q=q, dim=dim, seed=14).with_tree()
    check_attend(c)


@pytest.mark.parametrize("heads,kv_heads", [(2, 2), (8, 1), (14, 2)])
def test_tree_of_many_nodes(heads, kv_heads):
    c = AttendCase([500, 150, 140], [130, 150, 1], heads=heads, kv_heads=kv_heads, seed=15).with_tree(parents=40)
    check_attend(c, "bf16")


def test_tree_softcap_and_rows_that_see_nothing():
    """Masks without the node's own bit: a root with no context before it sees nothing."""
    c = AttendCase([6, 70], [6, 9], seed=16).with_tree(selfless=True)
    c.softcap = 25.0
    got, ref, _ = check_attend(c)
    assert torch.all(got[0] == 0)


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("kv", ["bf16", "f16", "e4m3"])
def test_masked_rows_may_hold_anything(value, kv):
    """One cached row (K and V) that some queries do not see holds NaN or infinity; they must not notice."""
    if kv == "e4m3" and value == float("inf"):
        pytest.skip("e4m3 has no infinity")
    c = AttendCase([60, 150], [20, 140], kv=kv, seed=17)
    c.spoil_tails()
    bad = 45                                              # position of the spoiled row in sequence 0
    b, o = c.row_of(0, bad)
    for x in (c.k, c.v):
        row = torch.full((c.kv_heads, c.dim), value).to(x.dtype)
        x.view(torch.uint8)[b, :, o] = row.view(torch.uint8).view(c.kv_heads, -1)
    b2, o2 = c.row_of(1, 149)
    c.v.view(torch.uint8)[b2, :, o2] = torch.full((c.kv_heads, c.dim), value).to(c.v.dtype).view(torch.uint8).view(c.kv_heads, -1)
    got, err = run_attend(c)
    ref, wabs, _ = c.reference()
    assert err == 0
    tol = c.tolerance("f32", ref, wabs)
    clean = [i for i in range(20) if 40 + i < bad] + list(range(20, 20 + 139))
    assert torch.all((got[clean] - ref[clean]).abs() <= tol[clean])
    blind = [i for i in range(20) if 40 + i >= bad] + [20 + 139]
    assert not torch.isfinite(got[blind]).all(-1).any()   # a query that sees NaN or infinity says so


def test_masked_tree_nodes_may_hold_anything():
    c = AttendCase([40, 170], [8, 30], seed=18).with_tree(parents=3)
    c.spoil_tails()
    leaf = 29
    seen_by = [i for i in range(30) if leaf in c.ancestors[1][i]]
    b, o = c.row_of(1, 140 + leaf)
    c.v[b, :, o] = float("nan")
    c.k[b, :, o] = float("inf")
    got, err = run_attend(c)
    ref, wabs, _ = c.reference()
    assert err == 0
    tol = c.tolerance("f32", ref, wabs)
    clean = [n for n in range(38) if n - 8 not in seen_by]
    assert torch.all((got[clean] - ref[clean]).abs() <= tol[clean])


@pytest.mark.parametrize("kv,q,dim", [("bf16", "bf16", 128), ("f16", "f16", 64), ("e4m3", "bf16", 128),
                                      ("i8", "f16", 128)])
@pytest.mark.parametrize("form", ["plain", "cap", "window", "bias", "prefix"])
def test_accumulate(kv, q, dim, form):
    lens = [1, 7, 129, 700, 0]
    c = AttendCase(lens, [1] * 5, kv=kv, q=q, dim=dim, heads=6, kv_heads=2, seed=19, pad_rows=0)
    if form == "cap":
        c.softcap = 15.0
    if form == "window":
        c.window = 50
    if form == "bias":
        c.slopes = torch.tensor([0.5, 0.25, 0.125, 0.06, 0.03, 0.01])
    if form == "prefix":
        c.prefix = torch.tensor([1, 3, 129, 9, 0], dtype=torch.int32)
    width = c.tables.shape[1] * c.block
    start = torch.rand((5, 3, width + 5), generator=c.g)[:, :2]          # a strided view
    mass = torch.rand((5, 3, width + 5), generator=c.g).cuda()[:, :2]
    mass.copy_(start)
    got, ref, want = check_attend(c, mass=mass)
    m = mass.cpu().double() - start.double()
    # a weight: the score's error as for the outputs (relative), then float32 sums of up to G = 3 of them and the
    # running total (values up to 1 + 3: half a step of 2^-22)
    tol = 3e-4 * want + 2.0 ** -22
    assert torch.all((m[:, :, :width] - want).abs() <= tol)
    for s, t in enumerate(lens):                                          # beyond the sequence: untouched
        assert torch.equal(mass[s, :, t:].cpu(), start[s, :, t:])


def test_strided_queries_and_reused_workspace():
    """q rows of a wider buffer; one workspace for calls one after the other."""
    a = AttendCase([9, 140, 2000], [1, 30, 3], seed=20, q_pad=3)
    need = pa.attend_workspace_bytes(3, 8, 2, 128, 16, a.tables.shape[1], 30, pa.PA_BF16)
    ws = pa.new_workspace(need, "cuda")
    first, _ = run_attend(a, workspace=ws)
    again, _ = run_attend(a, workspace=ws)
    assert torch.equal(first, again)
    check_attend(a, workspace=ws)


def test_without_query_starts():
    c = AttendCase([9, 140, 33], [1, 1, 1], seed=21, pad_rows=0)
    with_starts, _ = run_attend(c)
    without, _ = run_attend(c, use_starts=False)
    assert torch.equal(with_starts, without)
    check_attend(c, use_starts=False)


def test_large_logits():
    c = AttendCase([300, 90], [17, 1], seed=22, q_mult=30.0)
    check_attend(c)


def test_deterministic():
    c = AttendCase([3000, 700, 1500], [9, 64, 1], seed=23)
    runs = [run_attend(c)[0] for _ in range(3)]
    assert torch.equal(runs[0], runs[1]) and torch.equal(runs[0], runs[2])


def test_another_stream_and_a_captured_graph():
    c = AttendCase([300, 90, 1200], [17, 1, 2], seed=24)
    want, _ = run_attend(c)
    side = torch.cuda.Stream()
    q, k, v = c.q.cuda(), c.k.cuda(), c.v.cuda()
    out = torch.zeros((c.rows, 8, 128), device="cuda")
    ws = pa.new_workspace(pa.attend_workspace_bytes(3, 8, 2, 128, 16, c.tables.shape[1], 17, pa.PA_BF16), "cuda")
    t, l, st = c.tables.cuda(), c.lens_t.cuda(), c.starts.cuda()

    def step():
        pa.attend(out, q, k, v, t, l, st, 17, 2, c.scale, 16, workspace=ws)

    step_graph = pa.StepGraph(step)
    out.zero_()
    for _ in range(3):
        step_graph.replay()
    torch.cuda.synchronize()
    n = sum(c.qlens)
    assert torch.equal(out[:n].cpu().double(), want[:n])
    out.zero_()
    torch.cuda.synchronize()
    pa.attend(out, q, k, v, t, l, st, 17, 2, c.scale, 16, workspace=ws, stream=side)
    side.synchronize()
    assert torch.equal(out[:n].cpu().double(), want[:n])


def test_bad_inputs_are_reported_and_skipped():
    c = AttendCase([40, 90, 30], [2, 3, 1], seed=25)
    ref, wabs, _ = c.reference()
    c.starts = torch.tensor([0, 2, 5, 500], dtype=torch.int32)            # beyond the rows of q
    got, err = run_attend(c)
    assert err == pa.PA_DEVERR_QUERY
    assert torch.all((got[:5] - ref[:5]).abs() <= c.tolerance("f32", ref, wabs)[:5])
    assert torch.all(got[5:] == 7.0)
    c.starts = torch.tensor([0, 2, 5, 6], dtype=torch.int32)
    c.lens_t = torch.tensor([40, -3, 30], dtype=torch.int32)
    got, err = run_attend(c)
    assert err == pa.PA_DEVERR_SEQ_LEN
    assert torch.all(got[2:5] == 0)
    c.lens_t = torch.tensor([40, 90, 30], dtype=torch.int32)
    c.tables[1, 1] = c.blocks + 5
    got, err = run_attend(c)
    assert err == pa.PA_DEVERR_BLOCK_ID
    assert torch.all((got[:2] - ref[:2]).abs() <= c.tolerance("f32", ref, wabs)[:2])


@pytest.mark.parametrize("kv,q", [("e4m3", "bf16"), ("e4m3", "f16"), ("i8", "bf16"), ("i8", "f16")])
@pytest.mark.parametrize("qlens,lens", [([30, 17], [30, 200]), ([120, 1], [700, 900]), ([300, 257], [300, 1100])])
def test_chunks_over_8_bit_caches(kv, q, qlens, lens):
    """Rows below, at and above those of one pair of CTAs; queries of very different magnitude in one tile."""
    c = AttendCase(lens, qlens, kv=kv, q=q, heads=8, kv_heads=2, seed=30)
    c.q_wide[: qlens[0] // 2] *= 2.0 ** -9
    c.q_wide[3:4] = 0
    check_attend(c, "f32")
    check_attend(c, c.qt)


@pytest.mark.parametrize("heads,kv_heads", [(3, 1), (10, 2), (48, 1)])
@pytest.mark.parametrize("kv", ["bf16", "f16", "e4m3"])
def test_chunk_head_groups(heads, kv_heads, kv):
    """Groups whose queries do not fill 128 rows: tiles of whole queries."""
    c = AttendCase([400, 190], [129, 60], heads=heads, kv_heads=kv_heads, kv=kv, seed=31)
    check_attend(c)


def test_few_long_segments_are_cut_and_joined():
    """One KV head over a long context: a segment in many pieces, joined in order."""
    c = AttendCase([20000], [40], heads=4, kv_heads=1, seed=32)
    first, _, _ = check_attend(c)
    again, _ = run_attend(c)
    assert torch.equal(first, again)
    check_attend(AttendCase([20000], [90], heads=4, kv_heads=1, dim=64, kv="f16", seed=33))
