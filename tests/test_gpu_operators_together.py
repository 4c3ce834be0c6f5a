"""The operators around the cache as a serving program calls them: captured and replayed, on several streams at once,
with shared and reused workspaces, at the largest batches and over pools whose offsets pass 32 bits."""

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import paged_kv_cache_144_gb300 as pa  # noqa: E402
from operator_cases import AttendCase, F64, check_attend, kept_positions, make_cache, run_attend, tables_for  # noqa: E402


class OnGpu:
    """A case's tensors on the GPU, its own workspace, and the call on them."""

    def __init__(self, c, mass=None):
        self.c, self.mass, self.max_q = c, mass, max(c.qlens)
        self.q, self.k, self.v = c.q.cuda(), c.k.cuda(), c.v.cuda()
        self.tables, self.lens, self.starts = c.tables.cuda(), c.lens_t.cuda(), c.starts.cuda()
        self.out = torch.zeros((c.rows, c.heads, c.dim), device="cuda")
        self.need = pa.attend_workspace_bytes(len(c.lens), c.heads, c.kv_heads, c.dim, c.block, c.tables.shape[1],
                                              self.max_q, pa.dtype_code(self.k), accumulate=mass is not None)
        self.ws = pa.new_workspace(self.need, "cuda")

    def __call__(self, stream=None, ws=None):
        c = self.c
        ws = self.ws if ws is None else ws
        if self.mass is not None:
            pa.attend_accumulate(self.out, self.q, self.k, self.v, self.tables, self.lens, self.mass, c.kv_heads,
                                 c.scale, c.block, workspace=ws, stream=stream)
        else:
            pa.attend(self.out, self.q, self.k, self.v, self.tables, self.lens, self.starts, self.max_q, c.kv_heads,
                      c.scale, c.block, workspace=ws, stream=stream)


@pytest.mark.parametrize("kv,dim", [("bf16", 128), ("f16", 64), ("e4m3", 128)])
@pytest.mark.parametrize("scale", [0.0, -0.09])
def test_scales_of_any_sign(kv, dim, scale):
    for qlens in ([1, 1, 1], [20, 90, 1]):
        c = AttendCase([20, 300, 1], qlens, kv=kv, dim=dim, heads=8, kv_heads=2, seed=1)
        c.scale = scale
        check_attend(c)


@pytest.mark.parametrize("cap", [2.0 ** -10, 512.0])
@pytest.mark.parametrize("qlens", [[1, 1, 1], [20, 90, 1]])
def test_softcap_at_its_limits(cap, qlens):
    """cap - 2 cap / (1 + 2^(2 x log2 e / cap)): the sum and the quotient are off by 2^-21.5 together, relative, so the
    score by up to cap * 2^-21.5 (1.7e-4 at 512), a weight by twice that."""
    c = AttendCase([20, 300, 1], qlens, seed=17)
    c.softcap = cap
    got, err = run_attend(c)
    ref, wabs, _ = c.reference()
    n = sum(qlens)
    assert err == 0
    assert torch.all((got - ref).abs()[:n] <= (c.tolerance("f32", ref, wabs) + 2 * cap * 2.0 ** -21.5 * wabs)[:n])


@pytest.mark.parametrize("kv,q,dim", [("bf16", "bf16", 128), ("f16", "f16", 64), ("e4m3", "bf16", 128), ("i8", "f16", 128)])
@pytest.mark.parametrize("rows", [17, 33, 64])
def test_few_rows_of_wide_tables(kv, q, dim, rows):
    """Tables of many positions, whose rows few or many of 64 the tensor cores take."""
    qlens = [rows // 4 + (rows % 4 > 0), 3, 1]
    c = AttendCase([900, 130, 61], qlens, kv=kv, q=q, dim=dim, heads=8, kv_heads=2, seed=18, width=100000)
    check_attend(c)
    check_attend(c.with_tree(), spoil=False)


@pytest.mark.parametrize("qlens", [[1, 1], [8, 40], [150, 3]])
def test_sequences_that_share_their_blocks(qlens):
    """Two tables that name the same blocks, as after a fork: each row as if it were alone."""
    c = AttendCase([400, 400], qlens, seed=2)
    c.tables[1] = c.tables[0]
    check_attend(c, spoil=False)


@pytest.mark.parametrize("L", [1, 3])
def test_most_sequences_and_more_counters_than_the_fixed_area(L):
    """4096 sequences of 0 to 8 tokens with 32 KV heads; before and after it, a small call on the same workspace."""
    S, H, B, D = 4096, 32, 8, 64
    g = torch.Generator(device="cuda").manual_seed(3)
    k, v = (torch.randn((S + 5, H, B, D), generator=g, device="cuda").half() for _ in range(2))
    tables = torch.randperm(S + 5, generator=g, device="cuda")[:S].to(torch.int32).view(S, 1)
    lens = torch.randint(0, 9, (S,), generator=g, device="cuda", dtype=torch.int32)
    qlens = lens.clamp(max=L)
    starts = torch.zeros(S + 1, dtype=torch.int32, device="cuda")
    starts[1:] = qlens.cumsum(0)
    n = int(starts[-1])
    q = torch.randn((n, H, D), generator=g, device="cuda").half()
    out = torch.full((n, H, D), 7.0, device="cuda")
    small = OnGpu(AttendCase([70, 900], [30, 100], seed=4))
    need = max(pa.attend_workspace_bytes(S, H, H, D, B, 1, L, pa.PA_F16), small.need)
    ws = pa.new_workspace(need, "cuda")
    small(ws=ws)
    want_small = small.out.clone()
    pa.attend(out, q, k, v, tables, lens, starts, L, H, 0.125, B, workspace=ws)
    small.out.zero_()
    small(ws=ws)
    assert pa.get_device_error() == 0
    assert torch.equal(small.out, want_small)
    # plain form: row r of sequence s at position P sees t <= P
    seq = torch.repeat_interleave(torch.arange(S, device="cuda"), qlens.long())
    pos = (lens - qlens).long()[seq] + torch.arange(n, device="cuda") - starts.long()[seq]
    K, V = (x[tables[:, 0].long()].double()[seq] for x in (k, v))        # [n, H, B, D]
    z = torch.einsum("nhd,nhtd->nht", q.double(), K) * 0.125
    z = z.masked_fill(torch.arange(B, device="cuda") > pos[:, None, None], -float("inf"))
    p = torch.softmax(z, 2)
    ref, wabs = torch.einsum("nht,nhtd->nhd", p, V), torch.einsum("nht,nhtd->nhd", p, V.abs())
    c = small.c
    assert torch.all((out.double() - ref).abs() <= c.tolerance("f32", ref, wabs))


def test_weights_in_rows_of_any_stride():
    """mass is a view: rows apart by odd numbers of elements, starting off every alignment."""
    c = AttendCase([50, 333, 0, 7], [1, 1, 1, 1], seed=5, pad_rows=0)
    width = c.tables.shape[1] * 16
    for off in (0, 1, 3):
        whole = torch.full((5, 3, width + 41), 2.0, device="cuda")
        mass = whole[:4, :2, off:off + width + 37]
        _, _, m = check_attend(c, mass=mass, spoil=False)
        add = (whole.cpu().double() - 2.0)
        got = add[:4, :2, off:off + width]
        # float32 next to 2: half a step is 2^-23; a weight is off by 2e of itself (see tolerance)
        assert torch.all((got - m).abs() <= 3e-4 * m + 2.0 ** -22)
        add[:4, :2, off:off + width] = 0
        assert torch.all(add == 0)
        for s, t in enumerate(c.lens):
            assert torch.all(got[s, :, t:] == 0)


def test_calls_on_two_streams_at_once():
    calls = [OnGpu(AttendCase([3000, 80], [1, 1], seed=6)), OnGpu(AttendCase([2000, 500], [300, 64], seed=7)),
             OnGpu(AttendCase([1500, 900], [40, 2], kv="e4m3", seed=8))]
    for x in calls[2:]:
        x.c.k_scale = x.c.k_scale.cuda()
        x.c.v_scale = x.c.v_scale.cuda()

    def run(x, stream=None):
        c = x.c
        pa.attend(x.out, x.q, x.k, x.v, x.tables, x.lens, x.starts, x.max_q, c.kv_heads, c.scale, c.block,
                  workspace=x.ws, stream=stream, k_scale=c.k_scale, v_scale=c.v_scale)

    want = []
    for x in calls:
        run(x)
        torch.cuda.synchronize()
        want.append(x.out.clone())
        x.out.zero_()
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for _ in range(20):
        for x, s in zip(calls, streams):
            run(x, s)
    torch.cuda.synchronize()
    assert pa.get_device_error() == 0
    for x, w in zip(calls, want):
        assert torch.equal(x.out, w)


def test_two_graphs_on_one_workspace():
    """Captured calls of different shapes take turns on a workspace of the larger's size."""
    a, b = OnGpu(AttendCase([700, 90], [200, 3], seed=9)), OnGpu(AttendCase([2500, 33, 5], [1, 1, 1], seed=10))
    ws = pa.new_workspace(max(a.need, b.need), "cuda")
    want = []
    for x in (a, b):
        x()
        torch.cuda.synchronize()
        want.append(x.out.clone())
    ga, gb = pa.StepGraph(lambda: a(ws=ws)), pa.StepGraph(lambda: b(ws=ws))
    for i in range(6):
        a.out.zero_()
        b.out.zero_()
        for graph in ((ga, gb), (gb, ga), (ga, ga, gb))[i % 3]:
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a.out, want[0]) and torch.equal(b.out, want[1])


def test_a_captured_step_follows_its_inputs():
    """Rotary write, weighted decode step and eviction in one graph: replayed after lengths, slots, positions, queries
    and tables have changed in place."""
    hq, hk, d, block, budget = 8, 2, 128, 16, 40
    g = torch.Generator().manual_seed(12)
    c = AttendCase([60, 17], [1, 1], heads=hq, kv_heads=hk, seed=12, pad_rows=0, width=6)
    x = OnGpu(c, mass=torch.zeros((2, hk, 96), device="cuda"))
    kc0, vc0 = x.k.clone(), x.v.clone()
    extra = 6
    x.k = torch.cat([x.k, torch.zeros((extra, hk, block, d), dtype=x.k.dtype, device="cuda")])
    x.v = torch.cat([x.v, torch.zeros_like(x.k[:extra])])
    dst = torch.arange(c.blocks, c.blocks + extra, dtype=torch.int32).view(2, 3).cuda()
    inv = pa.rope_frequencies(d).cuda()
    k_new, v_new = (torch.zeros((2, hk, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q_in = torch.zeros((2, hq, d), dtype=torch.bfloat16, device="cuda")
    pos, slots = (torch.zeros(2, dtype=torch.int64, device="cuda") for _ in range(2))
    kept = torch.zeros((2, hk, budget), dtype=torch.int32, device="cuda")
    mass_out = torch.zeros((2, hk, budget), device="cuda")
    new = torch.zeros(2, dtype=torch.int32, device="cuda")
    x.q = torch.zeros((2, hq, d), dtype=torch.bfloat16, device="cuda")

    def step():
        pa.rope_and_cache(q_in, k_new, v_new, x.k, x.v, pos, slots, inv, block, q_out=x.q)
        x()
        pa.evict(x.k, x.v, x.mass, x.tables, x.lens, dst, kept, mass_out, new, block, budget=budget, recent=4, sinks=1)

    def fill(lens):
        x.k[:c.blocks], x.v[:c.blocks] = kc0, vc0
        x.mass.copy_(torch.rand((2, hk, 96), generator=g))
        x.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        pos.copy_(torch.tensor(lens) - 1)
        slots.copy_(torch.tensor([int(c.tables[s, (t - 1) // block]) * block + (t - 1) % block
                                  for s, t in enumerate(lens)]))
        for t, h in ((q_in, hq), (k_new, hk), (v_new, hk)):
            t.copy_(torch.randn((2, h, d), generator=g))

    fill([60, 17])
    graph = pa.StepGraph(step)
    for lens in ([60, 17], [33, 16], [41, 1]):
        fill(lens)
        before = x.mass.clone()
        kept.fill_(-7)
        inputs = [t.clone() for t in (x.k, x.v, x.mass)]
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (x.out, x.mass, kept, mass_out, new, x.k, x.v)]
        for t, i in zip((x.k, x.v, x.mass), inputs):
            t.copy_(i)
        kept.fill_(-7)
        step()                                              # the same calls, launched one by one
        torch.cuda.synchronize()
        assert pa.get_device_error() == 0
        for a, b in zip(got, (x.out, x.mass, kept, mass_out, new, x.k, x.v)):
            assert torch.equal(a, b)
        assert new.tolist() == [min(t, budget) for t in lens]
        add = (x.mass - before).double().cpu()
        for s, t in enumerate(lens):                        # each query head's weights sum to 1
            assert torch.all((add[s, :, :t].sum(1) - hq / hk).abs() <= 3e-4 * hq / hk + t * 2.0 ** -22)
            assert torch.all(add[s, :, t:] == 0)
            for h in range(hk):
                want = kept_positions(x.mass[s, h].cpu(), t, budget, 4, 1)
                assert kept[s, h, :len(want)].tolist() == want


def test_a_path_may_name_a_node_twice():
    g = torch.Generator().manual_seed(13)
    tables, blocks = tables_for([40], 16, g)
    k = make_cache("bf16", blocks, 2, 16, 128, g)[0]
    kd, vd = k.cuda(), k.cuda()
    new = torch.empty(1, dtype=torch.int32, device="cuda")
    path = torch.tensor([[5, 2, 5, 5]], dtype=torch.int32).cuda()
    pa.commit_tree(kd, vd, tables.cuda(), torch.tensor([40], dtype=torch.int32).cuda(),
                   torch.tensor([0, 9], dtype=torch.int32).cuda(), path, torch.tensor([4], dtype=torch.int32).cuda(), new, 16)
    want = k.clone()
    for i, node in enumerate([5, 2, 5, 5]):
        a, b = 31 + i, 31 + node
        want[tables[0, a // 16], :, a % 16] = k[tables[0, b // 16], :, b % 16]
    assert new.tolist() == [35]
    assert torch.equal(kd.cpu(), want) and torch.equal(vd.cpu(), want)


def test_pools_beyond_32_bit_offsets():
    """Blocks at the far end of pools of more than 2^31 elements: bit for bit what the same blocks give in small pools."""
    hk, block, d = 8, 16, 128
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB of device memory")
    blocks = 2 ** 31 // (hk * block * d) + 300
    for qlens in ([1, 1], [100, 40]):
        c = AttendCase([700, 90], qlens, heads=16, kv_heads=hk, seed=14)
        off = blocks - c.blocks
        x = OnGpu(c)
        x()
        want = x.out.clone()
        small_k, small_v = x.k, x.v
        x.k, x.v = (torch.empty((blocks, hk, block, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        x.k[off:], x.v[off:] = small_k, small_v
        x.tables += off
        x.out.zero_()
        x()
        assert pa.get_device_error() == 0
        assert torch.equal(x.out, want)
    # rotary write, commit and eviction
    n = 5
    g = torch.Generator().manual_seed(15)
    q, k, v = (torch.randn((n, h, d), generator=g).bfloat16().cuda() for h in (16, hk, hk))
    pos = torch.arange(n).cuda()
    slots = torch.tensor([3, 20, 7, -1, 33]).cuda()
    inv = pa.rope_frequencies(d).cuda()
    lens, starts = torch.tensor([200], dtype=torch.int32).cuda(), torch.tensor([0, 20], dtype=torch.int32).cuda()
    path, plen = torch.tensor([[3, 9, 19]], dtype=torch.int32).cuda(), torch.tensor([3], dtype=torch.int32).cuda()
    mass = torch.rand((1, hk, c.tables.shape[1] * block), generator=g).cuda()
    results = []
    for kc, vc, o in ((small_k, small_v, 0), (x.k, x.v, off)):
        tables = c.tables[:1].cuda() + o
        free = sorted(set(range(c.blocks)) - set(c.tables[0].tolist()))[:4]
        dst = torch.tensor([free], dtype=torch.int32).cuda() + o
        new, kept = torch.empty(1, dtype=torch.int32, device="cuda"), torch.zeros((1, hk, 64), dtype=torch.int32, device="cuda")
        mo = torch.zeros((1, hk, 64), device="cuda")
        qo = torch.zeros_like(q)
        pa.rope_and_cache(q, k, v, kc, vc, pos, torch.where(slots < 0, slots, slots + o * block), inv, block, q_out=qo)
        pa.commit_tree(kc, vc, tables, lens, starts, path, plen, new, block)
        pa.evict(kc, vc, mass, tables, lens, dst, kept, mo, new, block, budget=64, recent=8, sinks=2)
        assert pa.get_device_error() == 0
        results.append((qo, kept, mo, new, kc[o:o + c.blocks].clone(), vc[o:o + c.blocks].clone()))
    for a, b in zip(*results):
        assert torch.equal(a, b)


def test_graph_of_no_sequences_and_empty_batches():
    """Batches of nothing: no launch, no error; and sequences of length zero among others."""
    c = AttendCase([0, 0, 5], [0, 0, 1], seed=16)
    check_attend(c)
    q = torch.empty((0, 8, 128), dtype=torch.bfloat16, device="cuda")
    k = torch.zeros((4, 2, 16, 128), dtype=torch.bfloat16, device="cuda")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    tables = torch.empty((0, 3), dtype=torch.int32, device="cuda")
    starts = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.attend(torch.empty((0, 8, 128), device="cuda"), q, k, k.clone(), tables, none, starts, 1, 2, 0.1, 16)
    pa.rope_and_cache(q, q[:, :2].contiguous(), q[:, :2].contiguous(), k, k.clone(), none.long(), none.long(),
                      pa.rope_frequencies(128).cuda(), 16)
    pa.commit_tree(k, k.clone(), tables, none, starts, torch.empty((0, 2), dtype=torch.int32, device="cuda"), none, none.clone(), 16)
    pa.evict(k, k.clone(), torch.empty((0, 2, 48), device="cuda"), tables, none, tables.clone(),
             torch.empty((0, 2, 4), dtype=torch.int32, device="cuda"), torch.empty((0, 2, 4), device="cuda"), none.clone(), 16, budget=4)
    assert pa.get_device_error() == 0


@pytest.mark.parametrize("kv,q,dim,heads,kv_heads", [("bf16", "bf16", 128, 8, 2), ("f16", "f16", 64, 6, 2),
                                                     ("e4m3", "bf16", 128, 40, 8), ("i8", "f16", 128, 64, 1)])
def test_a_workspace_serves_smaller_calls(kv, q, dim, heads, kv_heads):
    """Bytes for up to 50 sequences, 150 queries and 20 000 positions are enough for every smaller call."""
    code = {"bf16": pa.PA_BF16, "f16": pa.PA_F16, "e4m3": pa.PA_FP8_E4M3, "i8": pa.PA_INT8}[kv]
    for acc in (False, True):
        most = pa.attend_workspace_bytes(50, heads, kv_heads, dim, 16, 1250, 1 if acc else 150, code, accumulate=acc)
        for seqs in (1, 2, 7, 33, 50):
            for blocks in (1, 9, 64, 500, 1250):
                for L in ((1,) if acc else (1, 2, 3, 4, 5, 6, 7, 8, 12, 16, 17, 21, 32, 33, 64, 65, 100, 128, 129, 150)):
                    n = pa.attend_workspace_bytes(seqs, heads, kv_heads, dim, 16, blocks, L, code, accumulate=acc)
                    assert n <= most, (acc, seqs, blocks, L)
    ws = pa.new_workspace(pa.attend_workspace_bytes(50, heads, kv_heads, dim, 16, 1250, 150, code), "cuda")
    for seqs, L in ((1, 1), (3, 2), (2, 10), (2, 30), (1, 140)):
        c = AttendCase([200 + 31 * i for i in range(seqs)], [L] * seqs, kv=kv, q=q, dim=dim, heads=heads, kv_heads=kv_heads,
                       seed=19 + L)
        check_attend(c, workspace=ws)


@pytest.mark.parametrize("kv", ["bf16", "f16", "e4m3"])
@pytest.mark.parametrize("qlens", [[1, 1], [3, 1], [40, 130]])
def test_positions_before_a_window_may_hold_anything(kv, qlens):
    c = AttendCase([170, 300], qlens, kv=kv, seed=20)
    c.window = 37
    for s, (t, n) in enumerate(zip(c.lens, qlens)):
        for pos in range(0, t - n + 1 - 37):               # seen by no query
            b, o = c.row_of(s, pos)
            for x in (c.k, c.v):
                row = torch.full((c.kv_heads, c.dim), float("nan")).to(x.dtype)
                x.view(torch.uint8)[b, :, o] = row.view(torch.uint8).view(c.kv_heads, -1)
    c.spoil_tails()
    clean = AttendCase([170, 300], qlens, kv=kv, seed=20)  # the same numbers, unspoiled
    clean.window = 37
    ref, wabs, m = clean.reference()
    n = sum(qlens)
    got, err = run_attend(c)
    assert err == 0
    assert torch.all((got - ref).abs()[:n] <= c.tolerance("f32", ref, wabs)[:n])
    if max(qlens) == 1:
        mass = torch.zeros((2, c.kv_heads, c.tables.shape[1] * c.block), device="cuda")
        got, err = run_attend(c, mass=mass)
        assert err == 0
        assert torch.all((got - ref).abs()[:n] <= c.tolerance("f32", ref, wabs)[:n])
        assert torch.all((mass.cpu().double() - m).abs() <= 3e-4 * m + 2.0 ** -24)


def test_a_captured_call_with_more_counters_than_the_fixed_area():
    S, H, B, D = 2200, 32, 8, 64
    g = torch.Generator(device="cuda").manual_seed(21)
    k, v = (torch.randn((S, H, B, D), generator=g, device="cuda").half() for _ in range(2))
    tables = torch.randperm(S, generator=g, device="cuda").to(torch.int32).view(S, 1)
    lens = torch.randint(1, 9, (S,), generator=g, device="cuda", dtype=torch.int32)
    q = torch.randn((S, H, D), generator=g, device="cuda").half()
    want, out = torch.zeros((S, H, D), device="cuda"), torch.zeros((S, H, D), device="cuda")
    ws = pa.new_workspace(pa.attend_workspace_bytes(S, H, H, D, B, 1, 1, pa.PA_F16), "cuda")
    pa.attend(want, q, k, v, tables, lens, None, 1, H, 0.125, B, workspace=ws)
    graph = pa.StepGraph(lambda: pa.attend(out, q, k, v, tables, lens, None, 1, H, 0.125, B, workspace=ws, pdl=True))
    out.zero_()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert pa.get_device_error() == 0
    assert torch.equal(out, want)


def test_out_may_not_be_q():
    x = OnGpu(AttendCase([5, 9], [1, 1], pad_rows=0))
    with pytest.raises(ValueError, match="out must not be q"):
        pa.attend(x.q, x.q, x.k, x.v, x.tables, x.lens, x.starts, 1, 2, 0.1, 16, workspace=x.ws)


@pytest.mark.parametrize("kv", ["bf16", "f16", "e4m3"])
@pytest.mark.parametrize("most,group", [(100, 1), (100, 2), (300, 2)])
def test_most_sequences_on_the_tensor_cores(kv, most, group):
    """4096 sequences of 0 to 8 tokens, up to 8 of them queries, in a call that allows for many more queries."""
    S, H, B, D = 4096, 2, 8, 128
    g = torch.Generator(device="cuda").manual_seed(23)
    dt = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}[kv]
    qt = torch.float16 if kv == "f16" else torch.bfloat16
    k, v = (torch.randn((S + 5, H, B, D), generator=g, device="cuda").to(dt) for _ in range(2))
    tables = torch.randperm(S + 5, generator=g, device="cuda")[:S].to(torch.int32).view(S, 1)
    lens = torch.randint(0, 9, (S,), generator=g, device="cuda", dtype=torch.int32)
    qlens = torch.minimum(lens, torch.randint(0, 9, (S,), generator=g, device="cuda", dtype=torch.int32))
    starts = torch.zeros(S + 1, dtype=torch.int32, device="cuda")
    starts[1:] = qlens.cumsum(0)
    n = int(starts[-1])
    q = torch.randn((n, H * group, D), generator=g, device="cuda").to(qt)
    out = torch.full((n + 1, H * group, D), 7.0, device="cuda")
    scale = torch.tensor([0.8, 1.1], device="cuda") if kv == "e4m3" else None
    q_all = torch.cat([q, q[:1]])
    ws = pa.new_workspace(pa.attend_workspace_bytes(S, H * group, H, D, B, 1, most, pa.dtype_code(k)), "cuda")
    for _ in range(2):
        pa.attend(out, q_all, k, v, tables, lens, starts, most, H, 0.09, B, workspace=ws, k_scale=scale, v_scale=scale)
    assert pa.get_device_error() == 0
    assert torch.all(out[n] == 7.0)
    seq = torch.repeat_interleave(torch.arange(S, device="cuda"), qlens.long())
    pos = (lens - qlens).long()[seq] + torch.arange(n, device="cuda") - starts.long()[seq]
    K, V = (x[tables[:, 0].long()].double() * (1.0 if scale is None else scale.double()[None, :, None, None]) for x in (k, v))
    K, V = (x[seq].repeat_interleave(group, 1) for x in (K, V))
    z = torch.einsum("nhd,nhtd->nht", q.double(), K) * 0.09
    z = z.masked_fill(torch.arange(B, device="cuda") > pos[:, None, None], -float("inf"))
    p = torch.softmax(z, 2)
    ref, wabs = torch.einsum("nht,nhtd->nhd", p, V), torch.einsum("nht,nhtd->nhd", p, V.abs())
    c = AttendCase([1], [1], kv=kv)
    c.q = q
    assert torch.all((out[:n].double() - ref).abs() <= c.tolerance("f32", ref, wabs))
