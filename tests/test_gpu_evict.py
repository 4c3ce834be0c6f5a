"""pa_commit_tree and pa_evict: rows are moved, so caches, weights and positions are compared bit for bit; and the
operators of a serving loop run one after the other."""

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import paged_kv_cache_144_gb300 as pa  # noqa: E402
from operator_cases import AttendCase, F64, check_attend, kept_positions, make_cache, run_attend, tables_for  # noqa: E402


def _bytes(c):
    return c.view(torch.uint8)


# ------------------------------------------------------------------------------------------------ commit

@pytest.mark.parametrize("kv,dim", [("bf16", 128), ("f16", 64), ("e4m3", 128), ("i8", 128)])
@pytest.mark.parametrize("block", [8, 16, 128])
def test_commit_moves_the_path(kv, dim, block):
    g = torch.Generator().manual_seed(1)
    lens, qlens = [30, 64, 5, 300, 17], [7, 64, 5, 256, 1]
    paths = [[0, 2, 6], list(range(0, 64, 3)), [], sorted(torch.randperm(256, generator=g)[:256].tolist()), [0]]
    paths[3] = torch.randperm(256, generator=g).tolist()          # any order, the whole tree
    tables, blocks = tables_for(lens, block, g)
    k = make_cache(kv, blocks, 3, block, dim, g)[0]
    v = make_cache(kv, blocks, 3, block, dim, g)[0]
    width = max(len(p) for p in paths)
    path = torch.tensor([p + [9999] * (width - len(p)) for p in paths], dtype=torch.int32)
    n = torch.tensor([len(p) for p in paths], dtype=torch.int32)
    starts = torch.tensor([0] + list(torch.tensor(qlens).cumsum(0)), dtype=torch.int32)
    kd, vd = k.cuda(), v.cuda()
    new = torch.empty(5, dtype=torch.int32, device="cuda")
    pa.commit_tree(kd, vd, tables.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), starts.cuda(), path.cuda(),
                   n.cuda(), new, block)
    assert pa.get_device_error() == 0
    assert new.tolist() == [t - q + len(p) for t, q, p in zip(lens, qlens, paths)]
    for got, had in ((kd, k), (vd, v)):
        want = _bytes(had).clone()
        for s, p in enumerate(paths):
            first = lens[s] - qlens[s]
            for i, node in enumerate(p):
                a, b = first + node, first + i
                want[tables[s, b // block], :, b % block] = _bytes(had)[tables[s, a // block], :, a % block]
        assert torch.equal(_bytes(got).cpu(), want)


def test_commit_reports_bad_paths():
    g = torch.Generator().manual_seed(2)
    lens, qlens = [30, 30, 30, 3], [6, 6, 6, 4]
    tables, blocks = tables_for(lens, 16, g)
    k = make_cache("bf16", blocks, 2, 16, 128, g)[0]
    kd, vd = k.cuda(), k.cuda()
    starts = torch.tensor([0, 6, 12, 18, 22], dtype=torch.int32).cuda()
    path = torch.tensor([[1, 6, 0], [0, -1, 0], [3, 4, 5], [0, 1, 2]], dtype=torch.int32).cuda()
    n = torch.tensor([2, 2, 4, 2], dtype=torch.int32).cuda()      # node 6 of 6; node -1; longer than its row; T < L
    new = torch.empty(4, dtype=torch.int32, device="cuda")
    pa.commit_tree(kd, vd, tables.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), starts, path, n, new, 16)
    assert pa.get_device_error() == pa.PA_DEVERR_PATH
    assert new.tolist() == lens
    assert torch.equal(kd.cpu(), k) and torch.equal(vd.cpu(), k)


# ------------------------------------------------------------------------------------------------ evict

def _evict(lens, budget, recent, sinks, *, kv="bf16", dim=128, heads=2, block=16, seed=0, mass=None, pad=0):
    g = torch.Generator().manual_seed(seed)
    keep = [min(t, budget) for t in lens]
    both, blocks = tables_for(list(lens) + keep, block, g, width=-(-max(max(lens), 1) // block) + pad)
    S = len(lens)
    tables, dst = both[:S].contiguous(), both[S:, :max(1, -(-budget // block))].contiguous()
    if dst.shape[1] * block < min(budget, tables.shape[1] * block):
        dst = torch.cat([dst, torch.full((S, -(-budget // block) - dst.shape[1]), -1, dtype=torch.int32)], 1).contiguous()
    k, v = (make_cache(kv, blocks, heads, block, dim, g)[0] for _ in range(2))
    width = tables.shape[1] * block
    if mass is None:
        mass = torch.rand((S, heads, width), generator=g)
    else:
        mass = mass(S, heads, width, g)
    kd, vd = k.cuda(), v.cuda()
    kept = torch.full((S, heads, budget), -7, dtype=torch.int32, device="cuda")
    mo = torch.full((S, heads, budget), -7.0, device="cuda")
    new = torch.empty(S, dtype=torch.int32, device="cuda")
    pa.evict(kd, vd, mass.cuda(), tables.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), dst.cuda(), kept, mo, new,
             block, budget=budget, recent=recent, sinks=sinks)
    assert pa.get_device_error() == 0
    assert new.tolist() == keep
    kept, mo = kept.cpu(), mo.cpu()
    wk, wv = _bytes(k).clone(), _bytes(v).clone()
    for s, T in enumerate(lens):
        for h in range(heads):
            want = kept_positions(mass[s, h], T, budget, recent, sinks)
            assert kept[s, h].tolist() == want + [-7] * (budget - len(want)), (s, h)
            a, b = mo[s, h, :len(want)], mass[s, h, want]
            assert torch.equal(a.isnan(), b.isnan()) and torch.equal(a[~a.isnan()], b[~b.isnan()])
            assert torch.all(mo[s, h, len(want):] == -7)
            for i, t in enumerate(want):
                for w, src in ((wk, k), (wv, v)):
                    w[dst[s, i // block], h, i % block] = _bytes(src)[tables[s, t // block], h, t % block]
    assert torch.equal(_bytes(kd).cpu(), wk) and torch.equal(_bytes(vd).cpu(), wv)


@pytest.mark.parametrize("kv,dim", [("bf16", 128), ("f16", 64), ("e4m3", 128), ("i8", 128)])
@pytest.mark.parametrize("budget,recent,sinks", [(16, 4, 2), (33, 0, 0), (40, 40, 0), (40, 36, 4), (1, 0, 0), (1, 1, 0),
                                                 (500, 10, 4)])
def test_evict(kv, dim, budget, recent, sinks):
    _evict([0, 1, 16, 33, 34, 41, 120, 501], budget, recent, sinks, kv=kv, dim=dim, seed=3)


@pytest.mark.parametrize("block", [8, 32, 256, 1024])
def test_evict_block_sizes(block):
    _evict([700, 90, 1025], 130, 20, 4, block=block, seed=4)


def test_evict_ties_go_to_the_lower_position():
    _evict([300, 80], 50, 5, 2, seed=5, mass=lambda S, H, W, g: torch.zeros((S, H, W)))
    _evict([2500, 80], 1300, 5, 2, seed=5, mass=lambda S, H, W, g: torch.randint(0, 3, (S, H, W), generator=g).float())


def test_evict_odd_weights():
    """NaN counts below everything, minus zero equals zero, infinities and negative weights have their order."""
    def mass(S, H, W, g):
        m = torch.randn((S, H, W), generator=g)
        odd = torch.tensor([float("nan"), float("inf"), float("-inf"), 0.0, -0.0, 1e-42])
        at = torch.randint(0, 12, (S, H, W), generator=g)
        return torch.where(at < 6, odd[at.clamp(max=5)], m)
    for budget in (20, 150, 290):
        _evict([300, 299, 310], budget, 3, 1, seed=6, mass=mass)


def test_evict_long():
    _evict([5000, 3001], 1024, 64, 4, heads=1, seed=7)
    _evict([40000], 600, 64, 4, heads=1, dim=64, kv="f16", seed=8,
           mass=lambda S, H, W, g: torch.rand((S, H, W), generator=g) ** 8)


def test_evict_beyond_the_table():
    """A length outside the table's capacity is reported and clamped; a bad block id is reported, its row skipped."""
    g = torch.Generator().manual_seed(9)
    k = make_cache("bf16", 12, 1, 16, 128, g)[0]
    tables = torch.tensor([[0, 1, 2, 3], [4, 99, 6, 7]], dtype=torch.int32).cuda()
    dst = torch.tensor([[8], [9]], dtype=torch.int32).cuda()
    mass = torch.rand((2, 1, 64), generator=g).cuda()
    kept = torch.full((2, 1, 16), -7, dtype=torch.int32, device="cuda")
    mo = torch.zeros((2, 1, 16), device="cuda")
    new = torch.empty(2, dtype=torch.int32, device="cuda")
    pa.evict(k.cuda(), k.cuda(), mass, tables, torch.tensor([70, 64], dtype=torch.int32).cuda(), dst, kept, mo, new, 16,
             budget=16)
    assert pa.get_device_error() == pa.PA_DEVERR_SEQ_LEN | pa.PA_DEVERR_BLOCK_ID
    assert new.tolist() == [16, 16]


# ------------------------------------------------------------------------------------------------ together

def test_a_serving_run_of_the_operators():
    """Prompt chunk (rotary write, attend), draft (rotary write, attend_tree, commit_tree), decode steps that add up
    weights, an eviction, and a decode over the evicted cache; every attention against the plain form on the cache as
    it is then."""
    hq, hk, d, block = 8, 2, 128, 16
    g = torch.Generator().manual_seed(11)
    inv = pa.rope_frequencies(d).cuda()
    nblk = 40
    kc = torch.zeros((nblk, hk, block, d), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    bm = pa.BlockManager(nblk, block)
    for s in range(2):
        bm.add_sequence(s)

    def write(new):                                     # new tokens of each sequence: rotary write of their rows
        slots, pos = [], []
        for s, n in enumerate(new):
            for _ in range(n):
                pos.append(bm.lengths[s])
                slots.append(bm.append_slot(s)[0])
        n = len(slots)
        q, k, v = (torch.randn((n, h, d), generator=g).bfloat16().cuda() for h in (hq, hk, hk))
        pa.rope_and_cache(q, k, v, kc, vc, torch.tensor(pos).cuda(), torch.tensor(slots).cuda(), inv, block)
        return q

    def case(q, new, tables=None, lens=None):
        c = AttendCase([1], [1])
        c.lens, c.qlens = lens or [bm.lengths[s] for s in range(2)], list(new)
        width = -(-max(c.lens) // block)
        c.tables = torch.tensor([bm.block_table(s, width)[:width] for s in range(2)], dtype=torch.int32) if tables is None else tables
        c.lens_t = torch.tensor(c.lens, dtype=torch.int32)
        c.k, c.v, c.blocks = kc.cpu(), vc.cpu(), nblk
        c.k64, c.v64 = c.k.to(F64), c.v.to(F64)
        c.q_wide = c.q = q.cpu()
        c.rows = q.shape[0]
        c.starts = torch.tensor([0, new[0], sum(new)], dtype=torch.int32)
        return c

    q = write([100, 37])                                # prompts
    check_attend(case(q, [100, 37]), spoil=False)
    q = write([6, 9])                                   # drafts
    c = case(q, [6, 9]).with_tree(parents=3)
    check_attend(c, spoil=False)
    deepest = [max(a, key=len) for a in c.ancestors]
    width = max(len(p) for p in deepest)
    new = torch.empty(2, dtype=torch.int32, device="cuda")
    pa.commit_tree(kc, vc, c.tables.cuda(), c.lens_t.cuda(), c.starts.cuda(),
                   torch.tensor([p + [0] * (width - len(p)) for p in deepest], dtype=torch.int32).cuda(),
                   torch.tensor([len(p) for p in deepest], dtype=torch.int32).cuda(), new, block)
    for s in range(2):
        assert int(new[s]) == c.lens[s] - c.qlens[s] + len(deepest[s])
        bm.lengths[s] = int(new[s])
    mass = torch.zeros((2, hk, 160), device="cuda")
    total = torch.zeros((2, hk, 160), dtype=F64)
    for _ in range(3):                                  # decode steps
        q = write([1, 1])
        c = case(q, [1, 1])
        width = c.tables.shape[1] * block
        _, _, m = check_attend(c, mass=mass, spoil=False)
        total[:, :, :width] += m
    assert torch.all((mass.cpu().to(F64) - total).abs() <= 3e-4 * total + 2.0 ** -20)
    budget = 48
    dst = [[bm.allocate() for _ in range(3)] for _ in range(2)]
    kept = torch.empty((2, hk, budget), dtype=torch.int32, device="cuda")
    mo = torch.empty((2, hk, budget), device="cuda")
    pa.evict(kc, vc, mass, c.tables.cuda(), c.lens_t.cuda(), torch.tensor(dst, dtype=torch.int32).cuda(), kept, mo, new,
             block, budget=budget, recent=8, sinks=2)
    for s in range(2):
        for h in range(hk):
            want = kept_positions(mass[s, h].cpu(), c.lens[s], budget, 8, 2)
            assert kept[s, h, :len(want)].tolist() == want
    lens = new.tolist()
    q = torch.randn((2, hq, d), generator=g).bfloat16().cuda()
    e = case(q, [1, 1], tables=torch.tensor(dst, dtype=torch.int32), lens=lens)
    check_attend(e, spoil=False)
    assert pa.get_device_error() == 0
    run_attend(e)


@pytest.mark.parametrize("lens", [[40000, 20001], [300, 100000], [131072 + 5]])
@pytest.mark.parametrize("weights", ["spread", "few values", "equal"])
def test_evict_of_many_positions_in_clusters(lens, weights):
    """Positions shared by several CTAs; ties across their borders."""
    def mass(S, H, W, g):
        if weights == "equal":
            return torch.ones((S, H, W))
        m = torch.rand((S, H, W), generator=g) ** 6
        return m if weights == "spread" else (m * 40).floor()
    _evict(lens, 700, 64, 4, heads=2, dim=64, kv="f16", block=64, seed=21, mass=mass)
    _evict(lens, 301, 0, 0, heads=2, dim=64, kv="f16", block=64, seed=22, mass=mass)


def test_evict_of_many_positions_and_pairs():
    """More pairs than SMs, and tables longer than what one CTA's shared memory holds."""
    _evict([60000, 5, 777, 90], 40, 3, 2, heads=44, dim=64, kv="f16", block=1024, seed=23)
