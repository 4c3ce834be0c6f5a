"""pa_attend over many sequences of a few position tiles each: every CTA of the tensor-core kernel computes several whole
segments one after the other, whose two parts are joined through records that take turns.  Against the definition in 64 bits
(tolerance: operator_cases.AttendCase.tolerance) and bit for bit over repeated calls."""

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import paged_kv_cache_144_gb300 as pa  # noqa: E402
from operator_cases import AttendCase, F64, run_attend  # noqa: E402


def reference(c):
    """(out, sum of p |v|) of a case in 64 bits, a sequence at a time on the GPU."""
    G = c.heads // c.kv_heads
    out = torch.zeros((c.rows, c.heads, c.dim), dtype=F64)
    wabs = torch.zeros_like(out)
    n = 0
    for s, (T, L) in enumerate(zip(c.lens, c.qlens)):
        t = torch.arange(T)
        blk, off = c.tables[s, t // c.block].long(), t % c.block
        K, V = c.k64[blk, :, off].cuda(), c.v64[blk, :, off].cuda()              # [T, H_kv, d]
        q = c.q[n:n + L].to(F64).cuda().view(L, c.kv_heads, G, c.dim)
        see = torch.stack([c.visible(s, i) for i in range(L)]).cuda()             # [L, T]
        z = torch.einsum("lhgd,thd->lhgt", q, K) * c.scale
        p = torch.softmax(z.masked_fill(~see[:, None, None], -float("inf")), -1)
        out[n:n + L] = torch.einsum("lhgt,thd->lhgd", p, V).reshape(L, c.heads, c.dim).cpu()
        wabs[n:n + L] = torch.einsum("lhgt,thd->lhgd", p, V.abs()).reshape(L, c.heads, c.dim).cpu()
        n += L
    return out, wabs


KINDS = [("bf16", "bf16", 128), ("f16", "f16", 128), ("bf16", "bf16", 64), ("f16", "f16", 64), ("e4m3", "bf16", 128),
         ("i8", "f16", 128)]
# sequences, queries of each, query heads per KV head, tree: 80 to 256 rows per KV head
FORMS = [(64, 20, 4, True), (64, 32, 4, False), (64, 25, 8, True), (64, 32, 8, False), (256, 24, 4, False)]


@pytest.mark.parametrize("kv,q,dim", KINDS)
@pytest.mark.parametrize("seqs,queries,group,tree", FORMS)
def test_whole_segments_of_two_to_four_tiles(kv, q, dim, seqs, queries, group, tree):
    g = torch.Generator().manual_seed(seqs + queries)
    lens = torch.randint(129, 401, (seqs,), generator=g).tolist()
    lens[::5] = [200] * len(lens[::5])                    # two tiles, the shortest that are joined
    lens[3::11] = [70] * len(lens[3::11])                 # one tile: no record between two that have one
    c = AttendCase(lens, [queries] * seqs, kv=kv, q=q, dim=dim, heads=8 * group, kv_heads=8, seed=queries)
    if tree:
        c.with_tree()
    got, err = run_attend(c)
    assert err == 0
    ref, wabs = reference(c)
    n = sum(c.qlens)
    assert torch.all(got[n:] == 7.0)
    off = (got[:n] - ref[:n]).abs() - c.tolerance("f32", ref, wabs)[:n]
    assert off.max() <= 0, f"{int((off > 0).sum())} outputs off, worst by {float(off.max()):.3e}"
    for _ in range(4):
        again, err = run_attend(c)
        assert err == 0 and torch.equal(got, again)
