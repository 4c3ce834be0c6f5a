"""pa_attend with NaN in a query, or in a K row that queries see: those rows are NaN, never zero or finite, on every kernel that
serves the call.  Other sequences' rows keep their bits; the other rows of the same sequence are as exact as ever (rows that
share a warp share the moment at which their running maxima move, so their roundings may change)."""

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from operator_cases import AttendCase, run_attend  # noqa: E402
from test_gpu_attend_whole import reference  # noqa: E402

KINDS = [("bf16", "bf16", 128), ("f16", "f16", 64), ("e4m3", "bf16", 128)]
# queries of each sequence: single queries, few rows, one row tile, several row tiles
QUERIES = [1, 4, 24, 80]


@pytest.mark.parametrize("kv,q,dim", KINDS)
@pytest.mark.parametrize("queries", QUERIES)
def test_a_query_that_is_not_finite(kv, q, dim, queries):
    """NaN in one row of q, over segments that are whole and such that are cut."""
    c = AttendCase([90, 6000, 150, 800], [queries] * 4, kv=kv, q=q, dim=dim, heads=8, kv_heads=2, seed=44)
    clean, err = run_attend(c)
    ref, wabs = reference(c)
    tol = c.tolerance("f32", ref, wabs)
    rows = [(queries // 2, 1), (queries + queries // 3, 3), (3 * queries - 1, 6)]      # sequences 0, 1, 2
    for n, h in rows:
        c.q_wide[n, h, 5] = float("nan")
    got, err = run_attend(c)
    assert err == 0
    assert torch.equal(got[3 * queries:], clean[3 * queries:])
    for n, h in rows:
        assert torch.isnan(got[n, h]).all()
        got[n, h] = ref[n, h]
    n = 4 * queries
    assert torch.all((got[:n] - ref[:n]).abs() <= tol[:n])


@pytest.mark.parametrize("kv,q,dim", KINDS)
@pytest.mark.parametrize("queries", QUERIES)
def test_the_only_key_that_a_query_sees_is_nan(kv, q, dim, queries):
    """Position 0 holds NaN in K and every query sees it; the first query of a whole prompt sees nothing else."""
    c = AttendCase([queries, 90, 3000], [queries] * 3, kv=kv, q=q, dim=dim, heads=8, kv_heads=2, seed=45)
    clean, err = run_attend(c)
    x = c.k.view(torch.uint8) if kv == "e4m3" else c.k
    b, o = c.row_of(0, 0)
    row = torch.full((2, dim), float("nan")).to(c.k.dtype)
    x[b, :, o] = row.view(torch.uint8) if kv == "e4m3" else row
    got, err = run_attend(c)
    assert err == 0
    assert torch.isnan(got[:queries]).all()
    assert torch.equal(got[queries:], clean[queries:])
