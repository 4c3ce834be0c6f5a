"""NaN and infinity in the cache of one sequence of a batch: the rows that see them say so, every other row of the call is
what it was without them, and no wait of the pipelines depends on how long the affected rows take.

The limit of the waits is shortened to a few milliseconds (pa_debug_set_decode_wait), much less than the rows of the long
sequence take when they are computed again: a wait that depended on them would run out and set PA_DEVERR_TIMEOUT."""

import contextlib

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import paged_kv_cache_144_gb300 as pa  # noqa: E402
from operator_cases import AttendCase, run_attend  # noqa: E402
from test_gpu_attend_whole import reference  # noqa: E402


@contextlib.contextmanager
def wait_limit(ms):
    pa.pa_debug_set_decode_wait(ms * 1_000_000, False)
    try:
        yield
    finally:
        pa.pa_debug_set_decode_wait(0, False)


def put(c, which, s, t, value):
    """value in the K or V row of position t of sequence s, every head; returns what undoes it."""
    x = getattr(c, which)
    b, o = c.row_of(s, t)
    codes = x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x
    old = codes[b, :, o].clone()
    row = torch.full((c.kv_heads, c.dim), value).to(x.dtype)
    codes[b, :, o] = row.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else row

    def undo():
        codes[b, :, o] = old

    return undo


def check_one_bad_sequence(c, bad, which, t, value, ms):
    """Sequence `bad` holds `value` at position t; compares the call with the clean one and the 64-bit form."""
    rows = [sum(c.qlens[:bad]) + i for i in range(c.qlens[bad])]
    others = torch.ones(c.rows, dtype=torch.bool)
    others[rows] = False
    clean, err = run_attend(c)
    assert err == 0
    see = torch.tensor([bool(c.visible(bad, i)[t]) for i in range(c.qlens[bad])])
    undo = put(c, which, bad, t, value)
    need = pa.attend_workspace_bytes(len(c.lens), c.heads, c.kv_heads, c.dim, c.block, c.tables.shape[1], max(c.qlens),
                                     pa.dtype_code(c.k))
    ws = pa.new_workspace(need, "cuda")
    with wait_limit(ms):
        got, err = run_attend(c, workspace=ws)
    undo()
    assert err == 0, f"device error bits {err}"
    assert torch.equal(got[others], clean[others])
    ref, wabs = reference(c)                                  # (without the value, which the rows below do not see)
    tol = c.tolerance("f32", ref, wabs)
    mine = got[rows]
    assert torch.all((mine - ref[rows]).abs()[~see] <= tol[rows][~see])
    assert not torch.isfinite(mine[see]).any()
    after, err = run_attend(c, workspace=ws)                  # the workspace is ready for the next call
    assert err == 0 and torch.equal(after, clean)


KINDS = [("bf16", "bf16", 128), ("f16", "f16", 64), ("e4m3", "bf16", 128)]


@pytest.mark.parametrize("kv,q,dim", KINDS)
@pytest.mark.parametrize("which,value", [("v", float("nan")), ("v", float("inf")), ("k", float("nan"))])
def test_one_row_tile(kv, q, dim, which, value):
    """96 rows per KV head: the streams take position tiles in turn, the long sequence is cut over the device."""
    if kv == "e4m3" and value == float("inf"):
        pytest.skip("e4m3 has no infinity")
    c = AttendCase([300, 12000, 700, 150, 2000], [24] * 5, kv=kv, q=q, dim=dim, heads=8, kv_heads=2, seed=40)
    check_one_bad_sequence(c, 1, which, 11995, value, 20)


@pytest.mark.parametrize("kv,q,dim", KINDS)
def test_several_row_tiles(kv, q, dim):
    """320 rows per KV head: the streams are row tiles."""
    c = AttendCase([300, 6000, 700, 90], [80] * 4, kv=kv, q=q, dim=dim, heads=8, kv_heads=2, seed=41)
    check_one_bad_sequence(c, 1, "v", 5990, float("nan"), 20)


@pytest.mark.parametrize("kv,q,dim", KINDS)
def test_whole_segments_of_several_tiles(kv, q, dim):
    """Many sequences of two and three tiles, whole in a CTA each, one of them bad."""
    lens = [200 + 7 * (s % 20) for s in range(64)]
    c = AttendCase(lens, [20] * 64, kv=kv, q=q, dim=dim, heads=32, kv_heads=8, seed=42)
    check_one_bad_sequence(c, 37, "v", lens[37] - 3, float("nan"), 10)


@pytest.mark.parametrize("kv,q,dim", KINDS)
@pytest.mark.parametrize("group", [4, 8])
def test_few_rows(kv, q, dim, group):
    """16 and 32 rows per KV head on the decode kernel's variants; segments cut in several pieces, and whole ones."""
    lens = [1500 + 3 * (s % 7) for s in range(40 if group == 8 else 200)]
    c = AttendCase(lens, [4] * len(lens), kv=kv, q=q, dim=dim, heads=8 * group, kv_heads=8, seed=43)
    for bad in (11, 39):
        check_one_bad_sequence(c, bad, "v", lens[bad] - 2, float("nan"), 5)
