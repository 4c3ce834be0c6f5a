"""Host-side tests (no GPU) of the operators around the cache: refusals of the C entry points and of the binding,
option-struct layouts, frequency tables."""

import ctypes
import math

import pytest
import torch

import paged_kv_cache_144_gb300 as pa
from paged_kv_cache_144_gb300 import _lib

A, A2, A3, MIS = 0x10000, 0x20000, 0x30000, 0x10008   # fake device pointers: refused before any use


@pytest.fixture(scope="module")
def lib():
    return pa.load()


def _rope(lib, opt=None, **kw):
    a = dict(qo=A, qos=8 * 128, q=A2, qs=8 * 128, hq=8, k=A, v=A, src=pa.PA_BF16, ks=2 * 128, vs=2 * 128, kc=A, vc=A2,
             kv=pa.PA_BF16, nb=10, pos=A, sm=A, inv=A, r=128, il=0, sc=1.0, n=3, hk=2, d=128, b=16, ki=None, vi=None)
    a.update(kw)
    return lib.pa_rope_and_cache(a["qo"], a["qos"], a["q"], a["qs"], a["hq"], a["k"], a["v"], a["src"], a["ks"], a["vs"],
                                 a["kc"], a["vc"], a["kv"], a["nb"], a["pos"], a["sm"], a["inv"], a["r"], a["il"], a["sc"],
                                 a["n"], a["hk"], a["d"], a["b"], a["ki"], a["vi"],
                                 None if opt is None else ctypes.byref(opt), None)


def test_rope_refusals(lib):
    assert _rope(lib, n=0) == pa.PA_OK
    assert _rope(lib, n=-1) == pa.PA_ERR_SHAPE
    for r in (0, 3, 130, -2):
        assert _rope(lib, r=r) == pa.PA_ERR_SHAPE
    assert _rope(lib, d=96, r=96) == pa.PA_ERR_UNSUPPORTED
    assert _rope(lib, hq=0) == pa.PA_ERR_SHAPE
    for name in ("qo", "q", "k", "v", "kc", "vc", "pos", "sm", "inv"):
        assert _rope(lib, **{name: None}) == pa.PA_ERR_NULL, name
    assert _rope(lib, src=pa.PA_F32) == pa.PA_ERR_DTYPE
    assert _rope(lib, kv=pa.PA_F16) == pa.PA_ERR_DTYPE
    assert _rope(lib, kv=pa.PA_FP8_E4M3) == pa.PA_ERR_NULL
    assert _rope(lib, kv=pa.PA_INT8, ki=A, vi=A) == pa.PA_ERR_NULL
    assert _rope(lib, qs=100) == pa.PA_ERR_SHAPE
    assert _rope(lib, qos=100) == pa.PA_ERR_SHAPE
    assert _rope(lib, ks=100) == pa.PA_ERR_SHAPE
    assert _rope(lib, qo=A2, qos=9 * 128) == pa.PA_ERR_SHAPE      # in place with another stride
    assert _rope(lib, q=MIS) == pa.PA_ERR_ALIGN
    assert _rope(lib, qo=MIS) == pa.PA_ERR_ALIGN
    assert _rope(lib, qs=8 * 128 + 4) == pa.PA_ERR_ALIGN
    bad = pa.CacheWriteOptions()
    bad.struct_size = 0
    assert _rope(lib, bad) == pa.PA_ERR_SHAPE


def _attend(lib, opt=None, **kw):
    a = dict(out=A, od=pa.PA_F32, q=A, qd=pa.PA_BF16, qs=8 * 128, k=A, v=A2, kv=pa.PA_BF16, nb=100, ks=None, vs=None,
             bt=A, mb=16, sl=A, st=A, mq=4, n=9, s=3, hq=8, hk=2, d=128, sc=0.1, b=16, ws=None, wb=0)
    a.update(kw)
    return lib.pa_attend(a["out"], a["od"], a["q"], a["qd"], a["qs"], a["k"], a["v"], a["kv"], a["nb"], a["ks"], a["vs"],
                         a["bt"], a["mb"], a["sl"], a["st"], a["mq"], a["n"], a["s"], a["hq"], a["hk"], a["d"], a["sc"],
                         a["b"], a["ws"], a["wb"], None if opt is None else ctypes.byref(opt), None)


def test_attend_refusals(lib):
    assert _attend(lib, s=0) == pa.PA_OK
    assert _attend(lib, n=0) == pa.PA_OK
    assert _attend(lib, s=-1) == pa.PA_ERR_SHAPE
    assert _attend(lib, n=-1) == pa.PA_ERR_SHAPE
    assert _attend(lib, mq=0) == pa.PA_ERR_SHAPE
    assert _attend(lib, hq=9) == pa.PA_ERR_SHAPE
    assert _attend(lib, hq=65, hk=1, qs=65 * 128) == pa.PA_ERR_UNSUPPORTED
    assert _attend(lib, s=4097) == pa.PA_ERR_UNSUPPORTED
    assert _attend(lib, d=96) == pa.PA_ERR_UNSUPPORTED
    assert _attend(lib, b=12) == pa.PA_ERR_UNSUPPORTED
    assert _attend(lib, b=2048) == pa.PA_ERR_UNSUPPORTED
    assert _attend(lib, mb=0) == pa.PA_ERR_SHAPE
    assert _attend(lib, mb=1 << 24) == pa.PA_ERR_SHAPE
    assert _attend(lib, st=None) == pa.PA_ERR_SHAPE               # several queries need their starts
    assert _attend(lib, st=None, mq=1, n=2) == pa.PA_ERR_SHAPE    # fewer rows than sequences
    for name in ("out", "q", "k", "v", "bt", "sl"):
        assert _attend(lib, **{name: None}) == pa.PA_ERR_NULL, name
    assert _attend(lib, od=pa.PA_INT8) == pa.PA_ERR_DTYPE
    assert _attend(lib, qd=pa.PA_F32) == pa.PA_ERR_DTYPE
    assert _attend(lib, kv=pa.PA_F16) == pa.PA_ERR_DTYPE
    assert _attend(lib, kv=pa.PA_F32) == pa.PA_ERR_DTYPE
    assert _attend(lib, kv=pa.PA_FP8_E4M3) == pa.PA_ERR_NULL
    assert _attend(lib, kv=pa.PA_INT8, ks=A, vs=A) == pa.PA_ERR_NULL
    assert _attend(lib, kv=pa.PA_FP8_E4M3, ks=A, vs=A, d=64, qs=8 * 64) == pa.PA_ERR_UNSUPPORTED
    assert _attend(lib, nb=0) == pa.PA_ERR_SHAPE
    assert _attend(lib, nb=1 << 40) == pa.PA_ERR_SHAPE
    assert _attend(lib, qs=100) == pa.PA_ERR_SHAPE
    assert _attend(lib, qs=8 * 128 + 4) == pa.PA_ERR_ALIGN
    assert _attend(lib, q=MIS) == pa.PA_ERR_ALIGN
    assert _attend(lib, out=MIS) == pa.PA_ERR_ALIGN
    assert _attend(lib, k=MIS) == pa.PA_ERR_ALIGN


def test_attend_option_refusals(lib):
    O = pa.AttendOptions
    bad = O()
    bad.struct_size = 0
    assert _attend(lib, bad) == pa.PA_ERR_SHAPE
    for cap in (-1.0, math.nan, math.inf):
        assert _attend(lib, O(softcap=cap)) == pa.PA_ERR_SHAPE
    assert _attend(lib, O(window=-1)) == pa.PA_ERR_SHAPE
    assert _attend(lib, O(window=4, prefix_lens=A)) == pa.PA_ERR_UNSUPPORTED
    assert _attend(lib, O(window=4, tree_mask=A, tree_words=1)) == pa.PA_ERR_UNSUPPORTED
    assert _attend(lib, O(tree_mask=A, tree_words=1, slopes=A)) == pa.PA_ERR_UNSUPPORTED
    assert _attend(lib, O(tree_mask=A, tree_words=1, prefix_lens=A)) == pa.PA_ERR_UNSUPPORTED
    assert _attend(lib, O(tree_mask=A, tree_words=0)) == pa.PA_ERR_SHAPE
    assert _attend(lib, O(tree_mask=A, tree_words=1), mq=65) == pa.PA_ERR_SHAPE
    assert _attend(lib, O(mass=A, mass_stride_seq=2 * 256, mass_stride_head=256)) == pa.PA_ERR_UNSUPPORTED  # max_q_len 4
    assert _attend(lib, O(mass=A, mass_stride_seq=2 * 256, mass_stride_head=255), mq=1) == pa.PA_ERR_SHAPE
    assert _attend(lib, O(mass=A, mass_stride_seq=256, mass_stride_head=256), mq=1) == pa.PA_ERR_SHAPE


def test_attend_softcap_range(lib):
    for cap in (1e-40, 2.0 ** -11, 513.0, 1e6):
        assert _attend(lib, pa.AttendOptions(softcap=cap)) == pa.PA_ERR_UNSUPPORTED


def test_attend_workspace_refusals(lib):
    def n(**kw):
        a = dict(s=3, hq=8, hk=2, d=128, b=16, mb=16, mq=4, kv=pa.PA_BF16, acc=0)
        a.update(kw)
        return lib.pa_attend_workspace_bytes(a["s"], a["hq"], a["hk"], a["d"], a["b"], a["mb"], a["mq"], a["kv"], a["acc"])
    assert n(hq=9) == _lib.SIZE_MAX
    assert n(d=80) == _lib.SIZE_MAX
    assert n(kv=pa.PA_F32) == _lib.SIZE_MAX
    assert n(acc=1) == _lib.SIZE_MAX                               # weights need one query per sequence
    with pytest.raises(pa.PagedAttnError):
        pa.attend_workspace_bytes(3, 9, 2, 128, 16, 16, 4)


def _commit(lib, **kw):
    a = dict(k=A, v=A2, kv=pa.PA_BF16, nb=100, bt=A, mb=16, sl=A, st=A, p=A, pl=A, mp=8, nl=A2, s=3, hk=2, d=128, b=16)
    a.update(kw)
    return lib.pa_commit_tree(a["k"], a["v"], a["kv"], a["nb"], a["bt"], a["mb"], a["sl"], a["st"], a["p"], a["pl"],
                              a["mp"], a["nl"], a["s"], a["hk"], a["d"], a["b"], None)


def test_commit_refusals(lib):
    assert _commit(lib, s=0) == pa.PA_OK
    assert _commit(lib, s=-1) == pa.PA_ERR_SHAPE
    assert _commit(lib, mp=0) == pa.PA_ERR_SHAPE
    assert _commit(lib, mp=257) == pa.PA_ERR_UNSUPPORTED
    assert _commit(lib, nl=A) == pa.PA_ERR_SHAPE                   # new_lens must not be seq_lens
    for name in ("k", "v", "bt", "sl", "st", "p", "pl", "nl"):
        assert _commit(lib, **{name: None}) == pa.PA_ERR_NULL, name
    assert _commit(lib, kv=pa.PA_F32) == pa.PA_ERR_DTYPE
    assert _commit(lib, kv=pa.PA_INT8, d=64) == pa.PA_ERR_UNSUPPORTED
    assert _commit(lib, nb=0) == pa.PA_ERR_SHAPE
    assert _commit(lib, k=MIS) == pa.PA_ERR_ALIGN


def _evict(lib, **kw):
    a = dict(k=A, v=A2, kv=pa.PA_BF16, nb=100, m=A, ms=2 * 256, mh=256, bt=A, mb=16, sl=A, dt=A, md=4, kept=A, mo=A2,
             nl=A2, s=3, hk=2, d=128, b=16, budget=64, recent=8, sinks=2)
    a.update(kw)
    return lib.pa_evict(a["k"], a["v"], a["kv"], a["nb"], a["m"], a["ms"], a["mh"], a["bt"], a["mb"], a["sl"], a["dt"],
                        a["md"], a["kept"], a["mo"], a["nl"], a["s"], a["hk"], a["d"], a["b"], a["budget"], a["recent"],
                        a["sinks"], None)


def test_evict_refusals(lib):
    assert _evict(lib, s=0) == pa.PA_OK
    assert _evict(lib, s=-1) == pa.PA_ERR_SHAPE
    assert _evict(lib, budget=0) == pa.PA_ERR_SHAPE
    assert _evict(lib, recent=-1) == pa.PA_ERR_SHAPE
    assert _evict(lib, sinks=-1) == pa.PA_ERR_SHAPE
    assert _evict(lib, recent=60, sinks=5) == pa.PA_ERR_SHAPE
    assert _evict(lib, recent=2 ** 31 - 1, sinks=2 ** 31 - 1) == pa.PA_ERR_SHAPE
    assert _evict(lib, md=3) == pa.PA_ERR_SHAPE                    # 48 rows for a budget of 64
    assert _evict(lib, mh=255) == pa.PA_ERR_SHAPE
    assert _evict(lib, ms=256) == pa.PA_ERR_SHAPE
    assert _evict(lib, nl=A) == pa.PA_ERR_SHAPE
    assert _evict(lib, mo=A) == pa.PA_ERR_SHAPE
    for name in ("k", "v", "m", "bt", "sl", "dt", "kept", "mo", "nl"):
        assert _evict(lib, **{name: None}) == pa.PA_ERR_NULL, name
    assert _evict(lib, v=MIS) == pa.PA_ERR_ALIGN
    assert _evict(lib, b=24) == pa.PA_ERR_UNSUPPORTED


def test_option_struct_layout_matches_the_header(tmp_path):
    """The ctypes structure against a program compiled from the header."""
    import os
    import shutil
    import subprocess
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    names = [f for f, _ in pa.AttendOptions._fields_]
    src = "#include <stdio.h>\n#include <stddef.h>\n#include \"pa.h\"\nint main(void) {\n"
    src += "printf(\"%zu\\n\", sizeof(pa_attend_options));\n"
    src += "".join(f"printf(\"%zu\\n\", offsetof(pa_attend_options, {n}));\n" for n in names) + "return 0; }\n"
    (tmp_path / "o.c").write_text(src)
    subprocess.run([cc, "-I", os.path.dirname(_lib.HEADER), str(tmp_path / "o.c"), "-o", str(tmp_path / "o")], check=True)
    got = [int(x) for x in subprocess.run([str(tmp_path / "o")], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(pa.AttendOptions)] + [getattr(pa.AttendOptions, n).offset for n in names]


def test_host_tensors_are_refused():
    q = torch.zeros((2, 4, 64), dtype=torch.float16)
    kc = torch.zeros((8, 4, 16, 64), dtype=torch.float16)
    i = torch.zeros(2, dtype=torch.int32)
    t = torch.zeros((2, 2), dtype=torch.int32)
    pos = torch.zeros(2, dtype=torch.int64)
    m = torch.zeros((2, 4, 32))
    with pytest.raises(ValueError, match="CUDA tensor"):
        pa.attend(q.clone(), q, kc, kc, t, i, None, 1, 4, 0.1, 16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        pa.attend_tree(q.clone(), q, kc, kc, t, i, i, 1, pos.view(2, 1), 4, 0.1, 16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        pa.attend_accumulate(q.clone(), q, kc, kc, t, i, m, 4, 0.1, 16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        pa.rope_and_cache(q, q, q, kc, kc, pos, pos, torch.ones(32), 16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        pa.commit_tree(kc, kc, t, i, i, t, i, i.clone(), 16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        pa.evict(kc, kc, m, t, i, t, t, m, i.clone(), 16, budget=4)


def test_frequency_tables():
    f = pa.rope_frequencies(8, 10000.0)
    assert torch.allclose(f.double(), torch.tensor([1.0, 0.1, 0.01, 0.001], dtype=torch.float64), rtol=1e-6)
    assert torch.allclose(pa.rope_frequencies(8, scaling="linear", factor=4.0), f / 4)
    b = pa.rope_frequencies(8, scaling="base", factor=16.0)
    assert b[0] == 1.0 and abs(float(f[3] / b[3]) - 16.0) < 1e-4
    g = pa.rope_frequencies(128, 500000.0, scaling="bands", factor=8.0, original_positions=8192)
    p = pa.rope_frequencies(128, 500000.0)
    turns = p.double() * 8192 / (2 * math.pi)
    assert torch.equal(g[turns > 4], p[turns > 4]) and torch.allclose(g[turns < 1], p[turns < 1] / 8)
    mid = (turns > 1) & (turns < 4)
    assert torch.all(g[mid] < p[mid]) and torch.all(g[mid] > p[mid] / 8)
    for kw in (dict(rotary_dim=7), dict(rotary_dim=0), dict(rotary_dim=8, scaling="what"),
               dict(rotary_dim=2, scaling="base"), dict(rotary_dim=8, scaling="bands")):
        with pytest.raises(ValueError):
            pa.rope_frequencies(**kw)
