"""Host-side tests (no GPU) of the 4-bit cache's calls: refusals of the C entry points and of the binding."""

import ctypes
import math

import pytest
import torch

import int4_cases
import paged_kv_cache_144_gb300 as pa

A, A2, A3, MIS = 0x10000, 0x2000000, 0x4000000, 0x10008   # fake device pointers: refused before any use


@pytest.fixture(scope="module")
def lib():
    return pa.load()


def _norm(lib, norm="default", opt=None, **kw):
    a = dict(qo=A, qos=8 * 128, q=A2, qs=8 * 128, hq=8, k=A, v=A, src=pa.PA_BF16, ks=2 * 128, vs=2 * 128, kc=A, vc=A2,
             kv=pa.PA_BF16, nb=10, pos=A, sm=A, inv=A, r=128, il=0, sc=1.0, n=3, hk=2, d=128, b=16, ki=None, vi=None)
    a.update(kw)
    if norm == "default":
        norm = pa.NormOptions(q_weight=A, k_weight=A, weight_dtype=pa.PA_BF16, eps=1e-6)
    return lib.pa_norm_rope_and_cache(a["qo"], a["qos"], a["q"], a["qs"], a["hq"], a["k"], a["v"], a["src"], a["ks"], a["vs"],
                                      a["kc"], a["vc"], a["kv"], a["nb"], a["pos"], a["sm"], a["inv"], a["r"], a["il"],
                                      a["sc"], a["n"], a["hk"], a["d"], a["b"], None if norm is None else ctypes.byref(norm),
                                      a["ki"], a["vi"], None if opt is None else ctypes.byref(opt), None)


def test_norm_refusals(lib):
    assert _norm(lib, n=0) == pa.PA_OK
    assert _norm(lib, norm=None) == pa.PA_ERR_NULL
    short = pa.NormOptions()
    short.struct_size = 4
    assert _norm(lib, norm=short) == pa.PA_ERR_SHAPE
    for eps in (-1.0, math.inf, math.nan):
        assert _norm(lib, norm=pa.NormOptions(eps=eps)) == pa.PA_ERR_SHAPE
    assert _norm(lib, norm=pa.NormOptions(q_weight=A, weight_dtype=pa.PA_INT8)) == pa.PA_ERR_DTYPE
    assert _norm(lib, norm=pa.NormOptions(q_weight=A + 2, weight_dtype=pa.PA_F32)) == pa.PA_ERR_ALIGN
    assert _norm(lib, norm=pa.NormOptions(k_weight=A + 1, weight_dtype=pa.PA_F16)) == pa.PA_ERR_ALIGN
    for r in (-2, 3, 130):
        assert _norm(lib, r=r) == pa.PA_ERR_SHAPE
    for name in ("qo", "q", "k", "v", "kc", "vc", "pos", "sm", "inv"):
        assert _norm(lib, **{name: None}) == pa.PA_ERR_NULL, name
    assert _norm(lib, kv=pa.PA_F16) == pa.PA_ERR_DTYPE
    assert _norm(lib, kv=pa.PA_F32) == pa.PA_ERR_DTYPE
    assert _norm(lib, kv=pa.PA_FP8_E4M3) == pa.PA_ERR_NULL
    assert _norm(lib, d=96, r=96) == pa.PA_ERR_UNSUPPORTED
    assert _norm(lib, kv=pa.PA_INT4, d=64, r=64) == pa.PA_ERR_UNSUPPORTED
    for b in (4, 12, 2048):
        assert _norm(lib, kv=pa.PA_INT4, b=b) == pa.PA_ERR_UNSUPPORTED
    assert _norm(lib, qo=A2, qos=9 * 128) == pa.PA_ERR_SHAPE
    assert _norm(lib, q=MIS) == pa.PA_ERR_ALIGN
    assert _norm(lib, kc=MIS) == pa.PA_ERR_ALIGN


def _read(lib, opt=None, **kw):
    a = dict(ko=A, vo=A2, od=pa.PA_F32, kos=256, vos=256, kc=A3, vc=A3, kv=pa.PA_INT4, nb=10, ks=None, vs=None, sm=A, n=3,
             hk=2, d=128, b=16)
    a.update(kw)
    return lib.pa_read_cache(a["ko"], a["vo"], a["od"], a["kos"], a["vos"], a["kc"], a["vc"], a["kv"], a["nb"], a["ks"], a["vs"],
                             a["sm"], a["n"], a["hk"], a["d"], a["b"], None if opt is None else ctypes.byref(opt), None)


def test_read_refusals(lib):
    assert _read(lib, n=0) == pa.PA_OK
    assert _read(lib, n=-1) == pa.PA_ERR_SHAPE
    assert _read(lib, hk=0) == pa.PA_ERR_SHAPE
    for name in ("ko", "vo", "kc", "vc", "sm"):
        assert _read(lib, **{name: None}) == pa.PA_ERR_NULL, name
    assert _read(lib, od=pa.PA_INT8) == pa.PA_ERR_DTYPE
    assert _read(lib, kv=pa.PA_F32) == pa.PA_ERR_DTYPE
    assert _read(lib, kv=pa.PA_FP8_E4M3) == pa.PA_ERR_NULL
    assert _read(lib, kv=pa.PA_INT8, ks=A, vs=A) == pa.PA_ERR_NULL
    assert _read(lib, d=64) == pa.PA_ERR_UNSUPPORTED
    for b in (4, 24, 2048):
        assert _read(lib, b=b) == pa.PA_ERR_UNSUPPORTED
    assert _read(lib, nb=0) == pa.PA_ERR_SHAPE
    assert _read(lib, kos=255) == pa.PA_ERR_SHAPE
    assert _read(lib, kos=258) == pa.PA_ERR_ALIGN
    assert _read(lib, od=pa.PA_BF16, vos=260) == pa.PA_ERR_ALIGN
    assert _read(lib, vo=MIS + A2) == pa.PA_ERR_ALIGN
    assert _read(lib, vo=A) == pa.PA_ERR_SHAPE                      # one buffer for both
    assert _read(lib, vo=A + 512) == pa.PA_ERR_SHAPE                # v's rows start inside k's
    assert _read(lib, vo=A + 1024) == pa.PA_ERR_SHAPE               # v's first row is k's second
    assert _read(lib, vo=A + 512, kos=512, vos=512) == pa.PA_ERR_SHAPE   # side by side, but half a row in
    bad = pa.CacheWriteOptions()
    bad.struct_size = 0
    assert _read(lib, bad) == pa.PA_ERR_SHAPE


def test_other_calls_refuse_four_bits(lib):
    i4 = pa.PA_INT4
    assert lib.pa_commit_tree(A, A2, i4, 100, A, 16, A, A, A, A, 8, A2, 3, 2, 128, 16, None) == pa.PA_ERR_UNSUPPORTED
    assert lib.pa_evict(A, A2, i4, 100, A, 512, 256, A, 16, A, A, 16, A, A2, A3, 3, 2, 128, 16, 64, 0, 0,
                        None) == pa.PA_ERR_UNSUPPORTED
    assert lib.pa_decode(A, pa.PA_F32, A, pa.PA_BF16, 1024, A, A2, i4, 100, None, None, A, 16, A, 3, 8, 2, 128, 0.1, 16, 0,
                         None, 0, None) == pa.PA_ERR_DTYPE
    assert lib.pa_reshape_and_cache(A, A, pa.PA_BF16, 128, 128, A, A2, i4, 10, A, 3, 2, 64, 16, None, None,
                                    None) == pa.PA_ERR_UNSUPPORTED
    assert lib.pa_reshape_and_cache(A, A, pa.PA_BF16, 256, 256, A, A2, i4, 10, A, 3, 2, 128, 12, None, None,
                                    None) == pa.PA_ERR_UNSUPPORTED


def test_option_struct_layout():
    assert ctypes.sizeof(pa.NormOptions) == 40
    assert pa.NormOptions().struct_size == 40


def test_options_of_callers_built_before_sinks(lib):
    """Their struct ends with 4 bytes of padding, whose contents mean nothing."""
    o = pa.AttendOptions(window=8)
    old = pa.AttendOptions.sinks.offset
    assert old % 8 == 0
    o.struct_size, o.reserved, o.sinks = old, -1, -1
    args = (A, pa.PA_F32, A, pa.PA_BF16, 1024, A, A2, pa.PA_BF16, 100, None, None, A, 16, A, A, 4, 0, 3, 8, 2, 128, 0.1, 16,
            None, 0)
    assert lib.pa_attend(*args, ctypes.byref(o), None) == pa.PA_OK
    o.struct_size = ctypes.sizeof(o)
    assert lib.pa_attend(*args, ctypes.byref(o), None) == pa.PA_ERR_SHAPE
    o.sinks = 4
    assert lib.pa_attend(*args, ctypes.byref(o), None) == pa.PA_OK


def test_uint8_pools_of_three_dimensions(lib):
    """An E4M3 pool whose rows are flattened stays one."""
    four, eight = (torch.zeros(s, dtype=torch.uint8) for s in (pa.int4_cache_shape(3, 2, 16), (3, 2, 16 * 128)))
    assert pa.cache_dtype_code(four, 16) == pa.PA_INT4
    assert pa.cache_dtype_code(eight, 16) == pa.PA_FP8_E4M3
    assert pa.cache_dtype_code(four, 16, 64) == pa.PA_FP8_E4M3


def test_binding_refusals():
    q = torch.zeros((2, 4, 128), dtype=torch.bfloat16)
    c = torch.zeros(pa.int4_cache_shape(3, 2, 16), dtype=torch.uint8)
    with pytest.raises(ValueError):                                # not on a GPU
        pa.norm_rope_and_cache(q, q[:, :2], q[:, :2], c, c, None, torch.arange(2), None, 16)
    with pytest.raises(ValueError):
        pa.read_cache(q.float(), q.float(), c, c, torch.arange(2), 16)
    assert pa.cache_dtype_code(c) == pa.PA_INT4
    assert pa.cache_dtype_code(torch.zeros((3, 2, 16, 128), dtype=torch.uint8)) == pa.PA_FP8_E4M3
    assert pa.cache_dtype_code(torch.zeros((3, 2, 16, 128), dtype=torch.bfloat16)) == pa.PA_BF16


def test_pool_shapes_in_the_binding():
    from paged_kv_cache_144_gb300 import _ops
    _ops._t()
    c = torch.zeros(pa.int4_cache_shape(3, 2, 16), dtype=torch.uint8)
    assert _ops._cache(c, c.clone(), 16) == (3, 2, 128)
    for block in (8, 32, 17, 0):
        with pytest.raises(ValueError):
            if _ops._cache(c, c.clone(), block)[2] != 128:
                raise ValueError("another head size")
    with pytest.raises(ValueError):
        _ops._cache(c, c[:2].clone(), 16)
    with pytest.raises(ValueError):
        _ops._cache(c[:, :, :-1], c[:, :, :-1], 16)


def test_tiles_of_the_documented_layout():
    """Value 8 w + 2 j + e of a row in bits 16 e + 4 j of word w; the pairs after all codes."""
    codes = torch.arange(128).view(1, 128).repeat(8, 1) % 16
    codes[1] = 0
    tile = int4_cases.pack(codes, torch.full((8,), 2.0), torch.full((8,), -1.0))
    assert tile.numel() == 8 * 68
    words = tile[:512].view(torch.int32).view(8, 16)
    for w in range(16):
        want = sum(int(codes[0, 8 * w + 2 * j + e]) << (16 * e + 4 * j) for j in range(4) for e in range(2))
        assert int(words[0, w]) & 0xffffffff == want
    assert torch.all(words[1] == 0)
    assert torch.equal(tile[512:].view(torch.float16), torch.tensor([2.0, -1.0] * 8, dtype=torch.float16))
    back, scale, zero = int4_cases.unpack(tile, 8)
    assert torch.equal(back, codes) and torch.all(scale == 2) and torch.all(zero == -1)
