"""The workspace of attend_workspace_bytes for some sizes serves every call with fewer sequences, queries or blocks per
sequence: also where the decode kernel's launch shape changes with the batch (its per-sequence arrays take shared memory from
the rings, so the number of warps, and of their records, falls as the batch grows)."""

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import paged_kv_cache_144_gb300 as pa  # noqa: E402

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}


@pytest.mark.parametrize("kv,dim,group", [("bf16", 128, 4), ("bf16", 128, 16), ("f16", 64, 8), ("f16", 64, 40), ("e4m3", 128, 2),
                                          ("e4m3", 128, 64)])
@pytest.mark.parametrize("most", [4096, 3000, 600])
def test_accumulating_calls_of_every_smaller_batch(kv, dim, group, most):
    block = 8
    g = torch.Generator(device="cuda").manual_seed(1)
    k = torch.randn((most, 1, block, dim), device="cuda", generator=g).to(DT[kv])
    q = torch.randn((most, group, dim), device="cuda", generator=g).to(torch.float16 if kv == "f16" else torch.bfloat16)
    scale = torch.full((1,), 0.5, device="cuda") if kv == "e4m3" else None
    tables = torch.arange(most, dtype=torch.int32, device="cuda").view(-1, 1)
    lens = torch.full((most,), block, dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    mass = torch.zeros((most, 1, block), device="cuda")
    ws = pa.new_workspace(pa.attend_workspace_bytes(most, group, 1, dim, block, 1, 1, pa.dtype_code(k), accumulate=True), "cuda")
    sizes = list(range(most, 0, -61)) + [1 << i for i in range(13) if 1 << i <= most] + [1]
    total = torch.zeros(most, dtype=torch.int64)
    for n in sizes:
        pa.attend_accumulate(out[:n], q[:n], k, k, tables[:n], lens[:n], mass[:n], 1, 0.1, block, workspace=ws, k_scale=scale,
                             v_scale=scale)
        total[:n] += 1
    assert pa.get_device_error() == 0
    # the weights of a row sum to one: the totals of a (sequence, KV head) to the group's heads, once per call (float32 sums
    # of at most 90 calls of values up to the group's size, each weight off by at most 3e-4 relative)
    want = total.double() * group
    assert torch.all((mass.double().sum((1, 2)).cpu() - want).abs() <= 3e-4 * want)


@pytest.mark.parametrize("kv,dim", [("bf16", 128), ("f16", 64), ("e4m3", 128)])
def test_ragged_calls_of_every_smaller_batch(kv, dim):
    most, queries, block, group = 2000, 7, 8, 6
    g = torch.Generator(device="cuda").manual_seed(2)
    k = torch.randn((most, 1, block, dim), device="cuda", generator=g).to(DT[kv])
    v = torch.ones((most, 1, block, dim), device="cuda").to(DT[kv])
    q = torch.randn((most * queries, group, dim), device="cuda", generator=g).to(torch.float16 if kv == "f16" else torch.bfloat16)
    scale = torch.ones((1,), device="cuda") if kv == "e4m3" else None
    tables = torch.arange(most, dtype=torch.int32, device="cuda").view(-1, 1)
    lens = torch.full((most,), block, dtype=torch.int32, device="cuda")
    ws = pa.new_workspace(pa.attend_workspace_bytes(most, group, 1, dim, block, 1, queries, pa.dtype_code(k)), "cuda")
    for n in list(range(most, 0, -61)) + [1]:
        for length in (queries, 5, 2, 1):
            starts = torch.arange(n + 1, dtype=torch.int32, device="cuda") * length
            out = torch.zeros((n * length, group, dim), device="cuda")
            pa.attend(out, q[:n * length], k, v, tables[:n], lens[:n], starts, length, 1, 0.1, block, workspace=ws, k_scale=scale,
                      v_scale=scale)
            # every V is one: so is an average of them (weights and their sum: float32, P as two 16-bit parts: 2^-16)
            assert (out - 1.0).abs().max() <= 1e-4
    assert pa.get_device_error() == 0
