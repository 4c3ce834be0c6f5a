"""Steps whose decode reads its lengths, tables and first K/V rows early (pdl, early_kv), after kernels that write those: the
launch order that include/pa.h asks for (an ordinary cache write between them) gives what ordinary launches give."""

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import paged_kv_cache_144_gb300 as pa  # noqa: E402

HQ, HKV, D = 8, 2, 128


class Step:
    """S sequences of `length` tokens in blocks of B, as many spare blocks, and the newest tokens' rows."""

    def __init__(self, S, length, B, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.S, self.B = S, B
        per = -(-length // B)

        def rand(*shape):
            return torch.randn(shape, device="cuda", generator=g).to(torch.bfloat16)

        self.k, self.v = rand(2 * S * per, HKV, B, D), rand(2 * S * per, HKV, B, D)
        perm = torch.randperm(2 * S * per, device="cuda", generator=g).to(torch.int32)
        self.tables, self.spare = perm[:S * per].view(S, per).contiguous(), perm[S * per:].view(S, per).contiguous()
        self.lens = torch.full((S,), length, dtype=torch.int32, device="cuda")
        self.q, self.kn, self.vn = rand(S, HQ, D), rand(S, HKV, D), rand(S, HKV, D)
        self.turned, self.inv = torch.empty_like(self.q), pa.rope_frequencies(D).cuda()
        self.out = torch.zeros((S, HQ, D), device="cuda")
        self.ws = pa.new_workspace(pa.decode_workspace_bytes(S, HQ, HKV, D, B, per), "cuda")

    def slots_of(self, positions):
        return self.tables[torch.arange(self.S, device="cuda"), positions // self.B].long() * self.B + positions % self.B

    def run(self, lens, positions, slots, rope, overlap):
        """The newest rows' cache write, an ordinary launch, and the decode."""
        if rope:
            pa.rope_and_cache(self.q, self.kn, self.vn, self.k, self.v, positions, slots, self.inv, self.B, q_out=self.turned)
        else:
            pa.reshape_and_cache(self.kn, self.vn, self.k, self.v, slots, self.B)
        pa.decode(self.out, self.turned if rope else self.q, self.k, self.v, self.tables, lens, HKV, D ** -0.5, self.B,
                  workspace=self.ws, pdl=overlap, early_kv=overlap)
        assert pa.get_device_error() == 0
        return self.out.clone()


@pytest.mark.parametrize("rope", [False, True])
@pytest.mark.parametrize("B", [16, 256])
def test_after_a_block_copy(rope, B):
    """Every block of every sequence is copied from elsewhere right before the step; until then it holds NaN."""
    outs = []
    for overlap in (False, True):
        s = Step(24, 2000, B, 1)
        pairs = torch.stack([s.spare.flatten(), s.tables.flatten()], 1).contiguous()
        for x in (s.k, s.v):
            x[s.tables.flatten().long()] = float("nan")
        positions = (s.lens - 1).long()
        slots = s.slots_of(positions)
        torch.cuda.synchronize()
        pa.copy_blocks(s.k, s.v, pairs)
        outs.append(s.run(s.lens, positions, slots, rope, overlap))
    assert torch.isfinite(outs[0]).all() and torch.equal(outs[0], outs[1])


@pytest.mark.parametrize("rope", [False, True])
def test_after_a_commit(rope):
    """commit_tree moves rows and writes the lengths that the decode right behind the cache write reads."""
    outs = []
    for overlap in (False, True):
        s = Step(16, 1500, 16, 2)
        nodes = 40
        starts = torch.arange(17, dtype=torch.int32, device="cuda") * nodes
        path = torch.tensor([[0, 3, 7, 20, 39]] * 16, dtype=torch.int32, device="cuda")
        plens = torch.tensor([1 + i % 5 for i in range(16)], dtype=torch.int32, device="cuda")
        new = torch.full((16,), 1, dtype=torch.int32, device="cuda")
        positions = (s.lens - nodes + plens - 1).long()    # the newest position of the committed path
        slots = s.slots_of(positions)
        torch.cuda.synchronize()
        pa.commit_tree(s.k, s.v, s.tables, s.lens, starts, path, plens, new, s.B)
        outs.append(s.run(new, positions, slots, rope, overlap))
        assert torch.equal(new, s.lens - nodes + plens)
    assert torch.isfinite(outs[0]).all() and torch.equal(outs[0], outs[1])
