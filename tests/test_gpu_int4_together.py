"""The operators of a 4-bit cache one after the other, as a server runs them: a prompt's chunks and decode steps written with
norms and positions, attention over what was written (with and without a window and sinks), rows read back; on two streams at
once, on the largest batch, in one captured step."""

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import paged_kv_cache_144_gb300 as pa  # noqa: E402
from operator_cases import DT, F64, HALF_STEP, rope_reference  # noqa: E402

HQ, HK, D, B = 8, 2, 128, 16
EPS = 1e-6


class Server:
    """One model layer: weights, a pool, tables from a block manager, and the tokens so far in 64 bits."""

    def __init__(self, kv, seqs, seed, window=0, sinks=0, blocks=64):
        g = torch.Generator().manual_seed(seed)
        self.g, self.kv, self.window, self.sinks, self.seqs = g, kv, window, sinks, seqs
        self.qw, self.kw = (1 + 0.2 * torch.randn(D, generator=g) for _ in range(2))
        self.inv = pa.rope_frequencies(D)
        if kv == "i4":
            self.k = torch.zeros(pa.int4_cache_shape(blocks, HK, B), dtype=torch.uint8, device="cuda")
        else:
            self.k = torch.zeros((blocks, HK, B, D), dtype=DT[kv], device="cuda")
        self.v = torch.zeros_like(self.k)
        self.bm = pa.BlockManager(blocks, B, free_order=torch.randperm(blocks, generator=g).tolist())
        for s in range(seqs):
            self.bm.add_sequence(s)
        self.ws = pa.new_workspace(pa.attend_workspace_bytes(seqs, HQ, HK, D, B, blocks, 64, pa.cache_dtype_code(self.k)), "cuda")

    def step(self, counts, stream=None):
        """`counts` new tokens of each sequence: (out, queries, first rows, lengths before)."""
        g, n = self.g, sum(counts)
        q, k, v = (torch.randn((n, h, D), generator=g).to(torch.bfloat16) for h in (HQ, HK, HK))
        before = [self.bm.lengths[s] for s in range(self.seqs)]
        slots, pos = [], []
        for s, c in enumerate(counts):
            for i in range(c):
                slots.append(self.bm.append_slot(s)[0])
                pos.append(before[s] + i)
        slots, pos = torch.tensor(slots), torch.tensor(pos)
        starts = torch.tensor([0] + list(torch.tensor(counts).cumsum(0)), dtype=torch.int32)
        width = max(len(self.bm.block_table(s)) for s in range(self.seqs))
        tables = torch.tensor([self.bm.block_table(s, width) for s in range(self.seqs)], dtype=torch.int32)
        lens = torch.tensor([self.bm.lengths[s] for s in range(self.seqs)], dtype=torch.int32)
        dev = [t.cuda() for t in (q, k, v, slots, pos, starts, tables, lens, self.inv, self.qw, self.kw)]
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream or torch.cuda.current_stream()):
            dq, dk, dv, ds, dp, dst, dt, dl, di, dqw, dkw = dev
            pa.norm_rope_and_cache(dq, dk, dv, self.k, self.v, dp, ds, di, B, q_weight=dqw, k_weight=dkw, eps=EPS)
            out = torch.full((n, HQ, D), 7.0, device="cuda")
            pa.attend(out, dq, self.k, self.v, dt, dl, dst, max(counts), HK, D ** -0.5, B, workspace=self.ws,
                      window=self.window, sinks=self.sinks, pdl=True)
            rows = torch.arange(int(lens.max()))
            every = [tables[s].long()[rows[:int(lens[s])] // B] * B + rows[:int(lens[s])] % B for s in range(self.seqs)]
            read = [pa.read_cache(*(torch.zeros((len(e), HK, D), device="cuda") for _ in range(2)), self.k, self.v, e.cuda(), B)
                    for e in every]
        self.keep = dev
        return out, dq, starts, before, lens, read, (q, pos)

    def check(self, got):
        out, dq, starts, before, lens, read, (q, pos) = got
        torch.cuda.synchronize()
        assert pa.get_device_error() == 0
        # the queries: normed, turned, rounded to bf16
        x = q.to(F64)
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * self.qw.to(F64)
        x = rope_reference(x, pos, self.inv, False, 1.0)
        assert torch.all((dq.cpu().to(F64) - x).abs() <= HALF_STEP["bf16"] * x.abs() + 4e-6 * x.abs().amax(-1, keepdim=True) + 1e-7)
        # attention of those queries over the values that the cache stands for.  Bounds: attend_more (a 4-bit value is rounded to
        # float16 in calls of many rows; normed keys and queries are near one), for values of at most 6
        for s in range(self.seqs):
            T, k64, v64 = int(lens[s]), *(t.cpu().to(F64) for t in read[s])
            for i in range(int(starts[s]), int(starts[s + 1])):
                at = before[s] + i - int(starts[s])
                t = torch.arange(T)
                see = (t <= at) & ((t > at - self.window) | (t < self.sinks) if self.window else torch.ones(T, dtype=torch.bool))
                for h in range(HQ):
                    z = k64[see, h // 4] @ dq[i, h].cpu().to(F64) * D ** -0.5
                    ref = torch.softmax(z, 0) @ v64[see, h // 4]
                    wide = 2 * 1.3e-4 * 2 + 12 * 2.9e-4 * 2 + 2.0 ** -11 + (2.0 ** -8 if self.kv == "bf16" else 2.0 ** -11) ** 2
                    assert torch.all((out[i, h].cpu().to(F64) - ref).abs() <= 6 * wide + 2.0 ** -10)


@pytest.mark.parametrize("kv", ["i4", "bf16"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (20, 3)])
def test_prompt_chunks_then_decode_steps(kv, window, sinks):
    server = Server(kv, 3, seed=1, window=window, sinks=sinks)
    for counts in ([40, 7, 1], [30, 33, 25], [1, 1, 1], [1, 1, 1], [4, 4, 4]):
        server.check(server.step(counts))


def test_two_servers_on_two_streams():
    servers = [Server("i4", 2, seed=2), Server("i4", 2, seed=3, window=15, sinks=2)]
    streams = [torch.cuda.Stream() for _ in servers]
    for counts in ([50, 20], [1, 1], [1, 1], [16, 3]):
        got = [s.step(counts, stream) for s, stream in zip(servers, streams)]
        for s, x in zip(servers, got):
            s.check(x)


def test_forked_sequence_with_a_copied_block():
    """A shared prefix: the fork writes into a copy of the shared block, the parent's row stays."""
    server = Server("i4", 2, seed=4)
    server.check(server.step([21, 1]))
    server.bm.free(1)
    server.bm.fork(0, 1)
    pair = server.bm.copy_on_write(1, 1)
    pa.copy_blocks(server.k, server.v, torch.tensor([pair], dtype=torch.int32, device="cuda"))
    server.check(server.step([1, 1]))
    server.check(server.step([1, 1]))


def test_largest_batch():
    """4096 sequences of one query each over 4 bits: every sequence's row is that of a call of its own tokens."""
    g = torch.Generator().manual_seed(5)
    S, heads = 4096, 2
    lens = torch.randint(1, 40, (S,), generator=g)
    need = (lens + 7) // 8
    tables = torch.full((S, 5), -1, dtype=torch.int32)
    perm, at = torch.randperm(int(need.sum()), generator=g).to(torch.int32), 0
    for s in range(S):
        tables[s, :need[s]] = perm[at:at + int(need[s])]
        at += int(need[s])
    k, v = (torch.zeros(pa.int4_cache_shape(at, 1, 8), dtype=torch.uint8, device="cuda") for _ in range(2))
    x, y = (torch.randn((at * 8, 1, D), generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    pa.reshape_and_cache(x, y, k, v, torch.arange(at * 8, device="cuda"), 8)
    q = torch.randn((S, heads, D), generator=g).to(torch.bfloat16)
    out = torch.zeros((S, heads, D), device="cuda")
    ws = pa.new_workspace(pa.attend_workspace_bytes(S, heads, 1, D, 8, 5, 1, pa.PA_INT4), "cuda")
    pa.attend(out, q.cuda(), k, v, tables.cuda(), lens.to(torch.int32).cuda(), None, 1, 1, D ** -0.5, 8, workspace=ws)
    kf, vf = (torch.zeros((at * 8, 1, D), device="cuda") for _ in range(2))
    pa.read_cache(kf, vf, k, v, torch.arange(at * 8, device="cuda"), 8)
    assert pa.get_device_error() == 0
    kf, vf, got = kf.cpu().to(F64)[:, 0], vf.cpu().to(F64)[:, 0], out.cpu().to(F64)
    for s in range(0, S, 37):
        t = torch.arange(int(lens[s]))
        rows = tables[s].long()[t // 8] * 8 + t % 8
        z = q[s].to(F64) @ kf[rows].T * D ** -0.5
        ref = torch.softmax(z, -1) @ vf[rows]
        assert torch.all((got[s] - ref).abs() <= 6 * (2.6e-4 + 2.0 ** -15))


def test_one_captured_step_of_writes_attention_and_reads():
    server = Server("i4", 2, seed=6, window=12, sinks=1)
    server.step([30, 9])
    q, k, v = (torch.randn((2, h, D), generator=server.g).to(torch.bfloat16).cuda() for h in (HQ, HK, HK))
    slots = torch.tensor([server.bm.append_slot(s)[0] for s in range(2)]).cuda()
    width = max(len(server.bm.block_table(s)) for s in range(2))
    tables = torch.tensor([server.bm.block_table(s, width) for s in range(2)], dtype=torch.int32).cuda()
    lens = torch.tensor([31, 10], dtype=torch.int32).cuda()
    pos, inv = (lens - 1).long(), server.inv.cuda()
    qw = server.qw.cuda()
    bufs = [[torch.zeros((2, HQ, D), dtype=torch.bfloat16, device="cuda"), torch.zeros((2, HQ, D), device="cuda"),
             torch.zeros((2, HK, D), device="cuda"), torch.zeros((2, HK, D), device="cuda")] for _ in range(2)]

    def step(q_out, out, ko, vo):
        pa.norm_rope_and_cache(q, k, v, server.k, server.v, pos, slots, inv, B, q_weight=qw, k_weight=qw, q_out=q_out, pdl=True)
        pa.attend(out, q_out, server.k, server.v, tables, lens, None, 1, HK, D ** -0.5, B, workspace=server.ws, window=12, sinks=1,
                  pdl=True)
        pa.read_cache(ko, vo, server.k, server.v, slots, B, pdl=True)

    step(*bufs[0])
    graph = pa.StepGraph(lambda: step(*bufs[1]))
    for t in bufs[1]:
        t.zero_()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(*bufs):
        assert torch.equal(a, b) and a.abs().max() > 0


def test_the_plain_decode_refuses_a_4_bit_pool():
    k = torch.zeros(pa.int4_cache_shape(4, HK, B), dtype=torch.uint8, device="cuda")
    q = torch.zeros((1, HQ, D), dtype=torch.bfloat16, device="cuda")
    tables, lens = torch.zeros((1, 1), dtype=torch.int32, device="cuda"), torch.ones(1, dtype=torch.int32, device="cuda")
    ones = torch.ones(HK, device="cuda")
    for call in (pa.decode, pa.decode_noalloc):
        with pytest.raises(pa.PagedAttnError):
            call(torch.zeros_like(q), q, k, k.clone(), tables, lens, HK, 1.0, B, k_scale=ones, v_scale=ones)
