"""A step over 4-bit caches -- append, decode, weights, eviction -- at contexts that the calls
split over CTAs (workspaces, second kernels): replayed in graphs at once, on two streams at once,
and with one workspace for all calls of a stream."""
import pytest
import torch

import paged_kv_cache_310_gb300 as pkv

pytestmark = pytest.mark.gpu

HEADS, BS, D, HQ = 8, 16, 128, 32
SCALE = D ** -0.5


class Server:
    """Three sequences in a 4-bit pool, the longest of `length` tokens, and one step."""

    def __init__(self, seed, length, out_dtype=torch.bfloat16):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.gen, self.length, self.keep = gen, length, length // 3
        self.lens_host = [length, 41, length // 2]
        need = [-(-n // BS) for n in self.lens_host]
        fresh = -(-self.keep // BS)
        nb = sum(need) + 3 * fresh + 5
        self.kc, self.vc = (torch.zeros((nb, HEADS, BS, D * 5 // 8), dtype=torch.uint8, device="cuda") for _ in range(2))
        perm = torch.randperm(nb, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
        tables = torch.full((3, need[0]), -1, dtype=torch.int32)
        at = 0
        for s, c in enumerate(need):
            tables[s, :c] = perm[at:at + c]
            at += c
        self.tables, self.new = tables.cuda(), perm[at:at + 3 * fresh].reshape(3, fresh).cuda()
        self.lens = torch.tensor(self.lens_host, dtype=torch.int32).cuda()
        slots = [int(tables[s, j // BS]) * BS + j % BS for s, n in enumerate(self.lens_host) for j in range(n)]
        x = [torch.randn(len(slots), HEADS, D, generator=gen, device="cuda").bfloat16() for _ in range(2)]
        pkv.paged_kv4_append(*x, torch.tensor(slots).cuda(), self.kc, self.vc)
        last = [int(tables[s, (n - 1) // BS]) * BS + (n - 1) % BS for s, n in enumerate(self.lens_host)]
        self.slots = torch.tensor(last).cuda()
        self.k, self.v = (torch.empty(3, HEADS, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.q = torch.empty(3, HQ, D, dtype=torch.bfloat16, device="cuda")
        self.out = torch.empty(3, HQ, D, dtype=out_dtype, device="cuda")
        self.w = torch.rand(3, HEADS, length, generator=gen, device="cuda")
        self.w_next, self.w_out = torch.zeros_like(self.w), torch.zeros_like(self.w)
        self.keep_lens = torch.tensor([self.keep, 33, self.keep - 7], dtype=torch.int32).cuda()
        self.kept = torch.full((3, HEADS, self.keep), -1, dtype=torch.int32, device="cuda")

    def inputs(self):
        for x in (self.k, self.v, self.q):
            x.copy_(torch.randn(x.shape, generator=self.gen, device="cuda"))

    def needs(self):
        return [pkv.paged_attention_decode_kv4_workspace_bytes(3, HQ, self.length, self.q.dtype, self.kc),
                pkv.paged_attention_weights_workspace_bytes(3, HQ, self.length, self.kc)]

    def step(self, ws=None):
        n = self.length
        pkv.paged_kv4_append(self.k, self.v, self.slots, self.kc, self.vc)
        pkv.paged_attention_decode_kv4(self.q, self.kc, self.vc, self.tables, self.lens, SCALE, self.out, max_context_len=n,
                                       workspace=ws)
        pkv.paged_attention_weights(self.q, self.kc, self.tables, self.lens, SCALE, self.w, weights_out=self.w_next,
                                    max_context_len=n, workspace=ws)
        pkv.paged_kv_evict(self.w_next, self.tables, self.lens, self.keep_lens, self.new, self.kc, self.vc, self.w_out,
                           self.kept, recent=8, max_context_len=n)

    def results(self):
        return [t.clone() for t in (self.out, self.w_next, self.w_out, self.kept, self.kc, self.vc)]


@pytest.mark.parametrize("length", [300, 1300, 9000])
def test_steps_replay_in_graphs_at_once(length):
    servers = [Server(311_800, length), Server(311_801, length, torch.float32)]
    assert all((n > 0) == (length > 512) for s in servers for n in s.needs())
    for s in servers:
        s.inputs()
        s.step()
    torch.cuda.synchronize()
    graphs = []
    for s in servers:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.step()
        graphs.append(g)
    for _ in range(3):
        for s in servers:
            s.inputs()
        streams = [torch.cuda.Stream() for _ in servers]
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        replayed = [s.results() for s in servers]
        for s in servers:
            s.step()
        torch.cuda.synchronize()
        assert pkv.device_error() == 0
        for s, got in zip(servers, replayed):
            assert all(torch.equal(a, b) for a, b in zip(got, s.results()))


@pytest.mark.parametrize("length", [1300, 9000])
def test_eager_steps_on_two_streams_at_once(length):
    servers = [Server(311_810 + i, length) for i in range(2)]
    assert all(n > 0 for s in servers for n in s.needs())
    for s in servers:
        s.inputs()
        s.step()
    torch.cuda.synchronize()
    want = [s.results() for s in servers]
    streams = [torch.cuda.Stream() for _ in servers]
    for _ in range(25):
        for s, st in zip(servers, streams):
            with torch.cuda.stream(st):
                s.step()
    torch.cuda.synchronize()
    assert pkv.device_error() == 0
    for s, w in zip(servers, want):
        assert all(torch.equal(a, b) for a, b in zip(w, s.results()))


@pytest.mark.parametrize("length", [1300, 9000])
def test_calls_back_to_back_share_a_workspace(length):
    # one buffer for every call of a stream, beside the other decode's
    s = Server(311_820, length)
    s.inputs()
    s.step()
    torch.cuda.synchronize()
    want = s.results()
    wide = [torch.randn(s.kc.shape[0], HEADS, BS, D, device="cuda").bfloat16() for _ in range(2)]
    needs = s.needs() + [pkv.paged_attention_workspace_bytes(3, HQ, length, wide[0], partition_tokens=128)]
    assert all(n > 0 for n in needs)
    ws = torch.empty(max(needs), dtype=torch.uint8, device="cuda")
    other = [torch.empty(3, HQ, D, device="cuda") for _ in range(2)]
    kw = dict(max_context_len=length, workspace=ws)
    for _ in range(20):
        pkv.paged_attention_decode(s.q, *wide, s.tables, s.lens, SCALE, other[0], partition_tokens=128, **kw)
        pkv.paged_attention_decode_kv4(s.q, s.kc, s.vc, s.tables, s.lens, SCALE, s.out, **kw)
        pkv.paged_attention_decode(s.q, *wide, s.tables, s.lens, SCALE, other[1], partition_tokens=128, **kw)
        pkv.paged_attention_weights(s.q, s.kc, s.tables, s.lens, SCALE, s.w, weights_out=s.w_next, **kw)
        s.step(ws)
    torch.cuda.synchronize()
    assert pkv.device_error() == 0 and torch.equal(other[0], other[1])
    assert all(torch.equal(a, b) for a, b in zip(want, s.results()))
