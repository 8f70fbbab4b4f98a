"""4-bit caches and eviction together, and where they meet what a server does: pools whose
offsets pass 32 bits, a captured step replayed, calls on two streams at once, tensors that a
call refuses.  Values against tests/kv4_model.py."""
import numpy as np
import pytest
import torch

import kv4_model as model
import paged_kv_cache_310_gb300 as pkv

pytestmark = pytest.mark.gpu

HEADS, BS, D, HQ = 8, 16, 128, 32
SCALE = D ** -0.5


def test_blocks_past_four_gigabytes():
    nb = 460_000                                            # 4.7 GB a 4-bit pool
    kc, vc = (torch.empty((nb, HEADS, BS, D * 5 // 8), dtype=torch.uint8, device="cuda") for _ in range(2))
    gen = torch.Generator().manual_seed(311_300)
    blocks = [nb - 1, 3, nb - 2, 420_000, 210_001]
    n = 70
    table = torch.tensor([blocks], dtype=torch.int32)
    k, v = (torch.randn(n, HEADS, D, generator=gen) for _ in range(2))
    slots = torch.tensor([blocks[j // BS] * BS + j % BS for j in range(n)])
    pkv.paged_kv4_append(k.cuda(), v.cuda(), slots.cuda(), kc, vc)
    kh, vh = (model.widen(model.quantise(x.double().numpy())) for x in (k, v))
    q = torch.randn(1, HQ, D, generator=gen)
    lens = torch.tensor([n], dtype=torch.int32).cuda()
    out = torch.empty(1, HQ, D, device="cuda")
    pkv.paged_attention_decode_kv4(q.cuda(), kc, vc, table.cuda(), lens, SCALE, out, max_context_len=n)
    p = model.probabilities(q[0].double().numpy(), kh.transpose(1, 0, 2), SCALE)
    ref = np.matmul(p, vh.transpose(1, 0, 2)).reshape(HQ, D)
    assert pkv.device_error() == 0
    assert np.abs(out[0].cpu().double().numpy() - ref).max() <= 1e-4
    w = torch.zeros(1, HEADS, n, device="cuda")
    pkv.paged_attention_weights(q.cuda(), kc, table.cuda(), lens, SCALE, w, max_context_len=n)
    assert np.abs(w[0].cpu().double().numpy() - p.sum(1)).max() <= 1e-4
    # kept rows move between far blocks; widened blocks land in a far block of a 16-bit pool
    new = torch.tensor([[nb - 3, 7]], dtype=torch.int32)
    w_out, kept = torch.zeros_like(w), torch.full((1, HEADS, 20), -1, dtype=torch.int32, device="cuda")
    pkv.paged_kv_evict(w, table.cuda(), lens, torch.tensor([20], dtype=torch.int32).cuda(), new.cuda(), kc, vc, w_out, kept,
                       recent=4, max_context_len=n)
    wide_nb = 140_000                                       # 4.6 GB in bf16
    wide = [torch.empty((wide_nb, HEADS, BS, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    pairs = torch.tensor([[nb - 3, wide_nb - 1], [7, 0]]).cuda()
    pkv.paged_kv4_expand(pairs, kc, vc, *wide)
    assert pkv.device_error() == 0
    for h in range(HEADS):
        rows = model.kept_rows(w[0, h].cpu().numpy(), n, 20, 4)
        assert kept[0, h].tolist() == rows
        for got, held in zip(wide, (kh, vh)):
            moved = torch.cat([got[wide_nb - 1, h], got[0, h, :4]]).cpu()
            assert torch.equal(moved, torch.from_numpy(held[rows, h]).bfloat16())


def test_the_most_sequences_a_call_takes():
    n, d, bs = 65_535, 64, 8
    gen = torch.Generator(device="cuda").manual_seed(311_330)
    rand = lambda *shape: torch.randn(*shape, generator=gen, device="cuda")
    kc, vc = (torch.zeros((n, 1, bs, d * 5 // 8), dtype=torch.uint8, device="cuda") for _ in range(2))
    tables = torch.randperm(n, generator=gen, device="cuda").to(torch.int32)[:, None]
    lens = torch.randint(0, 3, (n,), generator=gen, device="cuda").to(torch.int32)
    slots = (tables.long() * bs + torch.arange(2, device="cuda")).flatten()
    pkv.paged_kv4_append(rand(2 * n, 1, d), rand(2 * n, 1, d), slots, kc, vc)
    wide = [torch.zeros((n, 1, bs, d), device="cuda") for _ in range(2)]
    pairs = torch.arange(n, device="cuda")[:, None].expand(n, 2).contiguous()
    pkv.paged_kv4_expand(pairs, kc, vc, *wide)
    k, v = (x[tables[:, 0].long(), 0, :2].double() for x in wide)               # [n, 2, d]
    q, out = rand(n, 2, d), torch.empty(n, 2, d, device="cuda")
    pkv.paged_attention_decode_kv4(q, kc, vc, tables, lens, 0.125, out, max_context_len=2)
    seen = torch.arange(2, device="cuda") < lens[:, None]                       # [n, 2]
    p = torch.softmax(torch.where(seen[:, None], 0.125 * q.double() @ k.mT, -1e300), -1) * seen[:, None]
    assert pkv.device_error() == 0
    # scores below 15 are good to 15 * 2^-21, a weight to twice that, times values below 5: 7e-5
    assert (out - p @ v).abs().max() <= 1e-4
    w = torch.full((n, 1, 2), 7.0, device="cuda")
    pkv.paged_attention_weights(q, kc, tables, lens, 0.125, w, tracked_lens=torch.zeros_like(lens), max_context_len=2)
    assert (torch.where(seen, w[:, 0] - p.sum(1), w[:, 0] - 7.0)).abs().max() <= 1e-4
    # the heavier row of each sequence becomes the first of a block that nobody reads
    spare = [torch.zeros((2 * n, 1, bs, d * 5 // 8), dtype=torch.uint8, device="cuda") for _ in range(2)]
    for s, c in zip(spare, (kc, vc)):
        s[:n] = c
    new = (2 * n - 1 - torch.arange(n, device="cuda")).to(torch.int32)[:, None]
    w_out, kept = torch.zeros_like(w), torch.full((n, 1, 1), -1, dtype=torch.int32, device="cuda")
    pkv.paged_kv_evict(w, tables, lens, torch.ones_like(lens), new, *spare, w_out, kept, max_context_len=2)
    best = torch.where((lens == 2) & (w[:, 0, 1] > w[:, 0, 0]), 1, 0)
    assert pkv.device_error() == 0
    assert torch.equal(kept[:, 0, 0].long(), torch.where(lens > 0, best, -1))
    some = (lens > 0).nonzero().flatten()
    for s, c in zip(spare, (kc, vc)):
        assert torch.equal(s[new[some, 0].long(), 0, 0], c[tables[some, 0].long(), 0, best[some]])


class Server:
    """Two sequences in a 4-bit pool, and one step: append, decode, weights, eviction."""

    def __init__(self, seed):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.gen, self.lens_host, self.keep = gen, [300, 41], 64
        self.kc, self.vc = (torch.zeros((64, HEADS, BS, D * 5 // 8), dtype=torch.uint8, device="cuda") for _ in range(2))
        perm = torch.randperm(64, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
        tables = torch.full((2, 19), -1, dtype=torch.int32)
        tables[0], tables[1, :3] = perm[:19], perm[19:22]
        self.tables, self.new = tables.cuda(), perm[22:30].reshape(2, 4).cuda()
        self.lens = torch.tensor(self.lens_host, dtype=torch.int32).cuda()
        slots = [int(tables[s, j // BS]) * BS + j % BS for s, n in enumerate(self.lens_host) for j in range(n)]
        x = [torch.randn(len(slots), HEADS, D, generator=gen, device="cuda").bfloat16() for _ in range(2)]
        pkv.paged_kv4_append(*x, torch.tensor(slots).cuda(), self.kc, self.vc)
        last = [int(tables[s, (n - 1) // BS]) * BS + (n - 1) % BS for s, n in enumerate(self.lens_host)]
        self.slots = torch.tensor(last).cuda()
        self.k, self.v = (torch.empty(2, HEADS, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.q = torch.empty(2, HQ, D, dtype=torch.bfloat16, device="cuda")
        self.out = torch.empty(2, HQ, D, device="cuda")
        self.w = torch.rand(2, HEADS, 304, generator=gen, device="cuda")
        self.w_next, self.w_out = torch.empty_like(self.w), torch.zeros_like(self.w)
        self.keep_lens = torch.tensor([self.keep, 33], dtype=torch.int32).cuda()
        self.kept = torch.full((2, HEADS, self.keep), -1, dtype=torch.int32, device="cuda")

    def inputs(self):
        for x in (self.k, self.v, self.q):
            x.copy_(torch.randn(x.shape, generator=self.gen, device="cuda"))

    def step(self):
        pkv.paged_kv4_append(self.k, self.v, self.slots, self.kc, self.vc)
        pkv.paged_attention_decode_kv4(self.q, self.kc, self.vc, self.tables, self.lens, SCALE, self.out, max_context_len=300)
        pkv.paged_attention_weights(self.q, self.kc, self.tables, self.lens, SCALE, self.w, weights_out=self.w_next,
                                    max_context_len=300)
        pkv.paged_kv_evict(self.w_next, self.tables, self.lens, self.keep_lens, self.new, self.kc, self.vc, self.w_out,
                           self.kept, recent=8, max_context_len=300)

    def results(self):
        # rows 301.. of the accumulators are never written: leave them out
        return [t.clone() for t in (self.out, self.w_next[:, :, :41], self.w_next[0, :, :300], self.w_out[0, :, :self.keep],
                                    self.w_out[1, :, :33], self.kept, self.kc, self.vc)]


def test_a_whole_step_replays_in_graphs_at_once():
    servers = [Server(311_310), Server(311_311)]
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


def test_eager_steps_on_two_streams_at_once():
    servers = [Server(311_320 + i) for i in range(2)]
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


def test_calls_back_to_back_share_a_workspace():
    # one buffer for every call of a stream, beside the other decode's
    s = Server(311_330)
    s.inputs()
    s.step()
    torch.cuda.synchronize()
    want = s.results()
    need = max(pkv.paged_attention_decode_kv4_workspace_bytes(2, HQ, 300, s.q.dtype, s.kc),
               pkv.paged_attention_weights_workspace_bytes(2, HQ, 300, s.kc))
    wide = [torch.randn(64, HEADS, BS, D, device="cuda").bfloat16() for _ in range(2)]
    need = max(need, pkv.paged_attention_workspace_bytes(2, HQ, 300, wide[0], partition_tokens=128))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    other = [torch.empty(2, HQ, D, device="cuda") for _ in range(2)]
    for _ in range(20):
        pkv.paged_attention_decode(s.q, *wide, s.tables, s.lens, SCALE, other[0], max_context_len=300, workspace=ws,
                                   partition_tokens=128)
        pkv.paged_attention_decode_kv4(s.q, s.kc, s.vc, s.tables, s.lens, SCALE, s.out, max_context_len=300, workspace=ws)
        pkv.paged_attention_decode(s.q, *wide, s.tables, s.lens, SCALE, other[1], max_context_len=300, workspace=ws,
                                   partition_tokens=128)
        pkv.paged_attention_weights(s.q, s.kc, s.tables, s.lens, SCALE, s.w, weights_out=s.w_next, max_context_len=300,
                                    workspace=ws)
    torch.cuda.synchronize()
    assert pkv.device_error() == 0 and torch.equal(other[0], other[1])
    assert all(torch.equal(a, b) for a, b in zip(want, s.results()))


def test_refused_tensors():
    s = Server(311_340)
    for call in (
            lambda: pkv.paged_kv4_append(s.k.transpose(0, 1), s.v, s.slots, s.kc, s.vc),          # not contiguous
            lambda: pkv.paged_kv4_append(s.k, s.v.float(), s.slots, s.kc, s.vc),                  # two dtypes
            lambda: pkv.paged_kv4_append(s.k, s.v, s.slots.int(), s.kc, s.vc),
            lambda: pkv.paged_kv4_append(s.k, s.v, s.slots.cpu(), s.kc, s.vc),
            lambda: pkv.paged_kv4_append(s.k[:, :4].contiguous(), s.v[:, :4].contiguous(), s.slots, s.kc, s.vc),
            lambda: pkv.paged_kv4_expand(s.slots, s.kc, s.vc, s.kc, s.vc),
            lambda: pkv.paged_attention_decode_kv4(s.q, s.kc, s.vc[:8], s.tables, s.lens, SCALE, s.out, max_context_len=300),
            lambda: pkv.paged_attention_decode_kv4(s.q, s.kc, s.vc, s.tables.long(), s.lens, SCALE, s.out, max_context_len=300),
            lambda: pkv.paged_attention_decode_kv4(s.q, s.kc, s.vc, s.tables, s.lens[:1], SCALE, s.out, max_context_len=300),
            lambda: pkv.paged_attention_decode_kv4(s.q, s.kc, s.vc, s.tables, s.lens, SCALE, s.out[:1], max_context_len=300),
            lambda: pkv.paged_attention_decode_kv4(s.q, s.kc, s.vc, s.tables, s.lens, SCALE, s.out.half(), max_context_len=300),
            lambda: pkv.paged_attention_decode_kv4(s.q, s.kc, s.vc, s.tables, s.lens, SCALE, s.out, max_context_len=400),
            lambda: pkv.paged_attention_weights(s.q, s.kc, s.tables, s.lens, SCALE, s.w[:, :, ::2], max_context_len=150),
            lambda: pkv.paged_attention_weights(s.q, s.kc, s.tables, s.lens, SCALE, s.w.double(), max_context_len=300),
            lambda: pkv.paged_attention_weights(s.q, s.kc, s.tables, s.lens, SCALE, s.w, weights_out=s.w_out[:1],
                                                max_context_len=300),
            lambda: pkv.paged_kv_evict(s.w, s.tables, s.lens, s.keep_lens, s.new, s.kc, s.vc, s.w, s.kept, max_context_len=300),
            lambda: pkv.paged_kv_evict(s.w, s.tables, s.lens, s.keep_lens, s.new[:, :3].contiguous(), s.kc, s.vc, s.w_out,
                                       s.kept, max_context_len=300),
            lambda: pkv.paged_kv_evict(s.w, s.tables, s.lens, s.keep_lens.long(), s.new, s.kc, s.vc, s.w_out, s.kept,
                                       max_context_len=300),
            lambda: pkv.paged_attention_decode(s.q, s.kc, s.vc, s.tables, s.lens, SCALE, s.out, max_context_len=300)):
        with pytest.raises(pkv.PagedKVError):
            call()
    assert pkv.device_error() == 0


def test_lengths_read_on_the_device_when_not_given():
    s = Server(311_350)
    s.inputs()
    s.step()
    want = s.results()
    pkv.paged_attention_decode_kv4(s.q, s.kc, s.vc, s.tables, s.lens, SCALE, s.out)
    pkv.paged_attention_weights(s.q, s.kc, s.tables, s.lens, SCALE, s.w, weights_out=s.w_next)
    pkv.paged_kv_evict(s.w_next, s.tables, s.lens, s.keep_lens, s.new, s.kc, s.vc, s.w_out, s.kept, recent=8)
    assert pkv.device_error() == 0
    assert all(torch.equal(a, b) for a, b in zip(want, s.results()))
