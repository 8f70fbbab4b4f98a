"""Single-token attention over 4-bit pools against float64 attention over the values the rows
stand for (tests/kv4_model.py).  Rows that no sequence owns hold 0xFF bytes -- (step, lo) =
NaN -- so that any use of one poisons the result.

Tolerance (f32 output): with X = the largest scale * sum_d |q_d k_d| of the case, fp32 sums of
D products are off by at most (D + 4) 2^-23 X (accumulators may truncate, so a step counts
2^-23), q's second fp16 part leaves 2^-21 X, and a score error e moves the weights' sum of
absolute changes by at most 2 e.  Weights in two fp16 parts, exp2 and the sums of a warp's
n/64 tiles, of lanes, warps and CTAs' shares add (n/16 + 64) 2^-23.  All of it times max |V|.
A 16-bit output adds half a step of the value: 2^-8 (bf16) or 2^-11 (f16) of it; for bf16
outputs a weight has one fp16 part, off by up to 2^-12 of itself, together 2^-12 max |V|."""
import numpy as np
import pytest
import torch

import kv4_model as model
import paged_kv_cache_310_gb300 as pkv

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF_STEP = {"f32": 0.0, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def layout(gen, lens, bs, extra=3):
    """(tables [S, width] padded with -1, number of blocks) over a shuffled pool."""
    need = [-(-n // bs) for n in lens]
    nb = sum(need) + extra
    perm = torch.randperm(nb, generator=gen).tolist()
    tables = torch.full((len(lens), max(need + [1])), -1, dtype=torch.int32)
    for s, c in enumerate(need):
        tables[s, :c] = torch.tensor([perm.pop() for _ in range(c)], dtype=torch.int32)
    return tables, nb


def fill(pool, tables, lens, rows):
    """rows[s]: [heads, n, bytes] written through the tables."""
    bs = pool.shape[2]
    for s, n in enumerate(lens):
        for j in range(n):
            pool[tables[s, j // bs], :, j % bs] = rows[s][:, j]


def kv_rows(gen, lens, heads, d, bias=0.5):
    mean = bias * torch.randn(heads, 1, d, generator=gen)
    return [torch.from_numpy(model.quantise((torch.randn(heads, n, d, generator=gen) + mean).double().numpy()))
            for n in lens]


class Case:
    def __init__(self, seed, lens, hq, hkv, d, bs, q_dtype, k_rows=None, q=None):
        gen = torch.Generator().manual_seed(seed)
        self.lens, self.scale = lens, d ** -0.5
        self.tables, nb = layout(gen, lens, bs)
        self.k = torch.full((nb, hkv, bs, d * 5 // 8), 255, dtype=torch.uint8)
        self.v = self.k.clone()
        fill(self.k, self.tables, lens, k_rows or kv_rows(gen, lens, hkv, d))
        fill(self.v, self.tables, lens, kv_rows(gen, lens, hkv, d))
        self.q = (torch.randn(len(lens), hq, d, generator=gen) if q is None else q).to(DT[q_dtype])
        self.max_len = max(lens + [0])

    def device(self):
        return [t.cuda() for t in (self.q, self.k, self.v, self.tables, torch.tensor(self.lens, dtype=torch.int32))]

    def reference(self):
        kv, vv = model.widen(self.k.numpy()), model.widen(self.v.numpy())
        q = self.q.double().numpy()
        ref = model.decode(q, kv, vv, self.tables.numpy(), self.lens, self.scale)
        x = vmax = 0.0
        hkv = self.k.shape[1]
        for s, n in enumerate(self.lens):
            if n:
                k = np.abs(model.rows_of(kv, self.tables[s].numpy(), n))
                x = max(x, np.matmul(np.abs(q[s]).reshape(hkv, -1, q.shape[2]), k.transpose(0, 2, 1)).max() * self.scale)
                vmax = max(vmax, np.abs(model.rows_of(vv, self.tables[s].numpy(), n)).max())
        d, n = q.shape[2], self.max_len
        tol = vmax * (2 * x * ((d + 4) * 2.0 ** -23 + 2.0 ** -21) + (n / 16 + 64) * 2.0 ** -23)
        return ref, tol, vmax

    def run(self, out_dtype="f32", **kw):
        q, k, v, tables, lens = self.device()
        out = torch.full(q.shape, 7.0, dtype=DT[out_dtype], device="cuda")
        kw.setdefault("max_context_len", self.max_len)
        pkv.paged_attention_decode_kv4(q, k, v, tables, lens, self.scale, out, **kw)
        return out

    def check(self, out_dtype="f32", **kw):
        out = self.run(out_dtype, **kw)
        assert pkv.device_error() == 0
        ref, tol, vmax = self.reference()
        tol += 2.0 ** -12 * vmax if out_dtype == "bf16" else 0
        err = np.abs(out.cpu().double().numpy() - ref)
        assert (err <= tol + HALF_STEP[out_dtype] * np.abs(ref)).all(), (err.max(), tol)
        return out


@pytest.mark.parametrize("q_dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("d,bs,group,hkv", [(64, 16, 1, 4), (128, 16, 1, 3), (128, 8, 4, 2), (64, 8, 3, 5), (128, 32, 8, 2),
                                            (64, 64, 7, 1), (128, 64, 5, 3), (64, 32, 8, 2), (128, 16, 16, 1),
                                            (64, 16, 9, 2), (128, 16, 2, 2)])
def test_parity(q_dtype, d, bs, group, hkv):
    lens = [1, 0, 15, 16, 17, 33, 64, 127, 129, 300, 2, 8]
    c = Case(310_800 + d + bs + group, lens, group * hkv, hkv, d, bs, q_dtype)
    out = c.check("f32")
    c.check(q_dtype)
    assert (out[1] == 0).all()


@pytest.mark.parametrize("lens,hq,hkv,d,bs", [([4097, 1, 5000], 8, 2, 128, 16), ([9001], 4, 1, 64, 8),
                                              ([70001], 16, 1, 128, 16), ([30011, 9000, 17], 2, 1, 64, 64),
                                              ([20000, 5], 5, 1, 128, 32),
                                              ([2049, 2048, 2047, 511], 16, 1, 128, 64)])
def test_long_contexts(lens, hq, hkv, d, bs):
    c = Case(310_830 + len(lens), lens, hq, hkv, d, bs, "f32")
    c.check("f32")
    c.check("f32", max_context_len=c.tables.shape[1] * bs)


@pytest.mark.parametrize("lens,hkv", [([64] * 5, 3), ([128] * 3, 1), ([65, 1, 64, 127], 1), ([1], 1), ([128], 1), ([192], 1),
                                      ([64 * 9] * 4 + [0] * 200 + [63] * 70 + [1] * 60, 2), ([0] * 300 + [700], 2)])
def test_shares_that_begin_and_end_anywhere(lens, hkv):
    # a CTA's share is at least two units of 64 tokens: items that fill one, cross one, share one
    Case(310_835 + len(lens), lens, 4 * hkv, hkv, 64, 8, "f16").check("f32")


def test_more_units_than_ctas():
    # 40 sequences x 16 heads: each CTA has several whole items and two parts
    gen = torch.Generator().manual_seed(310_836)
    lens = torch.randint(1, 1500, (40,), generator=gen).tolist()
    Case(310_837, lens, 16, 16, 64, 16, "bf16").check("f32")


@pytest.mark.parametrize("group", [1, 4, 8, 16])
@pytest.mark.parametrize("d", [64, 128])
def test_running_maximum_rising(group, d):
    # keys along the query, growing with the position: the maximum rises in every tile
    n, scale = 400, d ** -0.5
    gen = torch.Generator().manual_seed(310_840)
    q = torch.randn(1, 1, d, generator=gen).repeat(1, group, 1)
    u = q[0, 0] / q[0, 0].norm()
    grow = torch.linspace(-1, 1, n)[:, None] * (60 / (q[0, 0].norm() * scale)) * u
    rows = [torch.from_numpy(model.quantise((grow + 0.05 * torch.randn(n, d, generator=gen))[None].double().numpy()))]
    c = Case(310_841, [n], group, 1, d, 16, "f32", k_rows=rows, q=q)
    c.check("f32")


def test_scaled_queries_keep_their_precision():
    # rows of q of very different size, and scales of both signs
    for size, scale in ((1e-30, 1e29), (3e4, 1e-5), (1.0, -0.1), (1.0, 0.0)):
        gen = torch.Generator().manual_seed(310_850)
        q = size * torch.randn(3, 8, 64, generator=gen)
        c = Case(310_851, [40, 3, 200], 8, 2, 64, 16, "f32", q=q)
        c.scale = scale
        c.check("f32")


def test_placement_and_repeats_do_not_change_a_bit():
    outs = []
    for seed in (310_860, 310_861):
        gen = torch.Generator().manual_seed(310_862)
        lens = [700, 33, 260]
        c = Case(310_863, lens, 16, 2, 128, 16, "bf16")
        k, v = kv_rows(gen, lens, 2, 128), kv_rows(gen, lens, 2, 128)
        c.tables, nb = layout(torch.Generator().manual_seed(seed), lens, 16)
        c.k = torch.full((nb, 2, 16, 80), 255, dtype=torch.uint8)
        c.v = c.k.clone()
        fill(c.k, c.tables, lens, k)
        fill(c.v, c.tables, lens, v)
        outs += [c.run() for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(outs[0], o) for o in outs[1:])


def test_non_finite_inputs_reach_only_what_attends_to_them():
    gen = torch.Generator().manual_seed(310_870)
    lens = [400, 400, 400]                                  # split over CTAs
    rows = kv_rows(gen, lens, 2, 64)
    rows[1][0, 7, 32:] = 255                                # K of sequence 1, KV head 0, token 7: NaN
    c = Case(310_871, lens, 4, 2, 64, 16, "f32", k_rows=rows)
    c.v[c.tables[2, 1], 1, 3, 32:36] = 255                  # V of sequence 2, KV head 1, token 19: dims 0..31
    c.q[0, 3, 5] = float("inf")                             # a query of sequence 0, KV head 1
    out = c.run().cpu()
    assert pkv.device_error() == 0
    want = torch.zeros(3, 4, 64, dtype=torch.bool)
    want[0, 3] = True
    want[1, :2] = True
    want[2, 2:, :32] = True
    assert torch.equal(out.isnan(), want)


def test_bad_tables_and_lengths_set_the_flag():
    c = Case(310_880, [100, 20], 8, 2, 128, 16, "f16")
    c.tables[0, 3] = 1 << 20
    c.run()
    assert pkv.device_error() == 5
    c.tables[0, 3] = -7
    c.run()
    assert pkv.device_error() == 5
    c = Case(310_882, [300, 20, 0], 8, 2, 128, 16, "f16")
    out = c.run(max_context_len=299)
    assert pkv.device_error() == 5
    assert (out[0] == 7).all()                              # left as it was; the other one is done
    ref, tol, _ = c.reference()
    assert (np.abs(out[1].cpu().double().numpy() - ref[1]) <= tol + 2.0 ** -11 * np.abs(ref[1])).all()


def test_empty_batch_and_all_empty_sequences():
    c = Case(310_890, [0, 0], 8, 2, 64, 16, "f16")
    assert (c.run(max_context_len=0) == 0).all()
    assert (c.run(max_context_len=500) == 0).all() if c.tables.shape[1] * 16 >= 500 else True
    q, k, v, tables, lens = c.device()
    out = torch.empty(0, 8, 64, device="cuda")
    pkv.paged_attention_decode_kv4(q[:0], k, v, tables[:0], lens[:0], 0.1, out, max_context_len=16)
    assert pkv.device_error() == 0


def test_replays_in_graphs_that_share_nothing_but_inputs():
    c = Case(310_900, [900, 1, 350], 16, 4, 128, 16, "bf16")
    q, k, v, tables, lens = c.device()
    outs = [torch.empty(q.shape, device="cuda") for _ in range(3)]

    def call(out):
        pkv.paged_attention_decode_kv4(q, k, v, tables, lens, c.scale, out, max_context_len=900)

    call(outs[2])
    torch.cuda.synchronize()
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(outs[i])
        graphs.append(g)
    gen = torch.Generator(device="cuda").manual_seed(310_901)
    for _ in range(3):
        q.copy_(torch.randn(q.shape, generator=gen, device="cuda"))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graphs[0].replay()
        with torch.cuda.stream(side):                       # both graphs at once
            graphs[1].replay()
        torch.cuda.current_stream().wait_stream(side)
        call(outs[2])
        torch.cuda.synchronize()
        assert pkv.device_error() == 0
        assert torch.equal(outs[0], outs[2]) and torch.equal(outs[1], outs[2])


def test_calls_on_two_streams_at_once():
    cases = [Case(310_910 + i, [1500 + i, 37], 8, 2, 128, 16, "f16") for i in range(2)]
    want = [c.run() for c in cases]
    torch.cuda.synchronize()
    dev = [c.device() for c in cases]
    outs = [torch.empty(d[0].shape, device="cuda") for d in dev]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                q, k, v, tables, lens = dev[i]
                pkv.paged_attention_decode_kv4(q, k, v, tables, lens, cases[i].scale, outs[i],
                                               max_context_len=cases[i].max_len)
    torch.cuda.synchronize()
    assert pkv.device_error() == 0
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
