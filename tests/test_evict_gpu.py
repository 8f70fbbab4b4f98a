"""Attention weights and eviction on the GPU against the numpy models (tests/kv4_model.py).

Weights' tolerance: a score is off by at most e = X (D + 4) 2^-23, X the largest scale * sum_d
|q_d k_d| (fp32 sums of D products, of which a truncating accumulator loses up to 2^-23 each;
f32 queries against 4-bit rows lose another 2^-21 X), which changes a softmax weight by 2 e of
itself; exp2 and the sums over n tokens, in n/64 steps of a lane and a few of lanes, warps and
partitions, add (n/64 + 64) 2^-23 of it; a sum of G weights and the accumulator 2^-22 of it."""
import random

import numpy as np
import pytest
import torch

import kv4_model as model
import paged_kv_cache_310_gb300 as pkv
from paged_kv_cache_310_gb300.block_manager import BlockManager
from test_kv4_decode_gpu import DT, fill, kv_rows, layout

pytestmark = pytest.mark.gpu


def wide_rows(gen, lens, heads, d, dtype):
    return [torch.randn(heads, n, d, generator=gen).to(dtype) for n in lens]


class Step:
    """A batch with queries, a K pool of `pool` dtype and accumulators."""

    def __init__(self, seed, lens, hq, hkv, d, bs, pool, q_dtype=None, width=None):
        gen = torch.Generator().manual_seed(seed)
        self.lens, self.scale, self.max_len = lens, d ** -0.5, max(lens + [1])
        self.tables, nb = layout(gen, lens, bs)
        if pool == "kv4":
            self.k = torch.full((nb, hkv, bs, d * 5 // 8), 255, dtype=torch.uint8)
            rows = kv_rows(gen, lens, hkv, d)
        else:
            self.k = torch.full((nb, hkv, bs, d), float("nan"), dtype=DT[pool])
            rows = wide_rows(gen, lens, hkv, d, DT[pool])
        fill(self.k, self.tables, lens, rows)
        self.q = torch.randn(len(lens), hq, d, generator=gen).to(DT[q_dtype or pool])
        width = width or self.max_len + 3
        self.before = torch.rand(len(lens), hkv, width, generator=gen)
        for s, n in enumerate(lens):
            self.before[s, :, n:] = float("nan")            # never read
        self.split = pool == "kv4" and q_dtype == "f32"

    def run(self, tracked=None, in_place=False, **kw):
        dev = [t.cuda() for t in (self.q, self.k, self.tables, torch.tensor(self.lens, dtype=torch.int32), self.before)]
        q, k, tables, lens, w = dev
        out = w if in_place else torch.full_like(w, 7.0)
        t = None if tracked is None else torch.tensor(tracked, dtype=torch.int32).cuda()
        kw.setdefault("max_context_len", self.max_len)
        got = pkv.paged_attention_weights(q, k, tables, lens, self.scale, w, weights_out=None if in_place else out,
                                          tracked_lens=t, **kw)
        assert got is out
        return out

    def check(self, tracked=None, in_place=False, **kw):
        out = self.run(tracked, in_place, **kw).cpu().double().numpy()
        assert pkv.device_error() == 0
        kv, q = model.values(self.k), self.q.double().numpy()
        after = self.before.numpy() if in_place else np.full(self.before.shape, 7.0)
        ref = model.weights(q, kv, self.tables.numpy(), self.lens, self.scale, self.before.numpy(), tracked, after)
        hkv, d = self.k.shape[1], q.shape[2]
        for s, n in enumerate(self.lens):
            rows = model.rows_of(kv, self.tables[s].numpy(), n) if n else np.zeros((hkv, 0, d))
            x = np.matmul(np.abs(q[s]).reshape(hkv, -1, d), np.abs(rows).transpose(0, 2, 1)).max(initial=0) * abs(self.scale)
            rel = 2 * x * ((d + 4) * 2.0 ** -23 + (2.0 ** -21 if self.split else 0)) + (n / 64 + 64) * 2.0 ** -23 + 2.0 ** -22
            err = np.abs(out[s, :, :n] - ref[s, :, :n])
            assert (err <= rel * ref[s, :, :n]).all(), (s, n, (err / ref[s, :, :n]).max(), rel)
            same = out[s, :, n:] == ref[s, :, n:]
            assert (same | (np.isnan(out[s, :, n:]) & np.isnan(ref[s, :, n:]))).all()


LENS = [1, 0, 15, 16, 17, 33, 64, 129, 300, 1025]


@pytest.mark.parametrize("pool,q_dtype", [("f32", None), ("f16", None), ("bf16", None), ("kv4", "f16"), ("kv4", "bf16"),
                                          ("kv4", "f32")])
@pytest.mark.parametrize("d,bs,group,hkv", [(64, 16, 1, 3), (128, 16, 8, 2), (128, 8, 5, 1), (64, 64, 16, 1), (128, 32, 11, 2),
                                            (64, 8, 4, 2)])
def test_weights_parity(pool, q_dtype, d, bs, group, hkv):
    c = Step(311_000 + d + bs + group, LENS, group * hkv, hkv, d, bs, pool, q_dtype)
    c.check()
    c.check(tracked=[max(0, n - 1) for n in LENS], in_place=True)
    c.check(tracked=[0] * len(LENS))
    c.check(tracked=[n + 5 for n in LENS])


@pytest.mark.parametrize("pool,q_dtype", [("f32", None), ("f16", None), ("bf16", None), ("kv4", "f16"), ("kv4", "bf16"),
                                          ("kv4", "f32")])
@pytest.mark.parametrize("d,bs,group,hkv", [(64, 16, 1, 3), (128, 16, 8, 2), (128, 8, 5, 1), (64, 64, 16, 1), (128, 32, 16, 1)])
def test_weights_of_contexts_that_one_cta_sees_whole(pool, q_dtype, d, bs, group, hkv):
    for lens in ([512, 0, 1, 511, 300], [7, 128, 127], [1], [129, 20], [513, 512]):   # the last: two kernels
        c = Step(311_010 + d + bs + group + len(lens), lens, group * hkv, hkv, d, bs, pool, q_dtype)
        c.check()
        c.check(tracked=[max(0, n - 3) for n in lens], in_place=True)


@pytest.mark.parametrize("pool,q_dtype", [("f32", None), ("bf16", None), ("kv4", "f16")])
def test_weights_over_several_partitions(pool, q_dtype):
    Step(311_020, [5001, 4096, 700], 8, 2, 128, 16, pool, q_dtype, width=8192).check()


def test_weights_of_a_batch_whose_partitions_are_whole_contexts():
    # so many items that a partition holds 4,096 tokens, the whole of each context
    Step(311_025, [4000] + [40] * 950, 4, 2, 64, 64, "bf16").check()


def test_weights_of_a_step_sum_to_the_group():
    c = Step(311_030, [50, 1, 0, 777], 24, 4, 64, 8, "f16")
    c.before.zero_()
    out = c.run()
    for s, n in enumerate(c.lens):
        if n:
            assert torch.allclose(out[s, :, :n].sum(-1).cpu(), torch.full((4,), 6.0), rtol=1e-5)


@pytest.mark.parametrize("pool", ["f32", "f16", "bf16"])
def test_weights_with_infinite_and_nan_rows(pool):
    # -inf scores give a token no weight; a NaN row makes its KV head's weights NaN
    lens = [40, 40]
    c = Step(311_040, lens, 2, 2, 64, 16, pool)
    c.q = c.q.abs()
    c.k[c.tables[0, 0], 0, 5] = float("-inf")
    c.k[c.tables[1, 1], 1, 3] = float("nan")
    out = c.run(tracked=[0, 0]).cpu()
    assert pkv.device_error() == 0
    assert out[0, 0, 5] == 0 and not out[0, :, :40].isnan().any()
    assert abs(float(out[0, 0, :40].sum()) - 1) < 1e-5
    assert out[1, 1, :40].isnan().all() and not out[1, 0, :40].isnan().any()


def test_weights_flag_bad_tables_and_lengths():
    c = Step(311_050, [100, 20], 8, 2, 128, 16, "bf16")
    c.tables[0, 3] = 1 << 20
    c.run()
    assert pkv.device_error() == 5
    c = Step(311_051, [100, 20], 8, 2, 128, 16, "bf16")
    out = c.run(max_context_len=99)
    assert pkv.device_error() == 5
    assert (out[0] == 7).all() and not (out[1, :, :20] == 7).any()


# ------------------------------------------------------------------------------- eviction

def weights_like(gen, shape):
    w = torch.rand(shape, generator=gen) ** 4
    kind = torch.randint(0, 8, shape, generator=gen)
    w[kind == 0] = 0.0
    w[kind == 1] = 0.25                                     # many equal ones
    w[kind == 2] = -w[kind == 2]
    odd = torch.rand(shape, generator=gen)
    w[odd < 0.02] = float("nan")
    w[(odd > 0.02) & (odd < 0.03)] = float("inf")
    w[(odd > 0.03) & (odd < 0.04)] = float("-inf")
    w[(odd > 0.04) & (odd < 0.06)] = -0.0
    return w


class Evict:
    def __init__(self, seed, lens, keep, recent, hkv, d, bs, pool, shared=False):
        gen = torch.Generator().manual_seed(seed)
        self.lens, self.keep, self.recent = lens, keep, recent
        self.max_len, self.max_keep = max(lens + [1]), max([1] + keep)
        left = [min(n, k) for n, k in zip(lens, keep)]
        both, nb = layout(gen, lens + left, bs)
        self.tables, self.new = both[:len(lens)].contiguous(), both[len(lens):].contiguous()
        if shared and lens[0] >= bs:
            self.tables[1, 0] = self.tables[0, 0]           # a shared first block
        width = d * 5 // 8 if pool == "kv4" else d
        shape = (nb, hkv, bs, width)
        if pool == "kv4":
            self.k, self.v = (torch.randint(0, 256, shape, generator=gen, dtype=torch.uint8) for _ in range(2))
        else:
            self.k, self.v = (torch.randn(shape, generator=gen).to(DT[pool]) for _ in range(2))
        self.w = weights_like(gen, (len(lens), hkv, self.max_len + 5))

    def run(self):
        dev = [t.cuda() for t in (self.w, self.tables, self.new, self.k, self.v)]
        w, tables, new, k, v = dev
        lens, keep = (torch.tensor(x, dtype=torch.int32).cuda() for x in (self.lens, self.keep))
        out = torch.full_like(w, 7.0)
        kept = torch.full((len(self.lens), w.shape[1], self.max_keep), -1, dtype=torch.int32, device="cuda")
        pkv.paged_kv_evict(w, tables, lens, keep, new, k, v, out, kept, recent=self.recent, max_context_len=self.max_len)
        return out, kept, k, v

    def check(self):
        out, kept, k, v = (t.cpu() for t in self.run())
        assert pkv.device_error() == 0
        want_k, want_v, want_out = self.k.clone(), self.v.clone(), torch.full_like(self.w, 7.0)
        want_kept = torch.full(kept.shape, -1, dtype=torch.int32)
        bs = self.k.shape[2]
        for s, n in enumerate(self.lens):
            for h in range(self.w.shape[1]):
                rows = model.kept_rows(self.w[s, h].numpy(), n, self.keep[s], self.recent)
                want_kept[s, h, :len(rows)] = torch.tensor(rows, dtype=torch.int32)
                want_out[s, h, :len(rows)] = self.w[s, h, rows]
                for i, j in enumerate(rows):
                    a, b = int(self.tables[s, j // bs]), int(self.new[s, i // bs])
                    want_k[b, h, i % bs] = self.k[a, h, j % bs]
                    want_v[b, h, i % bs] = self.v[a, h, j % bs]
        assert torch.equal(kept, want_kept)
        assert torch.equal(out.view(torch.int32), want_out.view(torch.int32))
        for a, b in ((k, want_k), (v, want_v)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("pool,d", [("f32", 64), ("f16", 128), ("bf16", 64), ("kv4", 64), ("kv4", 128)])
@pytest.mark.parametrize("bs,recent", [(8, 0), (16, 7), (64, 40), (32, 10 ** 6)])
def test_evict_parity(pool, d, bs, recent):
    lens = [1, 0, 16, 63, 64, 65, 200, 130, 5, 300]
    keep = [1, 5, 4, 64, 10, 64, 0, 129, 7, 33]
    Evict(311_100 + bs + d, lens, keep, recent, 3, d, bs, pool, shared=True).check()


@pytest.mark.parametrize("n,keep,recent", [(4097, 4096, 1), (9000, 17, 16), (20000, 10000, 100), (4096, 1, 0), (8192, 8000, 0),
                                           (49152, 700, 5), (49153, 20001, 0), (70000, 33333, 1), (8191, 8190, 8190),
                                           (32768, 16384, 16384), (400001, 5, 2), (32767, 32767, 9)])
def test_evict_long(n, keep, recent):
    # with sequences so short that most of a cluster's CTAs have no row of them
    Evict(311_120, [n, 50, 3, 0, 1], [keep, 20, 2, 1, 1], recent, 1, 64, 16, "bf16").check()


@pytest.mark.parametrize("seqs,longest,heads", [(20, 1024, 8), (9, 2048, 3), (3, 3000, 2), (1, 9000, 2), (1, 16000, 1),
                                                (4, 33000, 8), (2, 40000, 3)])
def test_evict_with_every_number_of_threads(seqs, longest, heads):
    lens = [longest - 7 * s for s in range(seqs)]
    Evict(311_125, lens, [n // 3 + 1 for n in lens], 11, heads, 64, 16, "f16").check()


@pytest.mark.parametrize("value", [0.0, 1.0, float("nan"), float("-inf"), float("inf")])
def test_evict_equal_weights_keep_the_lowest_rows(value):
    for n, keep, heads in ((5000, 1234, 2), (20000, 12345, 1)):   # one CTA or a cluster a head
        c = Evict(311_130, [n], [keep], 34, heads, 64, 8, "f16")
        c.w.fill_(value)
        c.check()


def test_evict_weights_that_share_leading_bits():
    # the threshold is found after one, two or three passes of eleven bits
    for bits in (0x3F800000, 0x3F000000, 0x00000000, 0xBF800000):
        for spread in (0x01000000, 0x00400000, 0x00200000, 0x00010000, 0x00000800, 0x00000400, 0x00000100, 0x00000002):
            c = Evict(311_135, [700], [300], 10, 2, 64, 8, "f16")
            gen = torch.Generator().manual_seed(311_136)
            k = torch.randint(0, spread, c.w.shape, generator=gen) + bits
            k = torch.where(k >= 1 << 31, k - (1 << 32), k)
            c.w = k.to(torch.int32).view(torch.float32).contiguous()
            c.check()


def test_evict_flags_bad_lengths_and_blocks():
    c = Evict(311_140, [100, 20, 60], [10, 20, 30], 5, 2, 64, 16, "f16")
    c.lens[0] = c.max_len + 1                               # longer than the bound: skipped
    c.keep[2] = -1
    out, kept, k, v = c.run()
    assert pkv.device_error() == 5
    assert (kept[0] == -1).all() and (out[0] == 7).all() and (kept[2] == -1).all()
    assert (kept[1, :, :20].cpu() == torch.arange(20, dtype=torch.int32)).all()
    c = Evict(311_141, [100, 20], [50, 20], 5, 2, 64, 16, "f16")
    c.new[0, 1] = -1
    c.tables[1, 0] = 1 << 20
    before = c.k.clone()
    _, _, k, _ = c.run()
    assert pkv.device_error() == 5
    changed = (k.cpu() != before).flatten(1).any(1).nonzero().flatten().tolist()
    assert set(changed) <= set(c.new[0, [0, 2, 3]].tolist() + c.new[1, :2].tolist())
    c = Evict(311_142, [100], [50], 5, 2, 64, 16, "f16")    # more kept than `kept` has room for
    c.max_keep = 49
    out, kept, _, _ = c.run()
    assert pkv.device_error() == 5 and (kept == -1).all()


# --------------------------------------------------------------------------- a run of them

BS, HKV, HQ, D = 16, 2, 8, 128


@pytest.mark.parametrize("pool", ["bf16", "kv4"])
def test_serving_loop_under_memory_pressure(pool):
    """Sequences grow by decode steps, their weights are accumulated, and whenever one is
    longer than a budget it is evicted down to a part of it, in a pool that could not hold
    the whole contexts; one is forked before, so eviction also meets shared blocks.  The
    histories, kept as plain arrays and shortened by the model's rule from the library's
    accumulators, are the reference of every decode."""
    rng, gen = random.Random(311_200), torch.Generator().manual_seed(311_201)
    budget, keep, recent, nb = 120, 64, 24, 60
    bm = BlockManager(nb, BS)
    if pool == "kv4":
        kc = torch.full((nb, HKV, BS, D * 5 // 8), 255, dtype=torch.uint8, device="cuda")
    else:
        kc = torch.full((nb, HKV, BS, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    vc = kc.clone()
    slots_of = {}                                           # sequence -> row of the accumulators
    weights = torch.zeros(8, HKV, 256, device="cuda")
    tracked = torch.zeros(8, dtype=torch.int32)
    hist = {}

    def held(x):
        """The float64 values that appended bf16 rows are held as."""
        x = x.double().numpy()
        return model.widen(model.quantise(x)) if pool == "kv4" else x

    append = pkv.paged_kv4_append if pool == "kv4" else pkv.paged_kv_append
    decode = pkv.paged_attention_decode_kv4 if pool == "kv4" else pkv.paged_attention_decode

    def start(s, n):
        bm.add_sequence(s, n)
        k, v = (torch.randn(n, HKV, D, generator=gen).bfloat16() for _ in range(2))
        tables, _ = bm.block_tables([s])
        slots = torch.tensor([int(tables[0, j // BS]) * BS + j % BS for j in range(n)])
        append(k.cuda(), v.cuda(), slots.cuda(), kc, vc)
        hist[s] = [held(k).transpose(1, 0, 2), held(v).transpose(1, 0, 2)]
        slots_of[s] = len(slots_of)

    for s in range(4):
        start(s, rng.randint(20, 110))
    evicted = shared_evictions = together = 0
    for step in range(60):
        if step == 10:
            bm.fork(0, 9)
            slots_of[9] = len(slots_of)
            hist[9] = [x.copy() for x in hist[0]]
            weights[slots_of[9]] = weights[slots_of[0]]
            tracked[slots_of[9]] = tracked[slots_of[0]]
        ids = sorted(hist)
        slots, pairs = bm.append(ids)
        if pairs.numel():
            pkv.paged_block_copy(pairs.cuda(), kc, vc, host_pairs=pairs)
        k, v = (torch.randn(len(ids), HKV, D, generator=gen).bfloat16() for _ in range(2))
        append(k.cuda(), v.cuda(), slots.cuda(), kc, vc)
        kh, vh = held(k), held(v)
        for i, s in enumerate(ids):
            hist[s] = [np.concatenate([hist[s][0], kh[i][:, None]], 1), np.concatenate([hist[s][1], vh[i][:, None]], 1)]
        q = torch.randn(len(ids), HQ, D, generator=gen).bfloat16()
        tables, lens = bm.block_tables(ids)
        td, ld, qd = tables.cuda(), lens.cuda(), q.cuda()
        longest = int(lens.max())
        out = torch.empty(len(ids), HQ, D, device="cuda")
        decode(qd, kc, vc, td, ld, D ** -0.5, out, max_context_len=longest)
        at = [slots_of[s] for s in ids]
        w = weights[at]
        pkv.paged_attention_weights(qd, kc, td, ld, D ** -0.5, w, tracked_lens=tracked[at].cuda(), max_context_len=longest)
        weights[at] = w
        tracked[at] = lens
        torch.cuda.synchronize()
        assert pkv.device_error() == 0
        for i, s in enumerate(ids):
            p = model.probabilities(q[i].double().numpy(), hist[s][0], D ** -0.5)
            ref = np.matmul(p, hist[s][1]).reshape(HQ, D)
            assert hist[s][0].shape[1] == int(lens[i])
            assert np.abs(out[i].cpu().double().numpy() - ref).max() <= 2e-3
        # ---- shorten what has outgrown its budget
        over = [s for s, n in zip(ids, lens.tolist()) if n > budget]
        if over:
            old, n = bm.block_tables(over)
            shared_evictions += bm.stats()["shared_blocks"] > 0
            together = max(together, len(over))
            bm.compact(over, [keep] * len(over))
            new, left = bm.block_tables(over, max_blocks=-(-keep // BS))
            at = [slots_of[s] for s in over]
            w = weights[at]
            w_out = torch.zeros_like(w)
            kept = torch.full((len(over), HKV, keep), -1, dtype=torch.int32, device="cuda")
            pkv.paged_kv_evict(w, old.cuda(), n.cuda(), torch.full((len(over),), keep, dtype=torch.int32).cuda(), new.cuda(),
                               kc, vc, w_out, kept, recent=recent, max_context_len=int(n.max()))
            weights[at] = w_out
            tracked[at] = left
            for i, s in enumerate(over):
                for h in range(HKV):
                    rows = model.kept_rows(w[i, h].cpu().numpy(), int(n[i]), keep, recent)
                    assert kept[i, h].tolist() == rows
                idx = kept[i].cpu().numpy()
                hist[s] = [np.take_along_axis(x, idx[:, :, None].astype(np.int64), 1) for x in hist[s]]
            evicted += len(over)
    assert pkv.device_error() == 0
    assert evicted >= 4 and shared_evictions >= 1 and together >= 2
