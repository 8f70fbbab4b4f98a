"""Several new tokens per sequence, each with its own window, against tests/window_model.py."""
import numpy as np
import pytest
import torch

import paged_kv_cache_310_gb300 as pkv
from window_model import DT, Case

pytestmark = pytest.mark.gpu


def run(c, out_dtype=None, max_len=None, **kw):
    c.cuda()
    out = torch.full(c.q.shape, 7.0, dtype=DT[out_dtype or c.dtype], device="cuda")
    return pkv.paged_attention_prefill_window(c.g_q, c.g_k, c.g_v, c.g_tables, c.g_lens, c.g_start, c.scale, out,
                                              window=c.window, sinks=c.sinks,
                                              max_context_len=c.max_len if max_len is None else max_len, **kw)


SHAPES = [  # d, bs, group, hkv
    (128, 16, 8, 2), (128, 8, 1, 1), (64, 16, 4, 3), (64, 64, 16, 1), (128, 32, 5, 1), (64, 8, 7, 2), (128, 64, 2, 1)]
VIEWS = [  # lens, new, window, sinks
    ([1, 2, 40], [1, 2, 40], 1, 0), ([300, 17], [300, 1], 1, 3), ([130, 700, 64, 65], [130, 1, 30, 65], 64, 0),
    ([600, 0, 250], [400, 0, 7], 30, 4), ([500, 333], [260, 333], 130, 70), ([900, 901, 902], [5, 8, 3], 200, 16),
    ([700], [700], 300, 1), ([520, 100], [520, 90], 10, 130), ([400], [300], 1000, 2), ([260, 261], [259, 3], 257, 65)]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("d,bs,group,hkv", SHAPES)
@pytest.mark.parametrize("lens,new,window,sinks", VIEWS, ids=lambda x: str(x) if isinstance(x, int) else f"n{len(x)}")
def test_values(lens, new, window, sinks, d, bs, group, hkv, dtype):
    c = Case(314_000 + d + bs + window, lens, window, sinks, group * hkv, hkv, d, bs, dtype, new=new)
    ref = c.reference()
    for out_dtype in (dtype, "f32"):
        c.check(run(c, out_dtype), ref)
    assert pkv.device_error() == 0


@pytest.mark.parametrize("bs", [8, 16, 32, 64])
@pytest.mark.parametrize("sinks", [0, 1, 64, 65])
def test_every_offset_of_the_window_in_its_block(sinks, bs):
    lens = list(range(200, 200 + bs + 1))
    c = Case(314_100 + bs + sinks, lens, 70, sinks, 8, 2, 64, bs, "bf16", new=[1 + i % 40 for i in range(len(lens))])
    c.check(run(c))


@pytest.mark.parametrize("window,sinks", [(1, 0), (2, 0), (5, 1), (16, 0), (63, 2), (64, 0), (65, 0)])
@pytest.mark.parametrize("group", [1, 8])
def test_windows_far_shorter_than_a_tile(group, window, sinks):
    # at one query head per KV head a pair of tiles has 256 tokens: most of its chunks lie before
    # the window of most of its rows
    c = Case(314_150, [777, 1000], window, sinks, group, 1, 128, 16, "f16", new=[777, 601])
    c.check(run(c, "f32"))


def kernel_of(c):
    """Which kernel the call's estimates choose: sequences that share the new tokens out evenly."""
    group, sms, s, t = c.hq // c.hkv, 152, len(c.lens), sum(c.new)
    tq = 8 * (16 // group)
    items = lambda span: s * -(-t // (s * span)) * c.hkv
    keys = lambda span: min(c.max_len, c.window + c.sinks + span)
    cost = dict(rows=10 + (0.65e-3 if c.d == 64 else 0.85e-3) * items(16 // group) * (keys(16 // group) // 16 + 1),
                shared=12 + 2.1 * -(-items(tq) // sms) * (keys(tq) // 128 + 1),
                pairs=10 + 1.55 * -(-items(2 * tq) // sms) * (keys(2 * tq) // 64 + 1))
    return min(cost, key=cost.get)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("d,bs,group,hkv,lens,new,window,sinks", [
    (128, 16, 8, 2, [1200, 40], [1000, 3], 600, 5), (128, 8, 1, 3, [3000], [2500], 900, 0), (64, 16, 4, 4, [2500], [1100], 700, 70),
    (64, 64, 16, 2, [900, 700], [250, 201], 500, 1), (128, 32, 5, 2, [2000, 0, 1500], [600, 0, 700], 900, 33),
    (64, 8, 7, 2, [1111], [1000], 555, 130)])
def test_tiles_shared_by_two_warpgroups(d, bs, group, hkv, lens, new, window, sinks, dtype):
    c = Case(314_160 + d + bs, lens, window, sinks, group * hkv, hkv, d, bs, dtype, new=new)
    assert kernel_of(c) == "shared"
    ref = c.reference()
    for out_dtype in (dtype, "f32"):
        c.check(run(c, out_dtype), ref)
    assert pkv.device_error() == 0


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("d,bs,group,hkv,lens,new,window,sinks", [
    (128, 16, 8, 2, [4100], [4000], 64, 5), (128, 8, 1, 12, [3000, 30], [2900, 30], 1000, 0), (64, 16, 4, 8, [2000, 1999], [1500, 1501], 300, 70),
    (64, 64, 16, 4, [1200, 700], [1000, 650], 129, 1), (128, 32, 5, 4, [2000, 0, 1500], [1900, 0, 1400], 200, 33)])
def test_pairs_of_tiles(d, bs, group, hkv, lens, new, window, sinks, dtype):
    c = Case(314_170 + d + bs, lens, window, sinks, group * hkv, hkv, d, bs, dtype, new=new)
    assert kernel_of(c) == "pairs"
    ref = c.reference()
    for out_dtype in (dtype, "f32"):
        c.check(run(c, out_dtype), ref)
    assert pkv.device_error() == 0


@pytest.mark.parametrize("seqs", [33, 200, 1024, 1025, 2500])
@pytest.mark.parametrize("new,window,hq,kernel", [(16, 100, 8, "shared"), (40, 40, 16, "pairs")])
def test_many_sequences(new, window, hq, kernel, seqs):
    # up to 32 sequences a lane knows one, up to 1,024 a lane counts up to 32, beyond nobody counts
    gen = torch.Generator().manual_seed(314_180 + seqs)
    lens = torch.randint(new, 70 + new, (seqs,), generator=gen).tolist()
    new = [max(0, new - i % 5 * (i % 3)) for i in range(seqs)]
    c = Case(314_181 + seqs, lens, window, 2, hq, 1, 64, 8, "bf16", new=new)
    assert kernel_of(c) == kernel or seqs == 33
    c.check(run(c))
    assert pkv.device_error() == 0


def test_long_contexts():
    c = Case(314_200, [20_000, 5001], 4096, 64, 16, 2, 128, 16, "bf16", new=[8, 300])
    c.check(run(c))


@pytest.mark.parametrize("d", [64, 128])
def test_a_window_of_everything_is_plain_prefill(d):
    for window, sinks in ((700, 0), (2 ** 31 - 1, 0), (701, 2 ** 31 - 1)):
        c = Case(314_210, [700, 33, 0], window, sinks, 8, 2, d, 16, "bf16", new=[300, 33, 0])
        got = run(c)
        want = torch.empty_like(got)
        pkv.paged_attention_prefill(c.g_q, c.g_k, c.g_v, c.g_tables, c.g_lens, c.g_start, c.scale, want, max_context_len=700)
        ref = c.reference()
        c.check(got, ref)
        c.check(want, ref)


def test_one_new_token_is_the_windowed_decode():
    c = Case(314_220, [700, 33, 1, 300], 150, 5, 8, 2, 128, 16, "bf16", new=[1, 1, 1, 1])
    a = run(c, "f32")
    b = torch.empty_like(a)
    pkv.paged_attention_decode_window(c.g_q, c.g_k, c.g_v, c.g_tables, c.g_lens, c.scale, b, window=150, sinks=5,
                                      max_context_len=700)
    c.check(a)
    c.check(b)


def test_no_scale_and_a_negative_one():
    for window, sinks in ((20, 0), (77, 9)):
        c = Case(314_230, [500, 90], window, sinks, 4, 2, 64, 16, "bf16", new=[400, 90])
        for c.scale in (0.0, -0.4):
            c.check(run(c))


def test_bad_blocks_and_lengths():
    c = Case(314_240, [400, 50, 300], 100, 4, 8, 2, 64, 16, "bf16", new=[30, 50, 3])
    good = run(c).clone()
    for bad in (401, 29, -1):                               # above the bound, fewer than its new tokens, negative
        c.lens[0] = bad
        out = run(c, max_len=400)
        assert pkv.device_error() == 5 and (out[:30] == 7).all() and torch.equal(out[30:], good[30:])
    c.lens[0] = 400
    keep = c.tables.clone()
    for bad in (-2, c.blocks):
        c.tables[0, 0] = bad
        run(c)
        assert pkv.device_error() == 5
        c.tables = keep.clone()
        c.tables[0, 1:16] = bad                             # tokens 16 to 255: before the first new token's window
        assert torch.equal(run(c), good) and pkv.device_error() == 0
        c.tables = keep.clone()


def test_a_key_that_is_not_a_number_reaches_who_sees_it():
    c = Case(314_250, [300], 50, 0, 2, 1, 64, 16, "f16", new=[200], spike=1.0)
    c.k[c.tables[0, 180 // 16], 0, 180 % 16, 3] = float("nan")
    out = run(c).isnan().cpu()
    p = torch.arange(100, 300)
    assert torch.equal(out.all(-1).all(-1), (p >= 180) & (p < 230)) and torch.equal(out.any(-1).any(-1), out.all(-1).all(-1))


def test_captured_and_replayed():
    c = Case(314_260, [600, 90], 200, 4, 8, 2, 128, 16, "bf16", new=[40, 90]).cuda()
    out = torch.empty_like(c.g_q)
    call = lambda: pkv.paged_attention_prefill_window(c.g_q, c.g_k, c.g_v, c.g_tables, c.g_lens, c.g_start, c.scale, out,
                                                      window=200, sinks=4, max_context_len=600)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for step in range(3):
        c.q = torch.randn(c.q.shape, generator=torch.Generator().manual_seed(step)).to(c.q.dtype)
        c.g_q.copy_(c.q)
        g.replay()
        torch.cuda.synchronize()
        c.check(out)


def test_repeats_do_not_change_a_bit():
    c = Case(314_270, [1500, 700], 300, 4, 16, 2, 128, 16, "bf16", new=[900, 33])
    outs = [run(c) for _ in range(5)]
    assert all(torch.equal(outs[0], o) for o in outs[1:])


def test_binding_refusals():
    c = Case(314_280, [100, 50], 30, 4, 8, 2, 64, 16, "f16", new=[10, 50]).cuda()
    good = dict(q=c.g_q, k_cache=c.g_k, v_cache=c.g_v, block_tables=c.g_tables, context_lens=c.g_lens, query_start=c.g_start,
                scale=1.0, out=torch.empty_like(c.g_q), window=3, max_context_len=100)
    for bad in (dict(query_start=c.g_start[:2]), dict(query_start=c.g_start.long()), dict(window=0), dict(sinks=-1),
                dict(q=c.g_q.float()), dict(k_cache=c.g_k.float(), v_cache=c.g_v.float(), q=c.g_q.float())):
        with pytest.raises(pkv.PagedKVError):
            pkv.paged_attention_prefill_window(**{**good, **bad})
    assert pkv.device_error() == 0


# Cases of the kernels that take whole tiles, full and partial ones: d, group, hkv, lens, new, window, sinks, kernel
TILES = [(128, 8, 2, [3000, 40], [2700, 3], 600, 5, "pairs"), (64, 5, 4, [2500, 800], [2400, 301], 129, 70, "pairs"),
         (128, 7, 2, [1200, 900], [600, 31], 600, 0, "shared"), (64, 16, 2, [2500], [300], 700, 33, "shared")]


def tiles(i, dtype="bf16"):
    d, group, hkv, lens, new, window, sinks, kernel = TILES[i]
    c = Case(314_290 + i, list(lens), window, sinks, group * hkv, hkv, d, 16, dtype, new=new)
    assert kernel_of(c) == kernel
    return c


@pytest.mark.parametrize("i", range(len(TILES)))
def test_tiles_with_no_scale_and_a_negative_one(i):
    c = tiles(i)
    for c.scale in (0.0, -0.4):
        c.check(run(c))
    assert pkv.device_error() == 0


@pytest.mark.parametrize("out_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("i", range(len(TILES)))
def test_rows_behind_the_last_sequence_and_of_a_bad_one_stay(i, out_dtype):
    c = tiles(i)
    ref, tokens = c.reference(), c.q.shape[0]
    c.q = torch.cat([c.q, torch.full((77, *c.q.shape[1:]), float("nan"), dtype=c.q.dtype)])
    out = run(c, out_dtype)
    c.check(out[:tokens], ref)
    assert (out[tokens:] == 7).all() and pkv.device_error() == 0
    good, first = out.clone(), c.new[0]
    c.lens[0] = first - 1                                    # fewer than its new tokens
    out = run(c, out_dtype)
    assert pkv.device_error() == 5 and (out[:first] == 7).all() and torch.equal(out[first:], good[first:])


@pytest.mark.parametrize("i", range(len(TILES)))
def test_a_query_that_is_not_a_number_stays_alone(i):
    c = tiles(i, "f16")
    good = run(c).clone()
    for tok, head, x in ((0, 1, float("nan")), (200, 0, float("inf")), (c.q.shape[0] - 1, c.hq - 1, float("nan"))):
        keep = c.q.clone()
        c.q[tok, head, 5] = x
        out = run(c)
        assert out[tok, head].isnan().all()
        out[tok, head] = good[tok, head]
        assert torch.equal(out, good)
        c.q = keep


@pytest.mark.parametrize("i", range(len(TILES)))
def test_tiles_captured_and_replayed_on_two_streams(i):
    c = tiles(i).cuda()
    outs = [torch.empty_like(c.g_q) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in outs]
    graphs = []
    run(c)
    torch.cuda.synchronize()
    for out, s in zip(outs, streams):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=s):
            pkv.paged_attention_prefill_window(c.g_q, c.g_k, c.g_v, c.g_tables, c.g_lens, c.g_start, c.scale, out,
                                               window=c.window, sinks=c.sinks, max_context_len=c.max_len)
    for step in range(2):
        c.q = torch.randn(c.q.shape, generator=torch.Generator().manual_seed(step)).to(c.q.dtype)
        c.g_q.copy_(c.q)
        torch.cuda.synchronize()
        for _ in range(3):
            for g, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        ref = c.reference()
        for out in outs:
            c.check(out, ref)
