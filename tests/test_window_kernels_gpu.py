"""Each kernel of a windowed prefill on calls that the library says it takes it for, against
tests/window_model.py."""
import pytest
import torch

import paged_kv_cache_310_gb300 as pkv
from test_window_prefill_gpu import run
from window_model import Case

pytestmark = pytest.mark.gpu


def taken(c):
    return pkv.paged_attention_prefill_window_plan(len(c.lens), c.hq, c.q.shape[0], c.max_len, c.k, window=c.window, sinks=c.sinks)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("d,bs,group,hkv,lens,new,window,sinks,ctas", [
    (128, 16, 8, 2, [5000], [4], 4096, 4, 8), (128, 8, 5, 1, [900, 40, 0, 333], [7, 40, 0, 9], 200, 33, 4), (64, 64, 16, 2, [700, 300], [5, 1], 500, 1, 8),
    (64, 16, 3, 4, [400, 90, 91, 92], [33, 1, 30, 2], 64, 70, 4), (64, 32, 1, 8, [300, 301], [17, 2], 100, 0, 2),
    (128, 64, 12, 3, [1200, 1, 2], [3, 1, 2], 900, 130, 8), (128, 16, 8, 8, [300 + i for i in range(60)], [1 + i % 3 for i in range(60)], 50, 3, 1)])
def test_rows(d, bs, group, hkv, lens, new, window, sinks, ctas, dtype):
    c = Case(316_200 + d + bs, lens, window, sinks, group * hkv, hkv, d, bs, dtype, new=new)
    assert taken(c) == dict(kernel="rows", tokens_per_item=16 // group, ctas_per_item=ctas)
    ref = c.reference()
    for out_dtype in (dtype, "f32"):
        c.check(run(c, out_dtype), ref)
    assert pkv.device_error() == 0


@pytest.mark.parametrize("seqs", [33, 64, 100])
@pytest.mark.parametrize("each,window,hq,hkv,kernel", [(16, 1000, 32, 4, "shared_tiles"), (40, 40, 64, 4, "tile_pairs")])
def test_a_lane_that_counts_several_sequences(each, window, hq, hkv, kernel, seqs):
    gen = torch.Generator().manual_seed(316_210 + seqs)
    lens = torch.randint(window, 70 + window, (seqs,), generator=gen).tolist()
    new = [max(0, each - i % 5 * (i % 3)) for i in range(seqs)]
    c = Case(316_211 + seqs, lens, window, 2, hq, hkv, 64, 8, "bf16", new=new)
    assert taken(c)["kernel"] == kernel
    c.check(run(c))
    assert pkv.device_error() == 0


def test_rows_repeat_and_replay():
    c = Case(316_220, [900, 33, 500], 300, 4, 16, 2, 128, 16, "bf16", new=[5, 9, 1]).cuda()
    assert taken(c)["kernel"] == "rows"
    outs = [run(c) for _ in range(4)]
    assert all(torch.equal(outs[0], o) for o in outs[1:])
    out = torch.empty_like(c.g_q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkv.paged_attention_prefill_window(c.g_q, c.g_k, c.g_v, c.g_tables, c.g_lens, c.g_start, c.scale, out, window=300, sinks=4,
                                           max_context_len=900)
    for step in range(3):
        c.q = torch.randn(c.q.shape, generator=torch.Generator().manual_seed(step)).to(c.q.dtype)
        c.g_q.copy_(c.q)
        g.replay()
        torch.cuda.synchronize()
        c.check(out)
    assert pkv.device_error() == 0


def test_rows_of_no_sequence_and_of_a_bad_one_stay():
    c = Case(316_230, [400, 50, 300], 100, 4, 8, 2, 64, 16, "bf16", new=[30, 5, 3])
    assert taken(c)["kernel"] == "rows"
    ref, tokens = c.reference(), c.q.shape[0]
    c.q = torch.cat([c.q, torch.full((9, *c.q.shape[1:]), float("nan"), dtype=c.q.dtype)])
    good = run(c)
    c.check(good[:tokens], ref)
    assert (good[tokens:] == 7).all() and pkv.device_error() == 0
    for s, bad in ((0, 29), (1, 4), (2, -1), (2, 401)):
        keep = c.lens[s]
        c.lens[s] = bad
        out = run(c, max_len=400)
        a, b = int(c.start[s]), int(c.start[s + 1])
        assert pkv.device_error() == 5 and (out[a:b] == 7).all()
        assert torch.equal(out[:a], good[:a]) and torch.equal(out[b:], good[b:])
        c.lens[s] = keep
