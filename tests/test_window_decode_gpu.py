"""Single-token attention over a sliding window and the first tokens, against
tests/window_model.py: every row that is not attended to holds NaN, released blocks are -1."""
import numpy as np
import pytest
import torch

import paged_kv_cache_310_gb300 as pkv
from window_model import DT, Case

pytestmark = pytest.mark.gpu


def run(c, out_dtype=None, max_len=None, **kw):
    c.cuda()
    out = torch.full(c.q.shape, 7.0, dtype=DT[out_dtype or c.dtype], device="cuda")
    return pkv.paged_attention_decode_window(c.g_q, c.g_k, c.g_v, c.g_tables, c.g_lens, c.scale, out, window=c.window,
                                             sinks=c.sinks, max_context_len=c.max_len if max_len is None else max_len, **kw)


SHAPES = [  # d, bs, group, hkv
    (128, 16, 1, 2), (128, 8, 8, 2), (128, 32, 4, 1), (64, 16, 8, 2), (64, 64, 2, 3), (128, 64, 6, 1), (64, 8, 1, 4), (64, 32, 7, 1)]
WIDE = [(128, 16, 16, 1), (64, 8, 12, 2), (64, 64, 16, 3), (128, 32, 9, 2)]
VIEWS = [  # lens, window, sinks
    ([0, 1, 2, 3, 17], 1, 0), ([1, 2, 40, 300], 1, 1), ([5, 64, 65, 127, 128, 129, 130, 1000], 64, 0),
    ([100, 700, 131, 260], 128, 5), ([50, 0, 333, 1001], 129, 16), ([90, 91, 92, 93, 94, 95, 96, 97, 500], 30, 60),
    ([2500, 1200, 64, 900], 1000, 33), ([700, 650, 300], 200, 200), ([3000, 2999], 7, 130), ([640, 641], 640, 3)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("d,bs,group,hkv", SHAPES)
@pytest.mark.parametrize("lens,window,sinks", VIEWS, ids=lambda x: str(x) if isinstance(x, int) else f"n{len(x)}")
def test_values(lens, window, sinks, d, bs, group, hkv, dtype):
    c = Case(313_000 + d + bs + window, lens, window, sinks, group * hkv, hkv, d, bs, dtype)
    ref = c.reference()
    for out_dtype in {dtype, "f32"}:
        c.check(run(c, out_dtype), ref)
    assert pkv.device_error() == 0


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("d,bs,group,hkv", WIDE)
@pytest.mark.parametrize("lens,window,sinks", VIEWS[3:7], ids=lambda x: str(x) if isinstance(x, int) else f"n{len(x)}")
def test_groups_above_eight(lens, window, sinks, d, bs, group, hkv, dtype):
    c = Case(313_050 + d + bs + window, lens, window, sinks, group * hkv, hkv, d, bs, dtype)
    c.check(run(c))
    assert pkv.device_error() == 0


@pytest.mark.parametrize("bs", [8, 16, 32, 64])
@pytest.mark.parametrize("sinks", [0, 1, 63, 64, 65])
def test_every_offset_of_the_window_in_its_block(sinks, bs):
    # one sequence for each length: the window's oldest token at every row of its block
    for dtype, window in (("bf16", 70), ("f32", 130)):
        lens = list(range(200, 200 + 2 * bs + 1))
        c = Case(313_100 + bs + sinks, lens, window, sinks, 4, 2, 64, bs, dtype)
        c.check(run(c))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("lens,window,sinks", [([9000, 5000, 20_000], 4096, 64), ([8000], 7000, 0), ([4000, 12_345], 2049, 515)])
def test_windows_of_several_partitions(lens, window, sinks, dtype):
    c = Case(313_150, lens, window, sinks, 8, 2, 128, 16, dtype)
    c.check(run(c))
    c = Case(313_151, lens, window, sinks, 4, 1, 64, 32, dtype)
    c.check(run(c, "f32"))


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("d,hkv", [(128, 2), (64, 2), (64, 1)])
def test_a_window_of_everything_is_plain_decode(d, hkv, dtype):
    path = pkv.PATH_CUDA_CORE if dtype == "f32" else pkv.PATH_TENSOR_CORE
    for window, sinks in ((900, 0), (901, 5), (1 << 30, 0), (2 ** 31 - 1, 2 ** 31 - 1), (1, 900), (300, 600)):
        c = Case(313_200, [900, 1, 0, 350], window, sinks, 4 * hkv, hkv, d, 16, dtype)
        got = run(c)
        want = torch.empty_like(got)
        pkv.paged_attention_decode(c.g_q, c.g_k, c.g_v, c.g_tables, c.g_lens, c.scale, want, max_context_len=900, path=path)
        ref = c.reference()
        c.check(got, ref)
        c.check(want, ref)


def test_empty_and_single_tokens():
    for dtype in DT:
        c = Case(313_210, [0, 0, 1, 0], 5, 3, 8, 2, 64, 8, dtype, spike=1.0)
        out = run(c)
        assert (out[[0, 1, 3]] == 0).all()
        c.check(out)
        c = Case(313_211, [0, 0], 5, 3, 8, 2, 64, 8, dtype)
        assert (run(c) == 0).all() and (run(c, max_len=8) == 0).all()


def test_bad_blocks_and_lengths():
    for dtype in ("f32", "bf16"):
        c = Case(313_220, [400, 50, 300], 100, 4, 8, 2, 64, 16, dtype)
        good = run(c).clone()
        # longer sequences than the bound, and negative lengths: flagged, their rows as they were
        out = run(c, max_len=300)
        assert pkv.device_error() == 5 and (out[0] == 7).all() and torch.equal(out[1:], good[1:])
        for bad in (401, -1, -(1 << 31), 2 ** 31 - 1):
            c.lens[2] = bad
            out = run(c, max_len=400)
            assert pkv.device_error() == 5 and (out[2] == 7).all() and torch.equal(out[:2], good[:2])
        c.lens[2] = 300
        # an id out of range in a block that counts; outside the view any entry will do
        keep = c.tables.clone()
        for bad in (-2, c.blocks, 2 ** 31 - 1):
            c.tables[0, 0] = bad                            # holds the sinks
            run(c)
            assert pkv.device_error() == 5
            c.tables = keep.clone()
            c.tables[0, 2:17] = bad                         # tokens 32 to 271: neither sink nor window
            assert torch.equal(run(c), good) and pkv.device_error() == 0
            c.tables = keep.clone()


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_scores_of_equal_size_and_no_scale(dtype):
    c = Case(313_230, [500, 30], 77, 9, 4, 2, 64, 16, dtype)
    c.scale = 0.0                                           # the mean of what is seen
    c.check(run(c))
    c.scale = -0.5
    c.check(run(c))


def test_a_maximum_that_rises_with_every_chunk():
    for dtype in ("bf16", "f32"):
        n, d = 2000, 128
        c = Case(313_240, [n], 1500, 4, 4, 1, d, 16, dtype)
        u = c.q[0, 0].float() / c.q[0, 0].float().norm()
        for j in c.seen[0]:
            c.k[c.tables[0, j // 16], 0, j % 16] = ((j - 1000) / 1000 * 50 * d ** 0.5 / c.q[0, 0].float().norm() * u).to(DT[dtype])
        c.q[:] = c.q[0, 0]
        ref = c.reference()
        # scores to 72 in log2 units: ten times the size that the tolerance is made for
        got = run(c).double().cpu().numpy()
        assert (np.abs(got - ref) <= 10 * (1e-5 if dtype == "f32" else 2e-3) * 20 + 2.0 ** -8 * np.abs(ref)).all()


@pytest.mark.parametrize("dtype", ["f16", "f32"])
def test_not_finite_where_it_is_seen(dtype):
    c = Case(313_250, [400, 400, 400], 100, 4, 4, 2, 64, 16, dtype)
    c.k[c.tables[0, 350 // 16], 0, 350 % 16, 3] = float("nan")
    c.v[c.tables[1, 0], 1, 2, 5] = float("nan")
    c.q[2, 1, 0] = float("inf")
    out = run(c).isnan().cpu()
    want = torch.zeros(3, 4, 64, dtype=torch.bool)
    want[0, :2] = True
    want[1, 2:, 5] = True
    want[2, 1] = True
    assert torch.equal(out, want)


def test_far_blocks_and_long_tables():
    nb, heads, bs, d = 140_000, 8, 16, 128                  # 4.6 GB a pool
    n, window, sinks = 1_000_003, 50, 3
    c = Case(313_260, [n, 40], window, sinks, 16, heads, d, bs, "bf16")
    far = torch.randperm(nb, generator=torch.Generator().manual_seed(1))[:c.blocks]
    far[:3] = torch.tensor([nb - 1, nb - 2, 131_073])
    k, v = (torch.full((nb, heads, bs, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k[far.cuda()], v[far.cuda()] = c.k.cuda(), c.v.cuda()
    ref = c.reference()
    tables = torch.where(c.tables < 0, c.tables, far.to(torch.int32)[c.tables.clamp(min=0).long()]).cuda()
    out = torch.empty(c.q.shape, dtype=torch.bfloat16, device="cuda")
    pkv.paged_attention_decode_window(c.q.cuda(), k, v, tables, torch.tensor(c.lens, dtype=torch.int32).cuda(), c.scale, out,
                                      window=window, sinks=sinks, max_context_len=n)
    assert pkv.device_error() == 0
    c.check(out, ref)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_sequences(dtype):
    gen = torch.Generator().manual_seed(313_270)
    lens = torch.randint(0, 60, (3000,), generator=gen).tolist()
    c = Case(313_271, lens, 9, 2, 2, 1, 64, 8, dtype)
    c.check(run(c))


def test_captured_on_two_streams_and_replayed():
    for dtype in ("bf16", "f32"):
        cases = [Case(313_280 + i, [1500, 20, 700 + i], 600, 4, 8, 2, 128, 16, dtype).cuda() for i in range(2)]
        outs = [torch.empty_like(c.g_q) for c in cases]

        def call(i):
            c = cases[i]
            pkv.paged_attention_decode_window(c.g_q, c.g_k, c.g_v, c.g_tables, c.g_lens, c.scale, outs[i], window=600, sinks=4,
                                              max_context_len=1501)

        graphs = []
        for i in range(2):
            call(i)
            torch.cuda.synchronize()
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1]):
                call(i)
        streams = [torch.cuda.Stream() for _ in range(2)]
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for _ in range(20):
            for g, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        for c, o in zip(cases, outs):
            c.check(o)
        # another length, below the bound that the capture had
        cases[0].g_lens[1] = 0
        graphs[0].replay()
        torch.cuda.synchronize()
        assert (outs[0][1] == 0).all() and pkv.device_error() == 0


def test_repeats_and_placement_do_not_change_a_bit():
    for dtype in DT:
        outs = []
        for order in (0, 1):
            c = Case(313_290, [5000, 33, 900], 2000, 20, 8, 2, 128, 16, dtype)
            if order:
                perm = torch.randperm(c.blocks, generator=torch.Generator().manual_seed(2))
                moved = torch.empty_like(perm)
                moved[perm] = torch.arange(c.blocks)
                c.k, c.v = c.k[perm].contiguous(), c.v[perm].contiguous()
                c.tables = torch.where(c.tables < 0, c.tables, moved[c.tables.clamp(min=0).long()].to(torch.int32))
            outs += [run(c) for _ in range(4)]
        assert all(torch.equal(outs[0], o) for o in outs[1:])


def test_binding():
    c = Case(313_300, [900, 100], 300, 4, 8, 2, 64, 16, "f16")
    want = run(c)
    assert torch.equal(pkv.paged_attention_decode_window(c.g_q, c.g_k, c.g_v, c.g_tables, c.g_lens, c.scale,
                                                         torch.empty_like(c.g_q), window=300, sinks=4), want)
    good = dict(q=c.g_q, k_cache=c.g_k, v_cache=c.g_v, block_tables=c.g_tables, context_lens=c.g_lens, scale=1.0,
                out=torch.empty_like(c.g_q), window=3, max_context_len=900)
    for bad in (dict(q=c.g_q.float()), dict(q=c.g_q[:1]), dict(out=good["out"].bfloat16()), dict(v_cache=c.g_v[:2]), dict(window=0),
                dict(sinks=-1), dict(block_tables=c.g_tables.long()), dict(context_lens=c.g_lens[:1]), dict(q=c.q),
                dict(q=c.g_q.transpose(1, 2)), dict(block_tables=c.g_tables[:, :5].contiguous())):
        with pytest.raises(pkv.PagedKVError):
            pkv.paged_attention_decode_window(**{**good, **bad})
    assert pkv.device_error() == 0
