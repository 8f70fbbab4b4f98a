"""Norms and position rotation of new tokens, into buffers and into the cache, against
tests/step_model.py: what both calls compute, where they write, and what they leave."""
import numpy as np
import pytest
import torch

import paged_kv_cache_310_gb300 as pkv
import step_model as model

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


class Case:
    """New tokens of `hq` query and `hkv` KV heads at random positions, seed of their own."""

    def __init__(self, seed, tokens, hq, hkv, d, dtype, rotary_dim, interleaved=False, norm="", factor=1.0, far=200_000,
                 fused=False):
        gen = torch.Generator().manual_seed(seed)
        self.dtype, self.d, self.interleaved, self.factor, self.gen = dtype, d, interleaved, factor, gen
        rows = torch.randn(tokens, hq + 2 * hkv, d, generator=gen).to(DT[dtype])
        split = rows.cuda().split([hq, hkv, hkv], 1)
        self.q, self.k, self.v = split if fused else [x.contiguous() for x in split]
        self.positions = torch.randint(0, far, (tokens,), generator=gen, dtype=torch.int32)
        self.inv_freq = torch.from_numpy(model.frequencies(rotary_dim))
        self.qw, self.kw = ((1 + 0.3 * torch.randn(d, generator=gen)).to(DT[dtype]) if n in norm else None for n in "qk")
        self.q_out = torch.full((tokens, hq, d), 7.0, dtype=DT[dtype], device="cuda")
        self.k_out = torch.full((tokens, hkv, d), 7.0, dtype=DT[dtype], device="cuda")

    def kw_args(self):
        dev = lambda t: None if t is None else t.cuda()
        return dict(interleaved=self.interleaved, factor=self.factor, q_weight=dev(self.qw), k_weight=dev(self.kw), eps=1e-5)

    def rotate(self, q_out=None, k_out=None):
        pkv.paged_qk_rotary(self.q, self.k, self.positions.cuda(), self.q_out if q_out is None else q_out,
                            self.k_out if k_out is None else k_out, self.inv_freq.cuda(), **self.kw_args())
        return self.q_out, self.k_out

    def want(self, name):
        x, w = (self.q, self.qw) if name == "q" else (self.k, self.kw)
        num = lambda t: None if t is None else t.double().cpu().numpy()
        return model.turn(num(x), self.positions.numpy(), self.inv_freq.numpy(), self.interleaved, self.factor, num(w), 1e-5)

    def check(self, name, got):
        want, size = self.want(name)
        assert model.close(got.double().cpu().numpy(), want, size, self.dtype).all()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rotary_dim", [(64, 64), (128, 128), (128, 16), (64, 48), (128, 112), (128, 0)])
@pytest.mark.parametrize("tokens,hq,hkv,norm", [(1, 4, 1, ""), (3, 5, 5, "q"), (37, 12, 3, "k"), (401, 7, 1, "qk")])
def test_values(tokens, hq, hkv, norm, d, rotary_dim, interleaved, dtype):
    c = Case(312_000 + tokens + d + rotary_dim, tokens, hq, hkv, d, dtype, rotary_dim, interleaved, norm)
    q, k = c.rotate()
    c.check("q", q)
    c.check("k", k)
    assert pkv.device_error() == 0


@pytest.mark.parametrize("tokens", [1, 5, 303, 304, 607, 608, 1215, 1217, 2433, 20_011])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (6, 2)])
def test_tokens_shared_out_to_ctas(tokens, hq, hkv):
    # several tokens to a CTA from 608 on, the last CTA partly filled
    c = Case(312_100 + tokens, tokens, hq, hkv, 64, "bf16", 64, norm="qk")
    q, k = c.rotate()
    c.check("q", q)
    c.check("k", k)


def test_many_heads():
    c = Case(312_150, 9, 512, 256, 128, "f16", 96, norm="k")  # more rows than a CTA loads at once
    q, k = c.rotate()
    c.check("q", q)
    c.check("k", k)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_positions_from_nothing_to_the_largest(dtype):
    c = Case(312_200, 12, 4, 2, 128, dtype, 128, factor=1.25)
    c.positions = torch.tensor([0, 1, 2, 3, 4095, 65_537, 131_071, 999_999, (1 << 20) - 1, (1 << 24) + 1, 1 << 30,
                                (1 << 31) - 1], dtype=torch.int32)
    q, k = c.rotate()
    for name, got in (("q", q), ("k", k)):
        want, size = c.want(name)
        # from 2^20 on a frequency's last bits count: position * 2^-52 radians, in the model and in the call
        size = size * (1 + 2 * c.positions.numpy()[:, None, None] * 2.0 ** -52 / model.REL)
        assert model.close(got.double().cpu().numpy(), want, size, dtype).all()
    assert torch.allclose(q[0].float(), 1.25 * c.q[0].float(), rtol=2 ** -8)  # position 0: the factor alone


@pytest.mark.parametrize("interleaved", [False, True])
def test_any_frequencies(interleaved):
    c = Case(312_210, 50, 3, 3, 64, "f32", 32, interleaved, far=3000)
    c.inv_freq = torch.cat([torch.tensor([0.0, -0.7, 6.5, 100.25, -2.0 ** -40, 2 * np.pi, 1e-300]),
                            torch.rand(9, generator=c.gen, dtype=torch.float64)])
    q, k = c.rotate()
    for name, got in (("q", q), ("k", k)):
        want, size = c.want(name)
        size = size * (1 + 3000 * 100.25 * 2.0 ** -51 / model.REL)
        assert model.close(got.double().cpu().numpy(), want, size, "f32").all()


def test_what_is_not_finite_stays_in_its_row():
    c = Case(312_220, 6, 4, 2, 64, "bf16", 32, norm="q")
    c.q[1, 2, 5] = float("nan")
    c.k[3, 1, 0] = float("inf")
    c.inv_freq[3] = float("nan")
    q, k = c.rotate()
    bad = torch.zeros(6, 4, 64, dtype=torch.bool)
    bad[1, 2] = True
    bad[:, :, [3, 19]] = True
    assert torch.equal(q.isnan().cpu(), bad)
    bad = torch.zeros(6, 2, 64, dtype=torch.bool)
    bad[:, :, [3, 19]] = True
    assert torch.equal(k.isnan().cpu(), bad | k.isnan().cpu() & (torch.arange(64) % 16 == 0)[None, None])
    assert not k[3, 1, 0].isfinite() and k[2, 1, 0].isfinite() and k[3, 0, 0].isfinite()


def test_rows_of_zeros():
    c = Case(312_225, 3, 2, 1, 128, "f16", 64, norm="qk")
    c.q.zero_()
    assert (c.rotate()[0] == 0).all()


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("tokens", [1, 33, 700])
def test_views_of_a_projection_in_place(tokens, dtype):
    c = Case(312_230 + tokens, tokens, 6, 2, 64, dtype, 32, norm="qk", fused=True)
    want = {n: c.want(n) for n in "qk"}
    v = c.v.clone()
    c.rotate(q_out=c.q, k_out=c.k)
    for n, got in (("q", c.q), ("k", c.k)):
        assert model.close(got.double().cpu().numpy(), *want[n], dtype).all()
    assert torch.equal(c.v, v)


def test_outputs_that_lie_apart():
    c = Case(312_240, 41, 6, 2, 128, "bf16", 128)
    wide = torch.full((41, 12, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    c.rotate(q_out=wide[:, 1:7], k_out=wide[:, 9:11])
    c.check("q", wide[:, 1:7])
    c.check("k", wide[:, 9:11])
    assert (wide[:, [0, 7, 8, 11]] == 5).all()


def test_padding_is_left_as_it_is():
    c = Case(312_250, 40, 3, 2, 64, "f32", 64)
    c.positions[5::7] = -1
    c.positions[39] = -(1 << 31)
    live = c.positions >= 0
    q, k = c.rotate()
    assert (q[~live.cuda()] == 7).all() and (k[~live.cuda()] == 7).all()
    for n, got in (("q", q), ("k", k)):
        want, size = c.want(n)
        assert model.close(got.double().cpu().numpy(), want, size, "f32")[live.numpy()].all()


def test_queries_or_keys_alone():
    c = Case(312_260, 9, 4, 2, 64, "f16", 64)
    none = torch.empty(9, 0, 64, dtype=torch.float16, device="cuda")
    kw = dict(c.kw_args())
    pkv.paged_qk_rotary(c.q, none, c.positions.cuda(), c.q_out, none, c.inv_freq.cuda(), **kw)
    pkv.paged_qk_rotary(none, c.k, c.positions.cuda(), none, c.k_out, c.inv_freq.cuda(), **kw)
    c.check("q", c.q_out)
    c.check("k", c.k_out)


# ------------------------------------------------------------------------------ into the cache

def pools(c, blocks, bs, heads):
    gen = torch.Generator().manual_seed(312_300)
    return [torch.randn(blocks, heads, bs, c.d, generator=gen).to(DT[c.dtype]).cuda() for _ in range(2)]


def append(c, slots, kc, vc, **kw):
    return pkv.paged_kv_append_rotary(c.q, c.k, c.v, c.positions.cuda(), slots.cuda(), kc, vc, c.q_out, c.inv_freq.cuda(),
                                      **{**c.kw_args(), **kw})


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("d,rotary_dim,interleaved,norm", [(64, 64, False, "qk"), (128, 32, True, ""), (128, 128, False, "k")])
@pytest.mark.parametrize("bs,tokens,hq,hkv", [(8, 1, 4, 4), (16, 33, 6, 2), (32, 130, 8, 1), (64, 700, 5, 5)])
def test_append(bs, tokens, hq, hkv, d, rotary_dim, interleaved, norm, dtype):
    c = Case(312_310 + tokens + d, tokens, hq, hkv, d, dtype, rotary_dim, interleaved, norm, fused=tokens > 100)
    blocks = tokens // 2 + 3
    kc, vc = pools(c, blocks, bs, hkv)
    was = [kc.clone(), vc.clone()]
    slots = torch.randperm(blocks * bs, generator=c.gen)[:tokens]
    slots[3::5] = -1 - slots[3::5]                      # padding
    out = append(c, slots, kc, vc)
    live = slots >= 0
    assert pkv.device_error() == 0
    assert (out[~live.cuda()] == 7).all()
    for n, got in (("q", out), ("k", kc.transpose(1, 2).reshape(-1, hkv, d)[slots.clamp(min=0).cuda()])):
        want, size = c.want(n)
        assert model.close(got.double().cpu().numpy(), want, size, dtype)[live.numpy()].all()
    # values bit for bit; every other row of both pools as it was
    rows = lambda x: x.transpose(1, 2).reshape(-1, hkv, d).clone()
    assert torch.equal(rows(vc)[slots[live].cuda()], c.v[live.cuda()])
    for pool, old in zip((kc, vc), was):
        a, b = rows(pool), rows(old)
        a[slots[live].cuda()] = b[slots[live].cuda()]
        assert torch.equal(a, b)


def test_append_is_rotation_then_append():
    for dtype in DT:
        c = Case(312_330, 65, 8, 2, 128, dtype, 128, norm="qk")
        kc, vc = pools(c, 12, 16, 2)
        kc2, vc2 = kc.clone(), vc.clone()
        slots = torch.randperm(12 * 16, generator=c.gen)[:65]
        out = append(c, slots, kc, vc).clone()
        q, k = c.rotate()
        pkv.paged_kv_append(k, c.v, slots.cuda(), kc2, vc2)
        assert torch.equal(out, q) and torch.equal(kc, kc2) and torch.equal(vc, vc2)


def test_values_keep_their_bits():
    c = Case(312_335, 4, 2, 2, 64, "bf16", 64)
    c.v.copy_(torch.arange(0x7f00, 0x7f00 + c.v.numel(), dtype=torch.int32).to(torch.int16).view(torch.bfloat16).view(c.v.shape))
    kc, vc = pools(c, 2, 8, 2)
    append(c, torch.arange(4), kc, vc)
    assert torch.equal(vc[0, :, :4].transpose(0, 1).view(torch.int16), c.v.view(torch.int16))


def test_bad_slots_and_negative_positions():
    c = Case(312_340, 6, 4, 2, 64, "f16", 64)
    kc, vc = pools(c, 4, 8, 2)
    was = [kc.clone(), vc.clone()]
    c.positions[1] = -3
    append(c, torch.tensor([-1, 5, 32, 1 << 40, -(1 << 62), (1 << 63) - 1]), kc, vc)
    assert pkv.device_error() == 5
    assert torch.equal(kc, was[0]) and torch.equal(vc, was[1]) and (c.q_out == 7).all()
    append(c, torch.tensor([-1, 5, 31, 2, -7, 0]), kc, vc)
    assert pkv.device_error() == 0
    assert (c.q_out[[0, 1, 4]] == 7).all() and not (c.q_out[[2, 3, 5]] == 7).all(-1).any()


def test_no_queries():
    c = Case(312_345, 10, 0, 3, 128, "f32", 64, norm="k")
    kc, vc = pools(c, 3, 8, 3)
    append(c, torch.arange(10), kc, vc)
    want, size = c.want("k")
    got = kc.transpose(1, 2).reshape(-1, 3, 128)[:10].double().cpu().numpy()
    assert model.close(got, want, size, "f32").all()


def test_blocks_past_four_gigabytes():
    nb, heads, bs, d = 140_000, 8, 16, 128              # 4.6 GB a pool
    c = Case(312_350, 5, 8, heads, d, "bf16", 128)
    kc, vc = (torch.zeros(nb, heads, bs, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    slots = torch.tensor([nb * bs - 1, 0, 131_072 * 16 + 3, 70_000 * 16, 139_000 * 16 + 9])
    append(c, slots, kc, vc)
    at = slots.cuda()
    c.check("k", kc[at // bs, :, at % bs])
    assert torch.equal(vc[at // bs, :, at % bs], c.v)
    assert int((kc != 0).any(-1).any(1).sum()) == 5


def test_a_captured_step_replayed_on_another_stream():
    c = Case(312_360, 8, 8, 2, 128, "bf16", 128, norm="qk")
    kc, vc = pools(c, 8, 8, 2)
    positions, inv_freq, kw = c.positions.cuda(), c.inv_freq.cuda(), c.kw_args()
    slots = torch.randperm(64, generator=c.gen)[:8].cuda()
    call = lambda: pkv.paged_kv_append_rotary(c.q, c.k, c.v, positions, slots, kc, vc, c.q_out, inv_freq, **kw)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    other = torch.cuda.Stream()
    for step in range(3):
        gen = torch.Generator(device="cuda").manual_seed(312_361 + step)
        for x in (c.q, c.k, c.v):
            x.copy_(torch.randn(x.shape, generator=gen, device="cuda"))
        c.positions = torch.randint(0, 5000, (8,), generator=c.gen, dtype=torch.int32)
        positions.copy_(c.positions)
        torch.cuda.synchronize()
        with torch.cuda.stream(other):
            g.replay()
        other.synchronize()
        c.check("q", c.q_out)
        c.check("k", kc[slots // 8, :, slots % 8])
        assert torch.equal(vc[slots // 8, :, slots % 8], c.v)


def test_binding_refusals():
    c = Case(312_370, 4, 4, 2, 64, "f16", 64)
    kc, vc = pools(c, 4, 8, 2)
    pos, f, slots = c.positions.cuda(), c.inv_freq.cuda(), torch.arange(4).cuda()
    good = dict(q=c.q, k=c.k, v=c.v, positions=pos, slot_mapping=slots, k_cache=kc, v_cache=vc, q_out=c.q_out, inv_freq=f)
    bad = [dict(q=c.q.float()), dict(q=c.q[:3]), dict(k=c.k[:, :1]), dict(v=c.v.cpu()), dict(positions=pos.long()),
           dict(positions=pos[::2]), dict(slot_mapping=slots.int()), dict(slot_mapping=slots[:3]), dict(q_out=c.q_out[:, :3]),
           dict(inv_freq=f.float()), dict(inv_freq=f[::2]), dict(inv_freq=f[:5]), dict(q=c.q.transpose(0, 1)), dict(v_cache=vc[:3]),
           dict(q_weight=torch.ones(32, dtype=torch.float16, device="cuda")), dict(k_weight=torch.ones(64, device="cuda")),
           dict(k_cache=torch.zeros(4, 2, 8, 40, dtype=torch.uint8, device="cuda")), dict(q=c.q[..., ::2])]
    for b in bad:
        with pytest.raises(pkv.PagedKVError):
            pkv.paged_kv_append_rotary(**{**good, **b})
    with pytest.raises(pkv.PagedKVError):
        pkv.paged_qk_rotary(c.q, c.k, pos, c.q_out, c.k_out[:, :1], f)
    pkv.paged_kv_append_rotary(**good)
    empty = lambda t: t[:0]
    pkv.paged_kv_append_rotary(empty(c.q), empty(c.k), empty(c.v), empty(pos), empty(slots), kc, vc, empty(c.q_out), f)
    assert pkv.device_error() == 0
