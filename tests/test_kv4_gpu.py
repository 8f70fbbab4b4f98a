"""The 4-bit cache's data movement on the GPU: append and expand against the numpy model, bit
for bit; whole-block copies and swaps of 4-bit pools; padding, bad slots and bad ids."""
import numpy as np
import pytest
import torch

import kv4_model as model
import paged_kv_cache_310_gb300 as pkv

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def pools(gen, nb, heads, bs, d):
    """Two 4-bit pools full of arbitrary bytes (rows that a call must leave as they are)."""
    return [torch.randint(0, 256, (nb, heads, bs, d * 5 // 8), generator=gen, dtype=torch.uint8) for _ in range(2)]


def same_bytes(a, b):
    return torch.equal(a.cpu().contiguous().view(torch.uint8), b.cpu().contiguous().view(torch.uint8))


def rows_like(gen, t, heads, d, dtype):
    """Rows with everything that the rounding meets: plain groups, constant ones, offsets far
    above the spread, tiny and huge values, ties, signed zeros, non-finite ones."""
    x = torch.randn(t, heads, d, generator=gen)
    kind = torch.randint(0, 10, (t, heads, d // 32, 1), generator=gen)
    g = x.view(t, heads, d // 32, 32)
    ticks = torch.randint(0, 31, g.shape, generator=gen).float() * 0.5      # halves: ties at step 1
    ticks[..., 0], ticks[..., 1] = 0.0, 15.0
    zeros = torch.where(torch.rand(g.shape, generator=gen) < 0.5, -0.0, 0.0)
    g = torch.where(kind == 1, torch.full_like(g, 1.0) * g[..., :1], g)     # constant
    g = torch.where(kind == 2, 1000.0 + 0.01 * g, g)
    g = torch.where(kind == 3, 1e-7 * g, g)
    g = torch.where(kind == 4, 30000.0 * g, g)
    g = torch.where(kind == 5, ticks, g)
    g = torch.where(kind == 6, zeros, g)
    out = g.reshape(t, heads, d).to(dtype)
    bad = torch.rand(out.shape, generator=gen) < 0.0005
    out[bad] = torch.tensor([float("nan"), float("inf"), float("-inf")], dtype=dtype)[
        torch.randint(0, 3, (int(bad.sum()),), generator=gen)]
    return out


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("t,heads,bs,d", [(1, 1, 8, 64), (1, 8, 16, 128), (7, 3, 8, 64), (33, 5, 64, 128),
                                          (257, 8, 16, 128), (1000, 2, 32, 64)])
def test_append_matches_the_model(dtype, t, heads, bs, d):
    gen = torch.Generator().manual_seed(310_710 + t + d)
    nb = -(-t // bs) * 2 + 3
    kc, vc = pools(gen, nb, heads, bs, d)
    k, v = rows_like(gen, t, heads, d, DT[dtype]), rows_like(gen, t, heads, d, DT[dtype])
    slots = torch.randperm(nb * bs, generator=gen)[:t]
    if t > 4:
        slots[2] = -1                                    # padding
        slots[4] = -(1 << 40)
    want = []
    for x, c in ((k, kc), (v, vc)):
        w = c.clone()
        q = torch.from_numpy(model.quantise(x.double().numpy()))
        for i, s in enumerate(slots.tolist()):
            if s >= 0:
                w[s // bs, :, s % bs] = q[i]
        want.append(w)
    kd, vd = kc.cuda(), vc.cuda()
    pkv.paged_kv4_append(k.cuda(), v.cuda(), slots.cuda(), kd, vd)
    assert pkv.device_error() == 0
    assert same_bytes(kd, want[0]) and same_bytes(vd, want[1])


def test_append_bad_slot_sets_the_flag_and_is_skipped():
    gen = torch.Generator().manual_seed(310_720)
    kc, vc = pools(gen, 4, 2, 16, 128)
    k = torch.randn(3, 2, 128, generator=gen)
    kd, vd = kc.cuda(), vc.cuda()
    pkv.paged_kv4_append(k.cuda(), k.cuda(), torch.tensor([5, 64, 1 << 40]).cuda(), kd, vd)
    assert pkv.device_error() == 5
    assert pkv.device_error() == 0
    kc[0, :, 5] = torch.from_numpy(model.quantise(k[0].double().numpy()))
    assert same_bytes(kd, kc)
    pkv.paged_kv4_append(k[:0].cuda(), k[:0].cuda(), torch.zeros(0, dtype=torch.int64).cuda(), kd, vd)
    assert pkv.device_error() == 0 and same_bytes(kd, kc)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n,heads,bs,d", [(1, 1, 8, 64), (3, 5, 8, 128), (9, 4, 16, 64), (40, 8, 64, 128),
                                          (70000, 1, 8, 64)])
def test_expand_matches_the_model(dtype, n, heads, bs, d):
    gen = torch.Generator().manual_seed(310_730 + n + d)
    x = rows_like(gen, 64 * heads * bs, 1, d, torch.float32).reshape(64, heads, bs, d)
    small = torch.from_numpy(model.quantise(x.double().numpy()))
    pick = torch.randint(0, 64, (n + 2,), generator=gen)
    kc, vc = small[pick].contiguous(), small[pick.flip(0)].contiguous()
    src = torch.randperm(n + 2, generator=gen)[:n]
    dst = torch.randperm(n + 1, generator=gen)[:n]
    wide = torch.from_numpy(model.widen(small.numpy())).to(DT[dtype])   # fp16 numbers: one rounding at most
    want = torch.full((n + 1, heads, bs, d), 7.0, dtype=DT[dtype])
    wantv = want.clone()
    want[dst] = wide[pick][src]
    wantv[dst] = wide[pick.flip(0)][src]
    ko = torch.full(want.shape, 7.0, dtype=DT[dtype], device="cuda")
    vo = ko.clone()
    pkv.paged_kv4_expand(torch.stack([src, dst], 1).contiguous().cuda(), kc.cuda(), vc.cuda(), ko, vo)
    assert pkv.device_error() == 0
    for got, w in ((ko, want), (vo, wantv)):
        assert torch.equal(got.cpu().isnan(), w.isnan())
        assert torch.equal(got.cpu().nan_to_num(), w.nan_to_num())


def test_expand_bad_ids_set_the_flag_and_are_skipped():
    gen = torch.Generator().manual_seed(310_740)
    x = torch.randn(4, 2, 16, 128, generator=gen)
    kc = torch.from_numpy(model.quantise(x.double().numpy()))
    out = torch.full((3, 2, 16, 128), 7.0, device="cuda")
    vo = out.clone()
    pairs = torch.tensor([[0, 2], [4, 1], [1, 3], [-1, 0], [1, -1], [1 << 40, 0]]).cuda()
    pkv.paged_kv4_expand(pairs, kc.cuda(), kc.cuda(), out, vo)
    assert pkv.device_error() == 5
    want = torch.full((3, 2, 16, 128), 7.0)
    want[2] = torch.from_numpy(model.widen(kc[0].numpy())).float()
    assert torch.equal(out.cpu(), want) and torch.equal(vo.cpu(), want)


def test_block_copy_and_swap_of_4bit_pools():
    gen = torch.Generator().manual_seed(310_750)
    kc, vc = pools(gen, 6, 3, 8, 64)
    kd, vd = kc.cuda(), vc.cuda()
    pkv.paged_block_copy(torch.tensor([[1, 4], [0, 5]]).cuda(), kd, vd)
    kc[4], kc[5], vc[4], vc[5] = kc[1], kc[0], vc[1], vc[0]
    assert pkv.device_error() == 0 and same_bytes(kd, kc) and same_bytes(vd, vc)
    hk = torch.empty((2, 3, 8, 40), dtype=torch.uint8).pin_memory()
    hv = torch.empty_like(hk).pin_memory()
    pkv.paged_block_swap_out(torch.tensor([2, 4]).cuda(), kd, vd, hk, hv)
    torch.cuda.synchronize()
    assert torch.equal(hk, kc[[2, 4]]) and torch.equal(hv, vc[[2, 4]])
    pkv.paged_block_swap_in(torch.tensor([3, 0]).cuda(), hk, hv, kd, vd)
    kc[3], kc[0], vc[3], vc[0] = kc[2].clone(), kc[4].clone(), vc[2].clone(), vc[4].clone()
    assert pkv.device_error() == 0 and same_bytes(kd, kc) and same_bytes(vd, vc)
