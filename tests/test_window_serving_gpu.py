"""A model's windowed layer as a server runs it: prompts in chunks, then single steps, then drafted
tokens, with norms, rotation and append in one call, attention over the window, and the blocks that
the window has left behind given to whoever needs one next.  Against 64 bits, from the layer's
inputs alone."""
import numpy as np
import pytest
import torch

import paged_kv_cache_310_gb300 as pkv
import step_model as model
from window_model import DT, TOL

pytestmark = pytest.mark.gpu

HQ, HKV, D, BS = 8, 2, 64, 16
SCALE, EPS = D ** -0.5, 1e-6


class Layer:
    """Three sequences under a window, in a pool that holds little more than their windows."""

    def __init__(self, dtype, window, sinks, rotary_dim, interleaved, blocks):
        self.gen = torch.Generator().manual_seed(315_000)
        self.dtype, self.window, self.sinks, self.rotary_dim, self.interleaved = dtype, window, sinks, rotary_dim, interleaved
        self.free, self.tables = list(range(blocks)), [[] for _ in range(3)]
        self.kc, self.vc = (torch.full((blocks, HKV, BS, D), float("nan"), dtype=DT[dtype], device="cuda") for _ in range(2))
        freq, factor = pkv.rotary_frequencies(rotary_dim, scaling="parts", factor=4.0, original_len=64)
        self.factor, self.freq = factor, freq
        self.weights = [(1 + 0.2 * torch.randn(D, generator=self.gen)).to(DT[dtype]) for _ in range(2)]
        self.rows = [([], [], []) for _ in range(3)]         # each sequence's inputs so far

    def step(self, new):
        """new[s] tokens more of each sequence; outputs checked; (tables, lens, start) of the calls."""
        gen, dt = self.gen, DT[self.dtype]
        q, k, v = (torch.randn(sum(new), h, D, generator=gen).to(dt) for h in (HQ, HKV, HKV))
        starts = np.concatenate([[0], np.cumsum(new)])
        positions, slots = [], []
        for s, n in enumerate(new):
            for x, rows in zip((q, k, v), self.rows[s]):
                rows.append(x[starts[s]:starts[s + 1]].double().numpy())
            before = sum(len(r) for r in self.rows[s][0][:-1])
            for p in range(before, before + n):
                if p // BS == len(self.tables[s]):
                    self.tables[s].append(self.free.pop())
                positions.append(p)
                slots.append(self.tables[s][p // BS] * BS + p % BS)
        lens = [sum(len(r) for r in rows[0]) for rows in self.rows]
        dev = lambda x, dtype: torch.tensor(x, dtype=dtype, device="cuda")
        q_out = torch.empty_like(q, device="cuda")
        pkv.paged_kv_append_rotary(q.cuda(), k.cuda(), v.cuda(), dev(positions, torch.int32), dev(slots, torch.int64), self.kc,
                                   self.vc, q_out, self.freq.cuda(), interleaved=self.interleaved, factor=self.factor,
                                   q_weight=self.weights[0].cuda(), k_weight=self.weights[1].cuda(), eps=EPS)
        width = max(len(t) for t in self.tables)
        tables = dev([t + [-1] * (width - len(t)) for t in self.tables], torch.int32)
        out = torch.empty(q.shape, device="cuda")
        kw = dict(window=self.window, sinks=self.sinks, max_context_len=max(lens))
        if all(n == 1 for n in new):
            pkv.paged_attention_decode_window(q_out, self.kc, self.vc, tables, dev(lens, torch.int32), SCALE, out, **kw)
        else:
            pkv.paged_attention_prefill_window(q_out, self.kc, self.vc, tables, dev(lens, torch.int32),
                                               dev(starts.tolist(), torch.int32), SCALE, out, **kw)
        assert pkv.device_error() == 0
        self.check(out.double().cpu().numpy(), new, starts)
        # blocks that no later token sees go back, and get NaN until they are written again
        for s, n in enumerate(lens):
            for b, block in enumerate(self.tables[s]):
                last = (b + 1) * BS - 1
                if block >= 0 and b * BS >= self.sinks and last <= n - self.window:
                    self.kc[block], self.vc[block] = float("nan"), float("nan")
                    self.free.append(block)
                    self.tables[s][b] = -1

    def check(self, out, new, starts):
        half, tol = model.HALF_STEP[self.dtype], TOL[self.dtype]
        for s, n in enumerate(new):
            q, k, v = (np.concatenate(r) for r in self.rows[s])
            at = np.arange(len(q))
            turn = lambda x, w: model.turn(x, at, self.freq.numpy(), self.interleaved, self.factor, w.double().numpy(), EPS)[0]
            q, k = turn(q, self.weights[0]), turn(k, self.weights[1])
            for i in range(n):
                p = len(q) - n + i
                seen = model.seen(p, self.window, self.sinks)
                mine = q[p].reshape(HKV, HQ // HKV, D)
                x = np.einsum("hgd,nhd->hgn", mine, k[seen]) * SCALE
                # q and k are rounded on the way: half a step of each in every product of a score
                off = 2.1 * half * np.einsum("hgd,nhd->hgn", abs(mine), abs(k[seen])).max() * SCALE
                e = np.exp(x - x.max(-1, keepdims=True))
                ref = np.einsum("hgn,nhd->hgd", e / e.sum(-1, keepdims=True), v[seen]).reshape(HQ, D)
                far = np.abs(out[starts[s] + i] - ref).max()
                assert far <= tol + (np.exp(2 * off) - 1) * np.abs(v[seen]).max(), (s, p, far)


@pytest.mark.parametrize("dtype,window,sinks,rotary_dim,interleaved", [
    ("bf16", 50, 4, 64, False), ("f16", 33, 0, 32, True), ("bf16", 64, 17, 16, False)])
def test_prompts_steps_and_drafts(dtype, window, sinks, rotary_dim, interleaved):
    layer = Layer(dtype, window, sinks, rotary_dim, interleaved, blocks=40)
    for new in ([40, 1, 17], [70, 33, 0], [5, 64, 50]):
        layer.step(new)
    for _ in range(40):
        layer.step([1, 1, 1])
    for new in ([4, 1, 3], [2, 0, 5], [3, 3, 3]):
        layer.step(new)
    held = sum(b >= 0 for t in layer.tables for b in t)
    assert held + len(layer.free) == 40 and held <= 3 * (window // BS + 2 + -(-sinks // BS))


def test_f32_steps():
    layer = Layer("f32", 45, 3, 64, False, blocks=24)
    for _ in range(130):
        layer.step([1, 1, 1])


def test_rotated_keys_in_a_4_bit_pool():
    # 4-bit pools take keys that paged_qk_rotary has turned
    gen = torch.Generator().manual_seed(315_100)
    n = 50
    q, k, v = (torch.randn(n, h, D, generator=gen).bfloat16().cuda() for h in (HQ, HKV, HKV))
    freq, _ = pkv.rotary_frequencies(D)
    pkv.paged_qk_rotary(q, k, torch.arange(n, dtype=torch.int32, device="cuda"), q, k, freq.cuda())
    pool = [torch.zeros((4, HKV, BS, D * 5 // 8), dtype=torch.uint8, device="cuda") for _ in range(2)]
    pkv.paged_kv4_append(k, v, torch.arange(n, device="cuda"), *pool)
    wide = [torch.empty((4, HKV, BS, D), device="cuda") for _ in range(2)]
    pkv.paged_kv4_expand(torch.arange(4, device="cuda")[:, None].repeat(1, 2).contiguous(), *pool, *wide)
    out = torch.empty(1, HQ, D, device="cuda")
    tables, lens = torch.arange(4, dtype=torch.int32, device="cuda")[None], torch.tensor([n], dtype=torch.int32, device="cuda")
    pkv.paged_attention_decode_kv4(q[-1:].contiguous(), *pool, tables, lens, SCALE, out, max_context_len=n)
    ref = torch.empty_like(out)
    pkv.paged_attention_decode_window(q[-1:].float().contiguous(), *wide, tables, lens, SCALE, ref, window=n, max_context_len=n)
    assert pkv.device_error() == 0 and (out - ref).abs().max() <= 1e-4
    rows = wide[0].transpose(1, 2).reshape(-1, HKV, D)[:n]
    assert (rows - k.float()).abs().max() <= (k.float().amax() - k.float().amin()) / 15  # a step at most
