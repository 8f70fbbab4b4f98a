"""Stream order around the rotary and the windowed calls, which let the next kernel start early and
start early themselves: a call whose output (and workspace) lies in memory that the call before was
given to read.  As tests/test_launch_order_gpu.py, with these calls as the first and as the second."""
import pytest
import torch

import paged_kv_cache_310_gb300 as pkv
from test_launch_order_gpu import Before, arena

pytestmark = pytest.mark.gpu

HEADS, HQ, BS, D = 8, 32, 16, 128


class First:
    """A call that many CTAs work on: its inputs (read to the end), its outputs, and the call."""

    def __init__(self, op, gen):
        rand = lambda *shape: torch.randn(*shape, generator=gen, device="cuda")
        perm = lambda n: torch.randperm(n, generator=gen, device="cuda")
        if op in ("rotary", "append_rotary"):
            tokens, freq = 20_000, torch.rand(D // 2, generator=gen, device="cuda", dtype=torch.float64)
            weight = rand(D).bfloat16()
            q, k, v = (rand(tokens, h, D).bfloat16() for h in (8, 4, 4))
            pos = torch.randint(0, 5000, (tokens,), generator=gen, device="cuda").to(torch.int32)
            q_out = torch.zeros_like(q)
            if op == "rotary":
                self.inputs, self.outs = [q, k, pos, freq, weight], [q_out, torch.zeros_like(k)]
                self.call = lambda x: pkv.paged_qk_rotary(x[0], x[1], x[2], *self.outs, x[3], q_weight=x[4], k_weight=x[4])
            else:
                self.inputs = [q, k, v, pos, perm(tokens), freq]
                self.outs = [q_out] + [torch.zeros(tokens // BS, 4, BS, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
                self.call = lambda x: pkv.paged_kv_append_rotary(x[0], x[1], x[2], x[3], x[4], self.outs[1], self.outs[2],
                                                                 self.outs[0], x[5])
            return
        kernel, seqs, new, n, window, dtype = {
            "decode": (None, 800, 0, 300, 100, torch.bfloat16), "decode_f32": (None, 400, 0, 300, 100, torch.float32),
            "rows": ("rows", 300, 2, 200, 20, torch.bfloat16), "shared": ("shared_tiles", 64, 20, 700, 600, torch.bfloat16),
            "pairs": ("tile_pairs", 6, 700, 800, 60, torch.bfloat16)}[op]
        width = -(-n // BS)
        pool = [rand(seqs * width, HEADS, BS, D).to(dtype) for _ in range(2)]
        tables = perm(seqs * width).to(torch.int32).view(seqs, width).contiguous()
        lens = torch.randint(max(1, n // 2, new), n + 1, (seqs,), generator=gen, device="cuda").to(torch.int32)
        q = rand(seqs * max(1, new), HQ, D).to(dtype)
        self.inputs, self.outs = [q, tables, lens], [torch.zeros_like(q)]
        kw = dict(window=window, sinks=3, max_context_len=n)
        if not new:
            self.call = lambda x: pkv.paged_attention_decode_window(x[0], *pool, x[1], x[2], 0.1, self.outs[0], **kw)
            return
        plan = pkv.paged_attention_prefill_window_plan(seqs, HQ, seqs * new, n, pool[0], window=window, sinks=3)
        assert plan["kernel"] == kernel
        self.inputs.append(torch.arange(0, seqs * new + 1, new, device="cuda").to(torch.int32))
        self.call = lambda x: pkv.paged_attention_prefill_window(x[0], *pool, x[1], x[2], x[3], 0.1, self.outs[0], **kw)


class Second:
    """A small call: bytes of its output and its workspace, and the call into given memory."""

    def __init__(self, op, gen):
        rand = lambda *shape: torch.randn(*shape, generator=gen, device="cuda")
        s, n = 8, 128
        k, v = (rand(64, 4, BS, D).half() for _ in range(2))
        tables = torch.randperm(64, generator=gen, device="cuda").to(torch.int32).view(s, 8).contiguous()
        lens = torch.tensor([100, 0, 37, 128, 0, 1, 90, 0], dtype=torch.int32, device="cuda")
        q, self.need = rand(s, 16, D).half(), 0
        if op == "decode":
            kw = dict(max_context_len=n, path=pkv.PATH_TENSOR_CORE)
            self.need = pkv.paged_attention_workspace_bytes(s, 16, n, k, path=pkv.PATH_TENSOR_CORE)
            self.call = lambda out, ws: pkv.paged_attention_decode(q, k, v, tables, lens, 0.1, out, workspace=ws, **kw)
        elif op == "decode_window":
            self.call = lambda out, ws: pkv.paged_attention_decode_window(q, k, v, tables, lens, 0.1, out, window=50, sinks=2,
                                                                          max_context_len=n)
        elif op == "prefill_window":
            q, lens = rand(s * n, 16, D).half(), torch.full((s,), n, dtype=torch.int32, device="cuda")
            start = torch.arange(0, s * n + 1, n, device="cuda").to(torch.int32)
            plan = pkv.paged_attention_prefill_window_plan(s, 16, s * n, n, k, window=50, sinks=2)
            assert plan["kernel"] == "tile_pairs"            # rows are what decode_window takes
            self.call = lambda out, ws: pkv.paged_attention_prefill_window(q, k, v, tables, lens, start, 0.1, out, window=50, sinks=2,
                                                                           max_context_len=n)
        else:
            pos, freq = torch.arange(s, device="cuda").to(torch.int32), torch.rand(D // 2, device="cuda", dtype=torch.float64)
            none = torch.empty(s, 0, D, dtype=torch.float16, device="cuda")
            self.call = lambda out, ws: pkv.paged_qk_rotary(q, none, pos, out, none, freq)
        self.shape, self.out_bytes = q.shape, q.numel() * 2


def check(first, second):
    first.call(first.inputs)
    torch.cuda.synchronize()
    want = [t.clone() for t in first.outs]
    ws = torch.empty(max(256, second.need), dtype=torch.uint8, device="cuda")
    want_out = torch.empty(second.shape, dtype=torch.float16, device="cuda")
    second.call(want_out, ws)
    torch.cuda.synchronize()
    need, n = second.need, len(first.inputs)
    for i in range(n):  # each input's end in turn under the second call's workspace and output
        order = [j for j in range(n) if j != i] + [i]
        buf, views, restore = arena([first.inputs[j] for j in order], 0, need + second.out_bytes + 4096)
        x = [views[order.index(j)] for j in range(n)]
        end = views[-1].data_ptr() - buf.data_ptr() + views[-1].numel() * views[-1].element_size()
        start = max(0, end - (need + second.out_bytes) // 2) // 256 * 256
        out_at = start + (need + 255) // 256 * 256
        out = buf[out_at:out_at + second.out_bytes].view(torch.float16).view(second.shape)
        for _ in range(6):
            restore()
            for t in first.outs:
                t.zero_()
            first.call(x)
            second.call(out, buf[start:start + max(256, need)])
            torch.cuda.synchronize()
            assert pkv.device_error() == 0
            assert torch.equal(out, want_out)
            assert all(torch.equal(got, w) for got, w in zip(first.outs, want))


@pytest.mark.parametrize("second", ["decode", "decode_window", "prefill_window", "rotary"])
@pytest.mark.parametrize("first", ["rotary", "append_rotary", "decode", "decode_f32", "rows", "shared", "pairs"])
def test_after_a_rotary_or_windowed_call(first, second):
    gen = torch.Generator(device="cuda").manual_seed(316_500)
    check(First(first, gen), Second(second, gen))


@pytest.mark.parametrize("second", ["decode_window", "prefill_window", "rotary"])
@pytest.mark.parametrize("first", ["append", "kv4_append", "expand", "weights"])
def test_a_rotary_or_windowed_call_after_the_others(first, second):
    gen = torch.Generator(device="cuda").manual_seed(316_510)
    check(Before(first, gen), Second(second, gen))
