"""Stream order between calls: a decode whose workspace and output lie in memory that the call
before was given to read.  That is what a caller's arena, or an allocator that hands out the
call's freed inputs again, comes to."""
import pytest
import torch

import paged_kv_cache_310_gb300 as pkv

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def arena(inputs, first, size):
    """The inputs' bytes in one buffer, each 256-byte aligned, `size` bytes after them; copies of
    the inputs as views of it; and a function that puts their values back."""
    at, places = first, []
    for x in inputs:
        places.append(at)
        at = (at + x.numel() * x.element_size() + 255) // 256 * 256
    buf = torch.empty(at + size, dtype=torch.uint8, device="cuda")
    views = [buf[p:p + x.numel() * x.element_size()].view(x.dtype).view(x.shape) for p, x in zip(places, inputs)]

    def restore():
        for v, x in zip(views, inputs):
            v.copy_(x)

    return buf, views, restore


class Before:
    """A call that many CTAs work on: its inputs (read to the end), outputs, and the call."""

    def __init__(self, op, gen):
        rand = lambda *shape: torch.randn(*shape, generator=gen, device="cuda")
        heads, bs, d = 8, 16, 128
        row = d * 5 // 8
        if op == "expand":
            n = 8192
            pools = [torch.randint(0, 100, (n, heads, bs, row), generator=gen, device="cuda", dtype=torch.uint8) for _ in range(2)]
            self.outs = [torch.zeros(n, heads, bs, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
            self.inputs = [torch.randperm(n, generator=gen, device="cuda")[:, None].repeat(1, 2).contiguous()]
            self.call = lambda x: pkv.paged_kv4_expand(x[0], *pools, *self.outs)
        elif op in ("append", "kv4_append"):
            tokens = 30_000
            wide = op == "append"
            self.outs = [torch.zeros(tokens // bs + 1, heads, bs, d if wide else row,
                                     dtype=torch.bfloat16 if wide else torch.uint8, device="cuda") for _ in range(2)]
            self.inputs = [rand(tokens, heads, d).bfloat16(), rand(tokens, heads, d).bfloat16(),
                           torch.randperm(tokens, generator=gen, device="cuda")]
            fn = pkv.paged_kv_append if wide else pkv.paged_kv4_append
            self.call = lambda x: fn(*x, *self.outs)
        else:
            seqs, n = 2000, 60
            pool = torch.randint(0, 100, (seqs * 4, heads, bs, row), generator=gen, device="cuda", dtype=torch.uint8)
            tables = torch.randperm(seqs * 4, generator=gen, device="cuda").to(torch.int32).view(seqs, 4).contiguous()
            lens = torch.randint(1, n, (seqs,), generator=gen, device="cuda").to(torch.int32)
            before = torch.rand(seqs, heads, n, generator=gen, device="cuda")
            self.outs = [torch.zeros_like(before)]
            self.inputs = [rand(seqs, 4 * heads, d).half(), before, tables, lens]
            self.call = lambda x: pkv.paged_attention_weights(x[0], pool, x[2], x[3], 0.1, x[1], weights_out=self.outs[0],
                                                              max_context_len=n)


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("op", ["append", "kv4_append", "expand", "weights"])
def test_a_decode_in_memory_that_the_call_before_reads(op, dtype):
    gen = torch.Generator(device="cuda").manual_seed(311_400)
    b = Before(op, gen)
    lens_host = [100, 0, 37, 128, 0, 1, 90, 0]
    heads, hq, bs, d, s = 4, 16, 16, 128, len(lens_host)
    k, v = (torch.randn(64, heads, bs, d, generator=gen, device="cuda").to(DT[dtype]) for _ in range(2))
    tables = torch.randperm(64, generator=gen, device="cuda").to(torch.int32).view(s, 8).contiguous()
    lens = torch.tensor(lens_host, dtype=torch.int32, device="cuda")
    q = torch.randn(s, hq, d, generator=gen, device="cuda").to(DT[dtype])
    kw = dict(max_context_len=128, path=pkv.PATH_TENSOR_CORE)
    need = pkv.paged_attention_workspace_bytes(s, hq, 128, k, path=pkv.PATH_TENSOR_CORE)

    # the results of both in memory of their own
    b.call(b.inputs)
    torch.cuda.synchronize()
    want = [t.clone() for t in b.outs]
    want_out = torch.empty_like(q)
    pkv.paged_attention_decode(q, k, v, tables, lens, d ** -0.5, want_out, workspace=torch.empty(need, dtype=torch.uint8,
                                                                                                device="cuda"), **kw)
    torch.cuda.synchronize()
    # each input's end in turn under the decode's output (its empty contexts are written first of
    # all) and then the workspace, whose list and counters are
    out_bytes = q.numel() * q.element_size()
    for i in range(len(b.inputs)):
        order = [x for j, x in enumerate(b.inputs) if j != i] + [b.inputs[i]]
        buf, views, restore = arena(order, 0, need + out_bytes + 4096)
        x = [views[sum(1 for m in range(len(b.inputs)) if m != i and m < j)] if j != i else views[-1] for j in range(len(b.inputs))]
        end = views[-1].data_ptr() - buf.data_ptr() + views[-1].numel() * views[-1].element_size()
        for ws_first in (False, True):
            start = max(0, end - (need + out_bytes) // 2) // 256 * 256
            ws_at = start if ws_first else start + (out_bytes + 255) // 256 * 256
            out_at = start + (need + 255) // 256 * 256 if ws_first else start
            ws = buf[ws_at:ws_at + need]
            out = buf[out_at:out_at + out_bytes].view(q.dtype).view(q.shape)
            for _ in range(8):
                restore()
                for t in b.outs:
                    t.zero_()
                b.call(x)
                pkv.paged_attention_decode(q, k, v, tables, lens, d ** -0.5, out, workspace=ws, **kw)
                torch.cuda.synchronize()
                assert pkv.device_error() == 0
                assert torch.equal(out, want_out)
                assert all(torch.equal(got, w) for got, w in zip(b.outs, want))
