"""Decode right behind the call that writes its context lengths: an append, which lets the next kernel
start at once, whose last token's row is the tensor of lengths, or a PyTorch kernel."""
import pytest
import torch

import paged_kv_cache_310_gb300 as pkv

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HEADS, BS, D, LONGEST = 2, 16, 128, 600


class Decode:
    def __init__(self, seqs, dtype, gen):
        width = -(-LONGEST // BS)
        self.k, self.v = (torch.randn(3 * width, HEADS, BS, D, generator=gen, device="cuda").to(DT[dtype]) for _ in range(2))
        self.tables = torch.randint(0, 3 * width, (seqs, width), generator=gen, device="cuda").to(torch.int32)
        self.q = torch.randn(seqs, 16, D, generator=gen, device="cuda").to(DT[dtype])
        need = pkv.paged_attention_workspace_bytes(seqs, 16, LONGEST, self.k, path=pkv.PATH_TENSOR_CORE)
        self.ws = torch.empty(need, dtype=torch.uint8, device="cuda")

    def __call__(self, lens):
        out = torch.full(self.q.shape, 7.0, dtype=self.q.dtype, device="cuda")
        return pkv.paged_attention_decode(self.q, self.k, self.v, self.tables, lens, D ** -0.5, out, max_context_len=LONGEST,
                                          workspace=self.ws, path=pkv.PATH_TENSOR_CORE)


def lengths(seqs, gen):
    """Lengths of very different sums, zeros among them."""
    sets = [torch.zeros(seqs), torch.full((seqs,), LONGEST), torch.randint(0, LONGEST + 1, (seqs,), generator=gen),
            torch.randint(0, 2, (seqs,), generator=gen) * LONGEST, torch.arange(seqs) % 65, torch.ones(seqs)]
    return [x.to(torch.int32).cuda() for x in sets]


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("tokens", [100, 40_000])
def test_behind_an_append_that_writes_the_lengths(tokens, dtype):
    gen = torch.Generator(device="cuda").manual_seed(316_700)
    decode, sets = Decode(64, dtype, gen), lengths(64, torch.Generator().manual_seed(1))
    want = [decode(x).clone() for x in sets]
    # a pool of f32 rows of 64 values: the last token's row of K is the 64 lengths, bit for bit
    kc, vc = (torch.zeros(tokens // 8 + 1, 1, 8, 64, device="cuda") for _ in range(2))
    rows = torch.randn(tokens, 1, 64, generator=gen, device="cuda")
    slots = torch.arange(tokens, device="cuda")
    lens = kc.view(-1, 64)[tokens - 1].view(torch.int32)
    for step in range(60):
        i, was = step * 5 % len(sets), (step * 5 + 1 + step % 3) % len(sets)
        lens.copy_(sets[was])
        rows[-1, 0].view(torch.int32).copy_(sets[i])
        torch.cuda.synchronize()
        pkv.paged_kv_append(rows, rows, slots, kc, vc)
        out = decode(lens)
        torch.cuda.synchronize()
        assert torch.equal(out, want[i]) and torch.equal(lens, sets[i])
    assert pkv.device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("seqs", [64, 1024, 1025, 2100])
def test_behind_a_kernel_that_writes_the_lengths(seqs, dtype):
    gen = torch.Generator(device="cuda").manual_seed(316_710)
    decode, sets = Decode(seqs, dtype, gen), lengths(seqs, torch.Generator().manual_seed(2))
    want = [decode(x).clone() for x in sets]
    lens = torch.empty(seqs, dtype=torch.int32, device="cuda")
    for step in range(40):
        lens.fill_(-5 if step % 2 else LONGEST + 1)             # nothing of this may be seen, or flagged
        lens.copy_(sets[step % len(sets)])
        out = decode(lens)
        torch.cuda.synchronize()
        assert torch.equal(out, want[step % len(sets)])
    assert pkv.device_error() == 0


def test_captured_and_replayed_behind_the_kernel_that_writes_them():
    gen = torch.Generator(device="cuda").manual_seed(316_720)
    decode, sets = Decode(64, "bf16", gen), lengths(64, torch.Generator().manual_seed(3))
    want = [decode(x).clone() for x in sets]
    given, lens = sets[0].clone(), sets[0].clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lens.copy_(given)
        out = decode(lens)
    for step in range(40):
        given.copy_(sets[step % len(sets)])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[step % len(sets)])
    assert pkv.device_error() == 0


@pytest.mark.parametrize("seqs", [64, 1500])
def test_lengths_out_of_bounds_are_flagged(seqs):
    gen = torch.Generator(device="cuda").manual_seed(316_730)
    decode = Decode(seqs, "bf16", gen)
    good = torch.full((seqs,), 100, dtype=torch.int32, device="cuda")
    want = decode(good).clone()
    for bad in (-1, 100_000, -(1 << 31), (1 << 31) - 1):
        lens = good.clone()
        lens[seqs - 3] = bad
        out = decode(lens)
        assert pkv.device_error() == 5
        assert (out[seqs - 3] == 7).all() and torch.equal(out[:seqs - 3], want[:seqs - 3]) and torch.equal(out[seqs - 2:], want[seqs - 2:])
