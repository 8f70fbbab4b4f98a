"""16-bit outputs of attention over 4-bit pools: the float64 result, known to within the kernel's
own 32-bit error, rounded once.

Each query has one element that is not 0, so a score is one product, which two fp16 numbers give
exactly.  With X the largest |score|: the scale is rounded twice (the factor, its product with
log2 e) and the scaled score once, 4 * 2^-24 X with the maximum's subtraction, and a score error
e changes a mean of values by at most 2 e max |V|: below 16 X 2^-23.  Weights in two fp16 parts
(2^-22 of a weight, and 2^-31 of the largest where a weight is small), exp2 (2^-22), the sums of n
values by steps of 16 (2^-23 each, accumulators may truncate), of lanes, warps and CTAs, and the
division: below (n / 16 + 64) 2^-23 max |V|.  So the output is the rounding of some number within
T = max |V| (16 X + n / 16 + 65) 2^-23 of the float64 result: the rounding being monotonic, it
lies between those of the result less T and plus T (65 and not 64: going through fp32 on the way
to 16 bits moves a bound by 2^-24 of it)."""
import numpy as np
import pytest
import torch

import kv4_model as model
import paged_kv_cache_310_gb300 as pkv
from test_kv4_decode_gpu import DT, Case

pytestmark = pytest.mark.gpu


def one_element_queries(seed, seqs, hq, d):
    gen = torch.Generator().manual_seed(seed)
    q = torch.zeros(seqs, hq, d)
    at = torch.randint(0, d, (seqs, hq, 1), generator=gen)
    return q.scatter_(2, at, 4 * torch.rand(seqs, hq, 1, generator=gen) - 2)


def check(c, dtype, out):
    kv, vv = model.widen(c.k.numpy()), model.widen(c.v.numpy())
    q = c.q.double().numpy()
    ref = torch.from_numpy(model.decode(q, kv, vv, c.tables.numpy(), c.lens, c.scale))
    own = [np.abs(model.rows_of(x, c.tables[s].numpy(), n)).max() for s, n in enumerate(c.lens) if n for x in (kv, vv)]
    x, vmax, n = np.abs(q).max() * max(own[0::2]) * c.scale, max(own[1::2]), max(c.lens)
    tol = vmax * (16 * x + n / 16 + 65) * 2.0 ** -23
    low, high = (ref - tol).float().to(DT[dtype]), (ref + tol).float().to(DT[dtype])
    wrong = ~((low <= out) & (out <= high))
    assert not wrong.any(), (int(wrong.sum()), wrong.numel(), float((out.double() - ref).abs().max()), tol)
    return tol


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("d,group", [(64, 1), (128, 4), (64, 8), (128, 8), (128, 5), (64, 16), (128, 9)])
def test_weights_keep_32_bits(d, group, dtype):
    lens = [2 + s % 5 for s in range(40)]
    c = Case(311_500 + d + group, lens, group, 1, d, 8, dtype, q=one_element_queries(311_501, len(lens), group, d))
    out = c.run(dtype).cpu()
    assert pkv.device_error() == 0
    check(c, dtype, out)


@pytest.mark.parametrize("group", [1, 4, 8, 16])
@pytest.mark.parametrize("d", [64, 128])
def test_small_weights_beside_a_heavy_token(d, group):
    """A first token with 2^14 to 2^16 times the weight of each other and values of 0, as heads
    that have nothing to say attend: what is left is the sum of the small weights, times 1.

    Each is within 2^-22 of itself and 2^-36 of the heavy one (2^-20 of itself at most) by its two
    fp16 parts, 2^-22 by exp2, and by the scores (the heavy one's, up to 16 in the log2 domain,
    and their difference: 16 * 5 * 2^-24 ln 2, below 2^-18); the sums of 16 tokens and the division
    add 2^-20.  Together below 2^-17 of the result.  (A heavy token in another warp, or parts that
    hold 2^-31 of it, up to 2^-15 of a weight, is what this would tell from it.)"""
    gen = torch.Generator().manual_seed(311_520)
    seqs, n = 24, 16                                        # one warp's tokens
    lens = [n] * seqs
    size = (14 + 2 * torch.rand(seqs, group, generator=gen)) * np.log(2) / d ** -0.5
    q = torch.zeros(seqs, group, d)
    q[:, :, 0] = size
    k = torch.zeros(1, n, d)
    k[0, 0, 0] = 1.0                                        # step 1/15 in fp16: the heavy token's score is what the row holds
    rows = [torch.from_numpy(model.quantise(k.double().numpy())) for _ in range(seqs)]
    c = Case(311_521, lens, group, 1, d, 16, "f32", k_rows=rows, q=q)
    one = torch.ones(1, n, d)
    one[0, 0] = 0
    for s in range(seqs):
        c.v[c.tables[s, 0], :, :] = torch.from_numpy(model.quantise(one.double().numpy()))
    out = c.run("f32").cpu().double()
    assert pkv.device_error() == 0
    ref = torch.from_numpy(model.decode(c.q.double().numpy(), model.widen(c.k.numpy()), model.widen(c.v.numpy()),
                                        c.tables.numpy(), lens, c.scale))
    assert 15 * 2.0 ** -16.1 < ref.min() and ref.max() < 15 * 2.0 ** -13.9
    off = (out / ref - 1).abs()
    assert off.max() <= 2.0 ** -17, float(off.max() * 2 ** 17)
