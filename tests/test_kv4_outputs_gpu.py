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


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("d,group", [(64, 1), (128, 4), (64, 8), (128, 8), (128, 5), (64, 16), (128, 9)])
def test_weights_keep_32_bits(d, group, dtype):
    lens = [2 + s % 5 for s in range(40)]
    c = Case(311_500 + d + group, lens, group, 1, d, 8, dtype, q=one_element_queries(311_501, len(lens), group, d))
    out = c.run(dtype).cpu()
    assert pkv.device_error() == 0
    check(c, dtype, out)
