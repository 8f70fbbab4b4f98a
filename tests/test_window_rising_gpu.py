"""Scores that rise from token to token, so that running maxima move and what was summed before is
rescaled, with values that fall as the scores rise: each token's weight times its value has the same
size, and a part that gets lost or keeps a wrong scale shows, however old it is."""
import copy
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_310_gb300 as pkv
import test_window_prefill_gpu as prefill
from window_model import DT, Case

gpu = pytest.mark.gpu

# Scores run from -total / 2 to total / 2 in log2 units, total <= 90, each a sum of D <= 128 products of
# one sign: 128 * 2^-23 * 45 = 6.9e-4 in the exponent, 4.8e-4 of a weight (f32: sums of 4 to 8 at a
# time, 16 * 2^-24 * 45, 3e-5).  Sums of at most 2^13 terms: 2^-10 at worst (f32: a thread adds a
# few hundred at most, 2^-15).  Weights in two 16-bit parts 2^-17, exp2 2^-22.  Once for the sum of
# products and once for the weights': 2.9e-3 and 1.3e-4 of the sum of |weight * value|.
REL = {"f16": 3e-3, "bf16": 3e-3, "f32": 1.3e-4}


def rising(c, total):
    """The case's keys along its first query, which all queries become, and its values falling."""
    gen = torch.Generator().manual_seed(int(total))
    q = c.q[0, 0].clone()
    c.q[:] = q
    u = q.float() / q.float().norm() ** 2 * math.log(2) / c.scale
    for s, rows in enumerate(c.seen):
        if len(rows):
            x = torch.from_numpy(total * (rows / c.lens[s] - 0.5)).float()[:, None, None]
            at = torch.from_numpy(rows)
            block = c.tables[s].long()[at // c.bs]
            c.k[block, :, at % c.bs] = (x * u).expand(-1, c.hkv, -1).to(DT[c.dtype])
            c.v[block, :, at % c.bs] = (torch.randn(len(rows), c.hkv, c.d, generator=gen) * 2.0 ** -x).to(DT[c.dtype])
    return c


def bounds(c):
    """What the outputs should be, and how far off they may be."""
    sizes = copy.copy(c)
    sizes.v = c.v.abs()
    return c.reference(), REL[c.dtype] * sizes.reference()


def within(got, ref, tol):
    return bool((np.abs(got.double().cpu().numpy() - ref) <= tol).all())


# lens, window, sinks, total: the maxima of a warp's tiles (decode: every 32nd tile of 16 at most) move
DECODE = [([2000], 1500, 4, 48), ([1100, 700, 1300], 1000, 0, 90), ([5000, 900], 1200, 64, 80)]


def decode_case(i, dtype, group=4, d=128):
    lens, window, sinks, total = DECODE[i]
    return rising(Case(316_400 + i, list(lens), window, sinks, 2 * group, 2, d, 16, dtype), 14 if dtype == "f16" else total)


@gpu
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("group,d", [(4, 128), (16, 128), (8, 64), (1, 64)])
@pytest.mark.parametrize("i", range(len(DECODE)))
def test_decode(i, group, d, dtype):
    c = decode_case(i, dtype, group, d).cuda()
    ref, tol = bounds(c)
    out = torch.empty(c.q.shape, device="cuda")
    pkv.paged_attention_decode_window(c.g_q, c.g_k, c.g_v, c.g_tables, c.g_lens, c.scale, out, window=c.window, sinks=c.sinks,
                                      max_context_len=c.max_len)
    assert within(out, ref, tol) and pkv.device_error() == 0


# d, group, hkv, lens, new, window, sinks, total, kernel
PREFILL = [(128, 8, 2, [3000, 40], [2700, 3], 600, 5, 90, "tile_pairs"), (64, 5, 4, [2500, 800], [2400, 301], 500, 70, 90, "tile_pairs"),
           (128, 7, 2, [1200, 900], [600, 31], 600, 0, 64, "shared_tiles"), (64, 16, 2, [2500], [300], 2400, 33, 90, "shared_tiles"),
           (128, 8, 2, [3000, 700], [5, 3], 2000, 4, 90, "rows")]


def prefill_case(i, dtype):
    d, group, hkv, lens, new, window, sinks, total, _ = PREFILL[i]
    return rising(Case(316_450 + i, list(lens), window, sinks, group * hkv, hkv, d, 16, dtype, new=new), 14 if dtype == "f16" else total)


@gpu
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("i", range(len(PREFILL)))
def test_prefill(i, dtype):
    c = prefill_case(i, dtype)
    plan = pkv.paged_attention_prefill_window_plan(len(c.lens), c.hq, c.q.shape[0], c.max_len, c.k, window=c.window, sinks=c.sinks)
    assert plan["kernel"] == PREFILL[i][-1]
    ref, tol = bounds(c)
    assert within(prefill.run(c, "f32"), ref, tol) and pkv.device_error() == 0


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("i", range(len(DECODE)))
def test_a_lost_part_would_show(i, dtype):
    # the same outputs in 64 bits without one of the old tiles, and with one whose scale is off
    c = decode_case(i, dtype)
    ref, tol = bounds(c)
    assert within(torch.from_numpy(ref), ref, tol)
    for j in (c.lens[0] - c.window, c.lens[0] - c.window // 2):
        for factor in (0.0, 0.5):
            wrong = copy.copy(c)
            wrong.v = c.v.clone()
            for t in range(j, j + 16):
                wrong.v[c.tables[0, t // 16].long(), :, t % 16] *= factor
            assert not within(torch.from_numpy(wrong.reference()), ref, tol), (j, factor)
