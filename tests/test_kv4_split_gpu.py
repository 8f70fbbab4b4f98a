"""Single-token attention over 4-bit pools where (sequence, KV head) items are split over CTAs
and joined: 16-bit outputs, non-finite inputs, rising maxima, shares that begin and end anywhere.
Each test asserts that its call needs a workspace, which only split items do.  Tolerances are
those of test_kv4_decode_gpu.py and test_kv4_outputs_gpu.py."""
import numpy as np
import pytest
import torch

import kv4_model as model
import paged_kv_cache_310_gb300 as pkv
from test_kv4_decode_gpu import DT, HALF_STEP, Case, kv_rows
from test_kv4_outputs_gpu import check as check_rounding
from test_kv4_outputs_gpu import one_element_queries

pytestmark = pytest.mark.gpu


def splits(c, max_len=None):
    return pkv.paged_attention_decode_kv4_workspace_bytes(len(c.lens), c.q.shape[1], max_len or c.max_len, c.q.dtype, c.k) > 0


# up to eight pieces of an item are joined at once, more in turn
LENGTHS = [[1300, 513, 0, 40], [2049, 1, 2048], [20000], [9001, 600]]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("d,bs,group,hkv", [(64, 16, 1, 2), (128, 8, 4, 1), (128, 16, 8, 2), (64, 64, 6, 1), (128, 32, 16, 1),
                                            (64, 16, 9, 1)])
@pytest.mark.parametrize("lens", LENGTHS, ids=lambda x: "-".join(map(str, x)))
def test_16_bit_outputs(lens, d, bs, group, hkv, dtype):
    q = one_element_queries(311_600, len(lens), group * hkv, d)
    c = Case(311_601 + d + bs + group, lens, group * hkv, hkv, d, bs, dtype, q=q)
    assert splits(c)
    out = c.run(dtype).cpu()
    assert pkv.device_error() == 0
    tol = check_rounding(c, dtype, out)
    wide = c.run("f32").cpu().double()
    # the same call with f32 outputs: either is within tol of the exact result, and one is rounded
    assert ((out.double() - wide).abs() <= HALF_STEP[dtype] * (wide.abs() + tol) + 2 * tol).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("group", [1, 8, 16])
def test_16_bit_outputs_of_more_units_than_ctas(group, dtype):
    # each CTA has several whole items and two parts
    gen = torch.Generator().manual_seed(311_610)
    lens = torch.randint(1, 1500, (40,), generator=gen).tolist()
    c = Case(311_611 + group, lens, 12 * group, 12, 64, 16, dtype)
    assert splits(c)
    c.check(dtype)


@pytest.mark.parametrize("lens,hkv", [([600] * 5, 3), ([1280] * 3, 1), ([513, 1, 512, 640], 1), ([513], 1), ([768], 1),
                                      ([128 * 9] * 4 + [0] * 200 + [127] * 70 + [1] * 60, 2), ([0] * 300 + [700], 2),
                                      ([128] * 700, 1), ([129, 1] * 320, 2)])
def test_shares_that_begin_and_end_anywhere(lens, hkv):
    # units of 128 tokens: items that fill a CTA's share, cross one, lie with others in one
    c = Case(311_620, lens, 4 * hkv, hkv, 64, 8, "f16")
    bound = max(c.max_len, 520)
    c.tables = torch.nn.functional.pad(c.tables, (0, max(0, 65 - c.tables.shape[1])), value=-1)
    assert splits(c, bound)
    c.check("f32", max_context_len=bound)


@pytest.mark.parametrize("n", [1500, 9000])
@pytest.mark.parametrize("group,out_dtype", [(1, "f32"), (4, "f32"), (8, "f32"), (16, "f32"), (8, "bf16"), (16, "bf16")])
def test_running_maximum_rising(n, group, out_dtype):
    d, scale = 64, 64 ** -0.5
    gen = torch.Generator().manual_seed(311_630)
    q = torch.randn(1, 1, d, generator=gen).repeat(1, group, 1).bfloat16().float()
    u = q[0, 0] / q[0, 0].norm()
    grow = torch.linspace(-1, 1, n)[:, None] * (60 / (q[0, 0].norm() * scale)) * u
    rows = [torch.from_numpy(model.quantise((grow + 0.05 * torch.randn(n, d, generator=gen))[None].double().numpy()))]
    c = Case(311_631, [n], group, 1, d, 16, out_dtype, k_rows=rows, q=q)
    assert splits(c)
    c.check(out_dtype)


@pytest.mark.parametrize("n", [1400, 9000])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_non_finite_inputs_reach_only_what_attends_to_them(n, dtype):
    gen = torch.Generator().manual_seed(311_640)
    lens = [n, n - 1, n]
    rows = kv_rows(gen, lens, 2, 64)
    rows[1][0, n // 2, 32:] = 255                           # K of sequence 1, KV head 0: NaN in one share
    c = Case(311_641, lens, 4, 2, 64, 16, dtype, k_rows=rows)
    assert splits(c)
    c.v[c.tables[2, (n - 5) // 16], 1, (n - 5) % 16, 32:36] = 255   # V of sequence 2, KV head 1, near its end: dims 0..31
    c.q[0, 3, 5] = float("inf")                             # a query of sequence 0, KV head 1
    out = c.run(dtype).cpu()
    assert pkv.device_error() == 0
    want = torch.zeros(3, 4, 64, dtype=torch.bool)
    want[0, 3] = True
    want[1, :2] = True
    want[2, 2:, :32] = True
    assert torch.equal(out.isnan(), want)


@pytest.mark.parametrize("out_dtype", ["f16", "f32"])
def test_bad_tables_and_lengths_set_the_flag(out_dtype):
    c = Case(311_650, [1500, 20], 8, 2, 128, 16, "f16")
    assert splits(c)
    for bad in (1 << 20, -7):
        c.tables[0, 60] = bad
        c.run(out_dtype)
        assert pkv.device_error() == 5
    c = Case(311_651, [1500, 20, 0, 700], 8, 2, 128, 16, "f16")
    out = c.run(out_dtype, max_context_len=1499)
    assert splits(c, 1499) and pkv.device_error() == 5
    assert (out[0] == 7).all() and (out[2] == 0).all()      # left as it was; the others are done
    ref, tol, _ = c.reference()
    for s in (1, 3):
        assert (np.abs(out[s].cpu().double().numpy() - ref[s]) <= tol + HALF_STEP[out_dtype] * np.abs(ref[s])).all()


@pytest.mark.parametrize("bound", [0, 16, 500, 512, 513, 9000])
def test_all_empty_sequences_under_any_bound(bound):
    c = Case(311_660, [0, 0, 0], 8, 2, 64, 16, "f16")
    c.tables = torch.full((3, max(1, -(-bound // 16))), -1, dtype=torch.int32)
    assert splits(c, bound) == (bound > 512)
    for out_dtype in ("f16", "f32"):
        assert (c.run(out_dtype, max_context_len=bound) == 0).all()
    assert pkv.device_error() == 0


def test_repeats_and_placement_do_not_change_a_bit():
    for dtype in ("f16", "bf16"):
        outs = []
        for order in (0, 1):
            c = Case(311_670, [1400, 33, 9000], 16, 2, 128, 16, dtype)
            if order:                                       # the same rows in other blocks
                perm = torch.randperm(c.k.shape[0], generator=torch.Generator().manual_seed(311_671))
                moved = torch.empty_like(perm)
                moved[perm] = torch.arange(perm.numel())
                c.k, c.v = c.k[perm].contiguous(), c.v[perm].contiguous()
                c.tables = torch.where(c.tables < 0, c.tables, moved[c.tables.clamp(min=0).long()].to(torch.int32))
            assert splits(c)
            outs += [c.run(dtype) for _ in range(3)]
        torch.cuda.synchronize()
        assert all(torch.equal(outs[0], o) for o in outs[1:])
