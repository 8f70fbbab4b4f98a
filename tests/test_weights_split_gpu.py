"""Attention weights of contexts that are too long for one CTA (scores kept in a workspace, a
second kernel that joins the partitions): infinite and NaN rows, bad tables and lengths, every
kind of pool.  Each test asserts that its call needs a workspace."""
import pytest
import torch

import paged_kv_cache_310_gb300 as pkv
from test_evict_gpu import Step

pytestmark = pytest.mark.gpu

KINDS = [("f32", None), ("f16", None), ("bf16", None), ("kv4", "f16"), ("kv4", "bf16"), ("kv4", "f32")]


def splits(c, max_len=None):
    return pkv.paged_attention_weights_workspace_bytes(len(c.lens), c.q.shape[1], max_len or c.max_len, c.k) > 0


@pytest.mark.parametrize("pool", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n", [700, 5000])
def test_infinite_and_nan_rows(pool, n):
    # -inf scores give a token no weight, wherever its partition; a NaN row makes its KV head's
    # weights NaN in every partition, and no other's
    c = Step(311_700, [n, n], 2, 2, 64, 16, pool)
    assert splits(c)
    c.q = c.q.abs()
    light = [5, n // 2, n - 1]
    for j in light:
        c.k[c.tables[0, j // 16], 0, j % 16] = float("-inf")
    c.k[c.tables[1, (n - 9) // 16], 1, (n - 9) % 16] = float("nan")
    out = c.run(tracked=[0, 0]).cpu()
    assert pkv.device_error() == 0
    assert (out[0, 0, light] == 0).all() and not out[0, :, :n].isnan().any()
    assert abs(float(out[0, 0, :n].double().sum()) - 1) < 1e-5
    assert out[1, 1, :n].isnan().all() and not out[1, 0, :n].isnan().any()


@pytest.mark.parametrize("q_dtype", ["f16", "f32"])
def test_nan_groups_of_4_bit_rows(q_dtype):
    n = 3000
    c = Step(311_710, [n, n], 8, 2, 128, 16, "kv4", q_dtype)
    assert splits(c)
    c.k[c.tables[1, 100], 0, 3, 64:68] = 255                # (step, lo) of one group
    out = c.run(tracked=[0, 0]).cpu()
    assert pkv.device_error() == 0
    assert out[1, 0, :n].isnan().all() and not out[1, 1, :n].isnan().any() and not out[0, :, :n].isnan().any()


@pytest.mark.parametrize("q_dtype", ["f16", "f32"])
@pytest.mark.parametrize("n", [300, 3000])
def test_an_infinite_query(q_dtype, n):
    c = Step(311_715, [n], 8, 2, 128, 16, "kv4", q_dtype)
    assert splits(c) == (n > 512)
    c.q[0, 2, 7] = float("inf")
    out = c.run(tracked=[0]).cpu()
    assert pkv.device_error() == 0
    assert out[0, 0, :n].isnan().all() and not out[0, 1, :n].isnan().any()


@pytest.mark.parametrize("pool,q_dtype", KINDS)
def test_bad_tables_and_lengths_set_the_flag(pool, q_dtype):
    c = Step(311_720, [1500, 20], 8, 2, 128, 16, pool, q_dtype)
    assert splits(c)
    for bad in (1 << 20, -7):
        c.tables[0, 60] = bad
        c.run()
        assert pkv.device_error() == 5
    c = Step(311_721, [1500, 20, 0], 8, 2, 128, 16, pool, q_dtype)
    out = c.run(max_context_len=1499)
    assert splits(c, 1499) and pkv.device_error() == 5
    assert (out[0] == 7).all() and not (out[1, :, :20] == 7).any() and (out[1, :, 20:] == 7).all() and (out[2] == 7).all()


@pytest.mark.parametrize("pool,q_dtype", KINDS)
def test_wide_bounds_and_untracked_rows(pool, q_dtype):
    # lengths far below the bound, so that most partitions are empty
    c = Step(311_730, [9, 0, 1200, 513], 12, 2, 64, 32, pool, q_dtype, width=8192)
    c.tables = torch.nn.functional.pad(c.tables, (0, 256 - c.tables.shape[1]), value=-1)
    assert splits(c, 8192)
    c.check(max_context_len=8192)
    c.check(tracked=[3, 0, 700, 0], in_place=True, max_context_len=8192)


def test_repeats_do_not_change_a_bit():
    for pool, q_dtype in KINDS:
        c = Step(311_740, [4000, 600], 16, 2, 128, 16, pool, q_dtype)
        assert splits(c)
        outs = [c.run(tracked=[0, 0]) for _ in range(4)]
        torch.cuda.synchronize()
        assert all(torch.equal(outs[0].nan_to_num(5.0), o.nan_to_num(5.0)) for o in outs[1:])


class Wide(Step):
    """A step under a bound on the lengths far above them, with accumulators as wide."""

    def run(self, tracked=None, in_place=False, *, bound):
        q, k, tables, lens, before = (t.cuda() for t in (self.q, self.k, self.tables,
                                                         torch.tensor(self.lens, dtype=torch.int32), self.before))
        w = torch.full((*before.shape[:2], bound), 5.0, device="cuda")
        w[:, :, :before.shape[2]] = before
        out = w if in_place else torch.full_like(w, 7.0)
        t = None if tracked is None else torch.tensor(tracked, dtype=torch.int32).cuda()
        tables = torch.nn.functional.pad(tables, (0, -(-bound // self.k.shape[2]) - tables.shape[1]), value=-1)
        pkv.paged_attention_weights(q, k, tables, lens, self.scale, w, weights_out=out, tracked_lens=t, max_context_len=bound)
        assert (out[:, :, before.shape[2]:] == (5.0 if in_place else 7.0)).all()
        return out[:, :, :before.shape[2]].contiguous()


@pytest.mark.parametrize("pool,q_dtype", [("kv4", "f16"), ("bf16", None)])
def test_batches_in_turns(pool, q_dtype):
    # 37 sequences of 64 heads under a bound of 524,289 tokens: 5 GB of scores, so two turns
    bound = 524_289
    lens = [(41 * s) % 700 + (5000 if s in (3, 19) else 0) for s in range(37)]
    c = Wide(311_750, lens, 64, 4, 64, 64, pool, q_dtype)
    one = pkv.paged_attention_weights_workspace_bytes(1, 64, bound, c.k)
    assert one < pkv.paged_attention_weights_workspace_bytes(37, 64, bound, c.k) < 30 * one
    c.check(bound=bound)
    c.check(tracked=[max(0, n - 1) for n in lens], in_place=True, bound=bound)
