"""What the library says about the kernel of a windowed prefill: the sizes that each kernel is
chosen for, what is refused, and that the tests of tests/test_window_prefill_gpu.py that name a
kernel, which choose it by a model of their own, reach that kernel."""
import ctypes

import pytest
import torch

import paged_kv_cache_310_gb300 as pkv
import test_window_prefill_gpu as prefill_tests
from paged_kv_cache_310_gb300 import _build

NAMES = dict(shared="shared_tiles", pairs="tile_pairs")


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return pkv.library()


def pool(heads, d, bs=16, dtype=torch.bfloat16, blocks=4):
    return torch.empty(blocks, heads, bs, d, dtype=dtype)


def plan(seqs, hq, tokens, longest, window, sinks=0, hkv=8, d=128, **kw):
    return pkv.paged_attention_prefill_window_plan(seqs, hq, tokens, longest, pool(hkv, d, **kw), window=window, sinks=sinks)


def test_the_sizes_that_each_kernel_is_for(lib):
    assert plan(1, 64, 4, 5000, 4096) == dict(kernel="rows", tokens_per_item=2, ctas_per_item=8)
    assert plan(64, 64, 256, 5000, 256, d=64)["kernel"] == "rows"
    assert plan(32, 64, 160, 20_000, 4096, 4) == dict(kernel="shared_tiles", tokens_per_item=16, ctas_per_item=1)
    assert plan(64, 64, 512, 8000, 1024)["kernel"] == "shared_tiles"
    assert plan(4, 64, 6000, 8000, 1024) == dict(kernel="tile_pairs", tokens_per_item=32, ctas_per_item=1)
    assert plan(4, 8, 6000, 8000, 1024)["tokens_per_item"] == 128      # one query head per KV head: a tile of as many tokens


def test_no_more_groups_of_rows_than_a_grid_takes(lib):
    # 60,000 sequences of one new token, one CTA each: two groups a sequence are counted
    assert plan(60_000, 16, 60_000, 1, 1, hkv=1, d=64)["kernel"] != "rows"
    assert plan(60, 16, 60, 1, 1, hkv=1, d=64)["kernel"] == "rows"


def test_windows_of_any_size(lib):
    for window, sinks in ((2 ** 31 - 1, 0), (1 << 40, 1 << 40), (2 ** 32 + 5, 0)):
        assert plan(4, 64, 6000, 8000, window, sinks) == plan(4, 64, 6000, 8000, 8000)


def test_nothing_to_do(lib):
    for seqs, tokens in ((0, 0), (0, 5), (3, 0)):
        assert plan(seqs, 64, tokens, 100, 10)["ctas_per_item"] == 0


def test_refusals(lib):
    for status, kw in ((1, dict(seqs=-1)), (1, dict(seqs=(1 << 20) + 1)), (1, dict(hq=60)), (2, dict(hq=8 * 17)), (1, dict(tokens=-1)),
                       (1, dict(longest=-1)), (2, dict(longest=(1 << 30) + 1)), (1, dict(window=0)), (1, dict(window=-2 ** 32 + 5)),
                       (1, dict(sinks=-1)), (2, dict(dtype=torch.float32)), (2, dict(hkv=4096, hq=4096)), (2, dict(bs=24)),
                       (2, dict(seqs=1 << 20, tokens=1 << 30, hq=1024, hkv=1024))):
        args = dict(seqs=4, hq=64, tokens=100, longest=1000, window=100)
        if "hkv" in kw:
            kw = dict(kw, blocks=1)
        with pytest.raises(pkv.PagedKVError) as e:
            plan(**{**args, **kw})
        assert e.value.status == status, kw
    d = pkv.CacheDesc(1 << 24, 16, 8, 128, pkv.BF16)
    out = pkv.WindowPlan()
    fn = lib.paged_attention_prefill_window_plan
    assert fn(4, 64, 100, 1000, 100, 0, ctypes.byref(d), ctypes.byref(out)) == 2   # rows past 32-bit coordinates
    d.num_blocks = 64
    assert fn(4, 64, 100, 1000, 100, 0, ctypes.byref(d), None) == 1
    assert fn(4, 64, 100, 1000, 100, 0, None, ctypes.byref(out)) == 1
    assert fn(4, 64, 100, 1000, 100, 0, ctypes.byref(d), ctypes.byref(out)) == 0


@pytest.mark.parametrize("name", ["seqs", "hq", "tokens", "longest"])
def test_sizes_past_32_bits_are_refused(lib, name):
    args = dict(seqs=4, hq=64, tokens=100, longest=1000, window=100)
    for wide in (2 ** 31, 2 ** 32 + args[name], -2 ** 32 + args[name], 1 << 70):
        with pytest.raises(pkv.PagedKVError) as e:
            plan(**{**args, name: wide})
        assert e.value.status == 1, wide


def named_sizes():
    """(kernel, seqs, hq, tokens, longest, window, sinks, hkv, d) of the tests that name their kernel."""
    for d, group, hkv, lens, new, window, sinks, kernel in prefill_tests.TILES:
        yield kernel, len(lens), group * hkv, sum(new), max(lens), window, sinks, hkv, d
    for test, kernel in ((prefill_tests.test_tiles_shared_by_two_warpgroups, "shared"), (prefill_tests.test_pairs_of_tiles, "pairs")):
        sizes = next(m.args[1] for m in test.pytestmark if m.args[0].startswith("d,bs"))
        for d, _, group, hkv, lens, new, window, sinks in sizes:
            yield kernel, len(lens), group * hkv, sum(new), max(lens), window, sinks, hkv, d


def test_the_kernels_that_other_tests_name(lib):
    found = [kernel for kernel, *sizes in named_sizes() if plan(*sizes)["kernel"] == NAMES[kernel]]
    assert len(found) == len(list(named_sizes())) == 15 and set(found) == {"shared", "pairs"}


def test_binding(lib):
    with pytest.raises(pkv.PagedKVError):
        pkv.paged_attention_prefill_window_plan(1, 8, 1, 1, torch.empty(4, 8, 16), window=1)
