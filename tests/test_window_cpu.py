"""The windowed calls without a GPU: what they refuse before any device work."""
import ctypes

import pytest
import torch

import paged_kv_cache_310_gb300 as pkv
from paged_kv_cache_310_gb300 import _build


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return pkv.library()


A = 0x10000


def desc(num_blocks=64, block_size=16, num_kv_heads=8, head_dim=128, dtype=pkv.BF16):
    return pkv.CacheDesc(num_blocks, block_size, num_kv_heads, head_dim, dtype)


def decode(lib, d=None, q=A, table=A, width=256, lens=A, S=4, Hq=64, L=4096, window=100, sinks=4, scale=0.1, out=A,
           out_dtype=pkv.BF16):
    return lib.paged_attention_decode_window(q, A, A, table, width, lens, S, Hq, L, window, sinks, scale, out, out_dtype,
                                             ctypes.byref(d or desc()), None)


def prefill(lib, d=None, q=A, table=A, width=256, lens=A, S=4, Hq=64, L=4096, window=100, sinks=4, scale=0.1, out=A,
            out_dtype=pkv.BF16, T=100, start=A):
    return lib.paged_attention_prefill_window(q, A, A, table, width, lens, start, S, Hq, T, L, window, sinks, scale, out,
                                              out_dtype, ctypes.byref(d or desc()), None)


@pytest.mark.parametrize("call", [decode, prefill])
def test_refusals_of_both_calls(lib, call):
    assert call(lib, S=0) == 0
    assert call(lib, window=0) == 1 and call(lib, window=-5) == 1 and call(lib, sinks=-1) == 1
    assert call(lib, Hq=60) == 1 and call(lib, Hq=8 * 17) == 2 and call(lib, S=-1) == 1 and call(lib, L=-1) == 1
    for bad in (desc(block_size=24), desc(head_dim=96), desc(dtype=pkv.KV4)):
        assert call(lib, d=bad) == 2
    assert call(lib, q=0) == 1 and call(lib, q=A + 8) == 1 and call(lib, out=0) == 1 and call(lib, lens=0) == 1
    assert call(lib, table=0) == 1 and call(lib, width=255) == 1           # the table covers max_context_len all the same
    assert call(lib, out_dtype=pkv.F16) == 2
    assert call(lib, scale=float("nan")) == 1


def test_refusals_of_one_call(lib):
    assert decode(lib, S=65536) == 1
    assert decode(lib, d=desc(dtype=pkv.F32), out_dtype=pkv.BF16) == 2           # the cache's dtype or f32
    assert prefill(lib, d=desc(dtype=pkv.F32), out_dtype=pkv.F32) == 2           # 16-bit caches only
    assert prefill(lib, d=desc(num_kv_heads=4096), Hq=4096) == 2
    assert prefill(lib, d=desc(num_blocks=1 << 24)) == 2                         # rows past 32-bit coordinates
    assert prefill(lib, start=0) == 1 and prefill(lib, T=-1) == 1 and prefill(lib, T=0) == 0
    assert prefill(lib, S=1 << 20, T=1 << 30, Hq=1024, d=desc(num_kv_heads=1024)) == 2  # more items than are counted
    assert prefill(lib, S=(1 << 20) + 1) == 1


def test_binding_refusals_without_a_gpu(lib):
    if torch.cuda.is_available():
        pytest.skip("GPU present")
    k = torch.zeros(2, 1, 16, 64)
    with pytest.raises(pkv.PagedKVError):
        pkv.paged_attention_decode_window(torch.zeros(1, 1, 64), k, k, torch.zeros(1, 2, dtype=torch.int32),
                                          torch.ones(1, dtype=torch.int32), 1.0, torch.zeros(1, 1, 64), window=3)
