"""The windowed calls without a GPU: workspace sizes, and what they refuse before any device work."""
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
           out_dtype=pkv.BF16, ws=A, wsb=1 << 40):
    return lib.paged_attention_decode_window(q, A, A, table, width, lens, S, Hq, L, window, sinks, scale, out, out_dtype, ws,
                                             wsb, ctypes.byref(d or desc()), None)


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
    assert decode(lib, d=desc(dtype=pkv.F32), Hq=72, out_dtype=pkv.F32) == 2     # f32: groups up to 8
    assert decode(lib, S=65536) == 1
    assert prefill(lib, d=desc(dtype=pkv.F32), out_dtype=pkv.F32) == 2           # 16-bit caches only
    f32 = dict(d=desc(dtype=pkv.F32), out_dtype=pkv.F32, window=3000)            # split over CTAs: a workspace
    assert decode(lib, ws=0, **f32) == 3 and decode(lib, wsb=16, **f32) == 3 and decode(lib, ws=A + 128, **f32) == 1
    assert prefill(lib, start=0) == 1 and prefill(lib, T=-1) == 1 and prefill(lib, T=0) == 0


def need(lib, S=64, Hq=64, L=100_000, window=1024, sinks=4, dtype=pkv.F32):
    return lib.paged_attention_decode_window_workspace_bytes(S, Hq, L, window, sinks, ctypes.byref(desc(dtype=dtype)))


def test_workspace_goes_by_the_window(lib):
    assert need(lib, dtype=pkv.BF16) == 0 and need(lib, window=10 ** 6, dtype=pkv.F16) == 0   # 16-bit caches: one kernel
    assert need(lib, L=100_000) == need(lib, L=2_000_000_000) > 0
    assert need(lib, window=2_000_000_000, sinks=0, L=5000) == need(lib, window=5000, sinks=0, L=5000) > 0
    assert need(lib, window=2 ** 31 - 1, sinks=2 ** 31 - 1, L=5000) == need(lib, window=5000, sinks=0, L=5000)
    assert need(lib, window=0) == 0 and need(lib, sinks=-1) == 0


def test_binding_refusals_without_a_gpu(lib):
    if torch.cuda.is_available():
        pytest.skip("GPU present")
    k = torch.zeros(2, 1, 16, 64)
    with pytest.raises(pkv.PagedKVError):
        pkv.paged_attention_decode_window(torch.zeros(1, 1, 64), k, k, torch.zeros(1, 2, dtype=torch.int32),
                                          torch.ones(1, dtype=torch.int32), 1.0, torch.zeros(1, 1, 64), window=3)
