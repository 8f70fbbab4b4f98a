"""The workspace of paged_attention_weights: the scores of a batch, but of long or ragged batches
no more than 4 GiB, or one sequence's own."""
import ctypes

import pytest

import paged_kv_cache_310_gb300 as pkv
from paged_kv_cache_310_gb300 import _build

MOST = 4 << 30


@pytest.fixture(scope="module")
def size():
    _build.build()
    lib = pkv.library()

    def size(seqs, hq, longest, hkv=8, dtype=pkv.KV4):
        d = pkv.CacheDesc(1 << 20, 16, hkv, 128, dtype)
        return lib.paged_attention_weights_workspace_bytes(seqs, hq, longest, ctypes.byref(d))

    return size


@pytest.mark.parametrize("seqs,hq,longest", [(256, 64, 131072), (65535, 64, 4096), (5000, 8, 100001), (9, 128, 1 << 20),
                                             (65535, 128, 1 << 24), (300, 64, 513)])
def test_bounded_whatever_the_batch(size, seqs, hq, longest):
    one = size(1, hq, longest)
    assert one >= 4 * hq * longest
    assert 0 < size(seqs, hq, longest) <= max(MOST + 256, 1.01 * one)


def test_whole_batches_below_the_bound(size):
    for seqs, hq, longest in ((64, 32, 2048), (8, 64, 32768), (120, 64, 131072)):
        assert seqs * hq * longest * 4 <= size(seqs, hq, longest) <= 1.01 * seqs * hq * longest * 4
    assert size(65535, 128, 512) == 0 and size(0, 64, 131072) == 0
