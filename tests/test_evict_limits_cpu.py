"""Eviction's number of recent rows past what 32 bits hold: all rows that are kept, not the number's
low 32 bits."""
import pytest
import torch

import paged_kv_cache_310_gb300 as pkv
from paged_kv_cache_310_gb300 import _build

MOST = 2 ** 31 - 1


@pytest.fixture
def passed(monkeypatch):
    _build.build()
    seen = []
    monkeypatch.setattr(pkv, "_one_device", lambda *t: 0)
    monkeypatch.setattr(pkv, "_call", lambda fn, device, *args: seen.append([t(a) if t.__name__ == "c_int" else a
                                                                             for t, a in zip(fn.argtypes, args)]))
    return seen


def recent_of(passed, recent):
    k = torch.zeros(4, 1, 16, 64)
    ints = lambda *shape: torch.zeros(*shape, dtype=torch.int32)
    pkv.paged_kv_evict(torch.zeros(1, 1, 40), ints(1, 3), ints(1), ints(1), ints(1, 1), k, k, torch.zeros(1, 1, 40), ints(1, 1, 16),
                       recent=recent, max_context_len=40)
    return passed.pop()[7].value


def test_recent(passed):
    for given, held in ((0, 0), (8, 8), (MOST, MOST), (MOST + 1, MOST), (2 ** 32, MOST), (2 ** 32 + 8, MOST), (1 << 70, MOST)):
        assert recent_of(passed, given) == held, given
    for given in (-1, -2 ** 32, -2 ** 32 + 8, -(1 << 70)):
        assert recent_of(passed, given) < 0, given
