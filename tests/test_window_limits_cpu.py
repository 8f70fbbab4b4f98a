"""Windows and sinks past what 32 bits hold: the binding passes them on as the largest that do,
which changes nothing for a sequence, and never as another number."""
import inspect

import pytest
import torch

import paged_kv_cache_310_gb300 as pkv
from paged_kv_cache_310_gb300 import _build

MOST = 2 ** 31 - 1


@pytest.fixture
def passed(monkeypatch):
    """Calls without a GPU, on CPU tensors: what would have gone to the library, by the C argument's place."""
    _build.build()
    seen = []
    monkeypatch.setattr(pkv, "_one_device", lambda *t: 0)
    monkeypatch.setattr(pkv, "_call", lambda fn, device, *args: seen.append([t(a) if t.__name__ == "c_int" else a
                                                                             for t, a in zip(fn.argtypes, args)]))
    return seen


def call(name, **kw):
    k = torch.zeros(4, 1, 16, 64)
    q = torch.zeros(1, 1, 64)
    args = dict(q=q, k_cache=k, v_cache=k, block_tables=torch.zeros(1, 4, dtype=torch.int32),
                context_lens=torch.ones(1, dtype=torch.int32), scale=1.0, out=torch.zeros_like(q), window=3, max_context_len=50)
    fn = getattr(pkv, name)
    if "query_start" in inspect.signature(fn).parameters:
        args["query_start"] = torch.tensor([0, 1], dtype=torch.int32)
    fn(**{**args, **kw})


def sizes(name, args):
    """(max_context_len, window, sinks) as C gets them."""
    first = 8 if name.endswith("decode_window") else 10
    return tuple(a.value for a in args[first:first + 3])


CALLS = ["paged_attention_decode_window", "paged_attention_prefill_window"]


@pytest.mark.parametrize("name", CALLS)
def test_large_windows_and_sinks_stay_large(passed, name):
    for given, held in ((1, 1), (MOST - 1, MOST - 1), (MOST, MOST), (MOST + 1, MOST), (2 ** 32 - 1, MOST), (2 ** 32, MOST),
                        (2 ** 32 + 5, MOST), (1 << 40, MOST), (2 ** 63 - 1, MOST), (1 << 70, MOST)):
        call(name, window=given, sinks=given)
        assert sizes(name, passed.pop()) == (50, held, held), given


@pytest.mark.parametrize("name", CALLS)
def test_negative_ones_stay_negative(passed, name):
    # so that the library refuses them
    for given in (-1, -MOST, -2 ** 31 - 1, -2 ** 32 + 5, -2 ** 32, -(1 << 70)):
        call(name, window=given, sinks=given)
        _, window, sinks = sizes(name, passed.pop())
        assert window < 0 and sinks < 0, given


@pytest.mark.parametrize("name", CALLS)
def test_a_bound_of_lengths_past_32_bits_is_refused(passed, name):
    for given in (MOST + 1, 2 ** 32 + 50, -2 ** 32 + 50, -2 ** 31 - 1):
        with pytest.raises(pkv.PagedKVError) as e:
            call(name, max_context_len=given)
        assert e.value.status == 1 and not passed
