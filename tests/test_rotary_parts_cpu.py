"""Frequencies scaled by parts: linear in the turns, which is what the header says, and how far that is
from rules that are linear in the dimension's index, which the header and the binding warn of."""
import math

import numpy as np

import paged_kv_cache_310_gb300 as pkv
import step_model as model
from paged_kv_cache_310_gb300 import _build


def by_index(dim, base, factor, original_len, fast, slow):
    plain, i = model.frequencies(dim, base), np.arange(dim // 2)
    at = lambda turns: dim * math.log(original_len / (2 * math.pi * turns)) / (2 * math.log(base))
    low, high = math.floor(at(fast)), math.ceil(at(slow))
    divided = np.clip((i - low) / (high - low), 0, 1)
    return plain / factor * divided + plain * (1 - divided)


def test_the_stated_difference():
    _build.build()
    f = pkv.rotary_frequencies(128, scaling="parts", factor=16.0, original_len=4096)[0].numpy()
    apart = by_index(128, 10000.0, 16.0, 4096, 32.0, 1.0) / f
    assert 2.9 < apart.max() < 3.1 and apart.min() > 0.9
    for text in (open(pkv.HEADER).read(), pkv.rotary_frequencies.__doc__):
        assert "by up to a factor of 3" in " ".join(text.replace("*", " ").split())


def test_frequencies_alone_with_four_turns():
    # a rule that is linear in the turns and has no factor of cosines and sines
    f, _ = pkv.rotary_frequencies(128, 500000.0, scaling="parts", factor=8.0, original_len=8192, fast_turns=4.0, slow_turns=1.0)
    plain = model.frequencies(128, 500000.0)
    turns = 8192 * plain / (2 * math.pi)
    want = np.where(turns > 4, plain, np.where(turns < 1, plain / 8, plain / 8 + (plain - plain / 8) * (turns - 1) / 3))
    assert np.allclose(f.numpy(), want, rtol=1e-12)
