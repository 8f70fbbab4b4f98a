"""Frequencies at the ends of what their arguments can be."""
import math

import pytest

import paged_kv_cache_310_gb300 as pkv
from paged_kv_cache_310_gb300 import _build


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()


@pytest.mark.parametrize("rotary_dim,base,factor", [(4, 1e300, 1e10), (128, 10000.0, 1e305), (4, 10000.0, 1e160), (64, 1e308, 1e2)])
def test_a_base_that_overflows_is_refused(rotary_dim, base, factor):
    # its frequencies would be 1, 0, 0, ...
    with pytest.raises(pkv.PagedKVError) as e:
        pkv.rotary_frequencies(rotary_dim, base, scaling="base", factor=factor)
    assert e.value.status == 1
    f, _ = pkv.rotary_frequencies(rotary_dim, base, scaling="linear", factor=factor)
    assert math.isclose(f[0], 1 / factor)


def test_the_largest_base_that_does_not():
    f, _ = pkv.rotary_frequencies(64, 1e300, scaling="base", factor=1e7)
    assert f[0] == 1 and (f > 0).all()


@pytest.mark.parametrize("rotary_dim", [2 ** 31, 2 ** 32 + 64, -2 ** 32 + 64, -2 ** 31 - 64, 1 << 70])
def test_sizes_past_32_bits_are_refused(rotary_dim, monkeypatch):
    # before anything is allocated, and not by their low 32 bits: the library would write 32 frequencies
    monkeypatch.setattr(pkv, "library", lambda: pytest.fail("reached the library"))
    with pytest.raises(pkv.PagedKVError) as e:
        pkv.rotary_frequencies(rotary_dim)
    assert e.value.status == 1
