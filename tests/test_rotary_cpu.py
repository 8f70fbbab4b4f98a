"""Rotary positions without a GPU: the frequencies of scaled rotations, and what the calls
refuse before any device work."""
import ctypes
import math
import struct

import numpy as np
import pytest
import torch

import paged_kv_cache_310_gb300 as pkv
import step_model as model
from paged_kv_cache_310_gb300 import _build


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return pkv.library()


def test_frequencies(lib):
    for dim, base in ((2, 10000.0), (16, 500.0), (64, 10000.0), (128, 1e6)):
        f, factor = pkv.rotary_frequencies(dim, base)
        assert factor == 1.0 and f.dtype == torch.float64 and f.device.type == "cpu"
        assert np.allclose(f.numpy(), model.frequencies(dim, base), rtol=1e-14, atol=0)


def test_scaled_frequencies(lib):
    plain = model.frequencies(128)
    f, factor = pkv.rotary_frequencies(128, scaling="linear", factor=4.0)
    assert factor == 1.0 and np.allclose(f.numpy(), plain / 4, rtol=1e-14)
    f, factor = pkv.rotary_frequencies(128, scaling="base", factor=8.0)
    assert factor == 1.0 and f[0] == 1.0 and math.isclose(f[-1], plain[-1] / 8, rel_tol=1e-12)
    f, factor = pkv.rotary_frequencies(128, scaling="parts", factor=16.0, original_len=4096)
    turns = 4096 * plain / (2 * math.pi)
    assert math.isclose(factor, 0.1 * math.log(16) + 1, rel_tol=1e-6)
    assert np.array_equal(f.numpy()[turns >= 32], pkv.rotary_frequencies(128)[0].numpy()[turns >= 32])
    assert np.allclose(f.numpy()[turns <= 1], plain[turns <= 1] / 16, rtol=1e-14)
    between = (turns > 1) & (turns < 32)
    keep = (turns[between] - 1) / 31
    assert between.any() and np.allclose(f.numpy()[between], plain[between] * (keep + (1 - keep) / 16), rtol=1e-13)
    for kw in (dict(scaling="linear"), dict(scaling="base"), dict(scaling="parts", original_len=100)):
        assert np.allclose(pkv.rotary_frequencies(64, **kw)[0].numpy(), model.frequencies(64), rtol=1e-13)  # by a factor of 1


@pytest.mark.parametrize("kw", [
    dict(rotary_dim=0), dict(rotary_dim=-2), dict(rotary_dim=7), dict(base=1.0), dict(base=math.inf), dict(base=math.nan),
    dict(scaling="linear", factor=0.5), dict(scaling="linear", factor=math.nan), dict(rotary_dim=2, scaling="base", factor=2.0),
    dict(scaling="parts", factor=2.0), dict(scaling="parts", factor=2.0, original_len=10, fast_turns=1.0),
    dict(scaling="parts", factor=2.0, original_len=math.inf), dict(scaling="other"),
])
def test_frequency_refusals(lib, kw):
    with pytest.raises(pkv.PagedKVError) as e:
        pkv.rotary_frequencies(kw.pop("rotary_dim", 64), **kw)
    assert e.value.status == 1


P = 0x100000000  # addresses that are only compared
STEP = 0x10000000


def rotary(inv_freq=P, dim=64, layout=0, factor=1.0, eps=1e-6, qw=0, kw=0):
    return struct.pack("@PiiffPP", inv_freq, dim, layout, factor, eps, qw, kw)


def qk(lib, q=P + STEP, qs=1024, k=P + 2 * STEP, ks=256, pos=P, tokens=5, hq=8, hkv=2, d=128, dtype=pkv.BF16, rot=None,
       qo=P + 3 * STEP, qos=1024, ko=P + 4 * STEP, kos=256):
    return lib.paged_qk_rotary(q, qs, k, ks, pos, tokens, hq, hkv, d, dtype, rot or rotary(), qo, qos, ko, kos, None)


def append(lib, q=P + STEP, qs=1024, k=P + 2 * STEP, ks=256, v=P + 3 * STEP, vs=256, pos=P, slots=P, tokens=5, hq=8, rot=None,
           qo=P + 4 * STEP, qos=1024, kc=P + 5 * STEP, vc=P + 6 * STEP, desc=None):
    d = desc or pkv.CacheDesc(64, 16, 2, 128, pkv.BF16)
    return lib.paged_kv_append_rotary(q, qs, k, ks, v, vs, pos, slots, tokens, hq, rot or rotary(), qo, qos, kc, vc,
                                      ctypes.byref(d), None)


@pytest.mark.parametrize("call", [qk, append])
def test_refusals_of_both_calls(lib, call):
    assert call(lib, tokens=0) == 0
    assert call(lib, tokens=-1) == 1
    assert call(lib, hq=-1) == 1 and call(lib, hq=65536) == 1
    for dim in (-16, 8, 24, 144, 256):
        assert call(lib, rot=rotary(dim=dim)) == 2, dim
    assert call(lib, rot=rotary(layout=2)) == 1
    assert call(lib, rot=rotary(factor=math.nan)) == 1 and call(lib, rot=rotary(factor=math.inf)) == 1
    assert call(lib, rot=rotary(inv_freq=0)) == 1 and call(lib, rot=rotary(inv_freq=P + 4)) == 1
    assert call(lib, rot=rotary(qw=P + 8)) == 1 and call(lib, rot=rotary(kw=P + 2)) == 1
    assert call(lib, rot=rotary(qw=P, eps=-1e-6)) == 1 and call(lib, rot=rotary(kw=P, eps=math.nan)) == 1
    for name in ("q", "k", "qo"):
        assert call(lib, **{name: 0}) == 1 and call(lib, **{name: P + STEP * 9 + 8}) == 1, name
    assert call(lib, pos=0) == 1
    # strides: below the token's own size, not a multiple of 16 bytes, far too large
    assert call(lib, qs=1016) == 1 and call(lib, qs=1028) == 1 and call(lib, ks=1 << 29) == 1 and call(lib, qos=512) == 1
    # overlaps: q_out over k; over q but not at its place; at q's place with another stride
    assert call(lib, qo=P + 2 * STEP) == 1 and b"overlaps" in lib.paged_kv_last_error()
    assert call(lib, qo=P + STEP + 256) == 1
    assert call(lib, qs=1040, qo=P + STEP) == 1
    # parts of one table lie beside each other; one element further they do not
    assert call(lib, qs=2048, qo=P + STEP + 2 * 1016, qos=2048) == 1


def test_refusals_of_qk_rotary(lib):
    assert qk(lib, dtype=pkv.KV4) == 2 and qk(lib, dtype=-1) == 2 and qk(lib, d=96) == 2
    assert qk(lib, ko=0) == 1 and qk(lib, hkv=-1) == 1
    assert qk(lib, ko=P + STEP) == 1 and qk(lib, ko=P + 3 * STEP) == 1 and qk(lib, ko=P + 2 * STEP + 16) == 1
    assert qk(lib, hq=0, hkv=0) == 0


def test_refusals_of_append_rotary(lib):
    assert append(lib, v=0) == 1 and append(lib, slots=0) == 1 and append(lib, kc=0) == 1 and append(lib, vc=P + 8) == 1
    assert append(lib, vs=128) == 1 and append(lib, qo=P + 3 * STEP) == 1
    assert append(lib, desc=pkv.CacheDesc(64, 16, 2, 128, pkv.KV4)) == 2
    assert append(lib, desc=pkv.CacheDesc(64, 12, 2, 128, pkv.BF16)) == 2


def test_binding_refusals_without_a_gpu(lib):
    if torch.cuda.is_available():
        pytest.skip("GPU present")
    t = torch.zeros(3, 2, 64)
    pos = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(pkv.PagedKVError):
        pkv.paged_qk_rotary(t, t, pos, t, t, None)
    with pytest.raises(pkv.PagedKVError):
        pkv.paged_kv_append_rotary(t, t, t, pos, pos.long(), torch.zeros(2, 2, 8, 64), torch.zeros(2, 2, 8, 64), t, None)
