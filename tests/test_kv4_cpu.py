"""4-bit caches without a GPU: the format's model against hand-worked rows and its own error
bound, and the library's argument checks, which answer before any device work."""
import ctypes

import numpy as np
import pytest
import torch

import kv4_model as model
import paged_kv_cache_310_gb300 as pkv
from paged_kv_cache_310_gb300 import _build


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return pkv.library()


def desc(num_blocks=64, block_size=16, num_kv_heads=8, head_dim=128, dtype=pkv.KV4):
    return pkv.CacheDesc(num_blocks, block_size, num_kv_heads, head_dim, dtype)


A = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10008)


def test_model_hand_worked_row():
    # one group 0, 1, ..., 15 twice: lo 0, step 1, every code its value; the other all 2.5
    x = np.concatenate([np.arange(32) % 16, np.full(32, 2.5)])
    row = model.quantise(x)
    assert row.shape == (40,)
    assert row[:16].tolist() == [0x10, 0x32, 0x54, 0x76, 0x98, 0xBA, 0xDC, 0xFE] * 2
    assert row[16:32].tolist() == [0] * 16                       # step 0: codes 0
    assert row[32:].view(np.float16).tolist() == [1.0, 0.0, 0.0, 2.5]
    assert model.widen(row).tolist() == x.tolist()


def test_model_ties_go_to_even_and_ends_are_held():
    # lo 0, step 2 (max 30): 1 / 2 = 0.5 -> 0, 3 / 2 = 1.5 -> 2, 5 / 2 = 2.5 -> 2
    x = np.zeros(32)
    x[:5] = [30, 1, 3, 5, 7]
    assert model.widen(model.quantise(x))[:5].tolist() == [30, 0, 4, 4, 8]
    big = np.zeros(64)
    big[0], big[1] = 1e9, -1e9
    got = model.widen(model.quantise(big))
    # lo = -65408; step = fp16(130816 / 15 = 8721.07) = 8720: 15 steps up are 65392, stored as its fp16 neighbour
    assert got[1] == -65408 and got[0] == float(np.float16(65392)) and np.isfinite(got).all()


def test_model_non_finite_groups():
    x = np.ones(64)
    x[3] = np.inf
    got = model.widen(model.quantise(x))
    assert np.isnan(got[:32]).all() and (got[32:] == 1).all()


def test_model_error_bound():
    # a value is at most half a step, and the roundings of lo, step and the sum, away
    rng = np.random.default_rng(310_700)
    x = (rng.standard_normal((500, 128)) * rng.uniform(0.01, 50, (500, 1)) + rng.standard_normal((500, 1))) \
        .astype(np.float32).astype(np.float64)
    got = model.widen(model.quantise(x))
    g = x.reshape(500, 4, 32)
    spread = (g.max(-1) - g.min(-1))[..., None]
    size = np.abs(g).max(-1)[..., None]
    # half a step of spread / 15; fp16 rounding (2^-11 relative, or 2^-25) of lo and of the value, and of step 15 times
    bound = spread / 30 * (1 + 2.0 ** -10) + 2.0 ** -10 * size + 15 * (spread / 15 * 2.0 ** -11 + 2.0 ** -25) + 2.0 ** -23
    assert (np.abs(got.reshape(g.shape) - g) <= bound).all()


def test_descriptor_of_a_4bit_pool():
    d = pkv.cache_desc(torch.empty((3, 2, 16, 80), dtype=torch.uint8))
    assert (d.num_blocks, d.num_kv_heads, d.block_size, d.head_dim, d.dtype) == (3, 2, 16, 128, pkv.KV4)
    assert pkv.cache_desc(torch.empty((3, 2, 16, 40), dtype=torch.uint8)).head_dim == 64
    with pytest.raises(pkv.PagedKVError):
        pkv.cache_desc(torch.empty((3, 2, 16, 64), dtype=torch.uint8))


def test_other_calls_refuse_4bit_pools(lib):
    d = desc()
    p = ctypes.byref(d)
    assert lib.paged_kv_append(A, A, A, 3, A, A, p, None) == 2
    assert lib.paged_attention_decode(A, A, A, A, 256, A, 4, 32, 4096, 1.0, A, 2, A, 1 << 30, p, None, None) == 2
    assert lib.paged_attention_prefill(A, A, A, A, 256, A, A, 4, 32, 64, 4096, 1.0, A, 2, A, 1 << 30, p, None) == 2
    assert lib.paged_kv_gather(A, A, A, 4, A, 1, 16, A, A, p, None) == 2
    assert lib.paged_attention_workspace_bytes(4, 32, 4096, p, None) == 0
    # whole-block moves take them (nothing to do here; bad ids are refused as for other pools)
    assert lib.paged_block_copy(A, None, 0, A, A, p, None) == 0
    pair = (ctypes.c_int64 * 2)(1, 64)
    assert lib.paged_block_copy(A, pair, 1, A, A, p, None) == 1
    assert lib.paged_block_swap_out(A, 0, A, A, A, A, p, None) == 0


def test_append_checks(lib):
    d = desc()

    def run(dtype=pkv.BF16, n=3, k=A, v=A, slots=A, kc=A, vc=A, d=d):
        return lib.paged_kv4_append(k, v, dtype, slots, n, kc, vc, ctypes.byref(d), None)

    assert run(n=0) == 0
    assert run(n=-1) == 1
    for bad in (dict(k=None), dict(v=None), dict(slots=None), dict(kc=None), dict(vc=None)):
        assert run(**bad) == 1
    assert run(k=ODD) == 1 and b"aligned" in lib.paged_kv_last_error()
    assert run(vc=ODD) == 1
    assert run(dtype=pkv.KV4) == 2 and run(dtype=-1) == 2
    assert run(d=desc(dtype=pkv.BF16)) == 2                  # not a 4-bit pool
    assert run(d=desc(head_dim=96)) == 2 and run(d=desc(block_size=4)) == 2
    assert run(d=desc(num_blocks=0)) == 1
    assert lib.paged_kv4_append(A, A, 2, A, 3, A, A, None, None) == 1
    assert run(d=desc(num_kv_heads=65535, block_size=64, head_dim=128), n=0) == 0
    assert run(d=desc(num_kv_heads=65536)) == 2


def test_expand_checks(lib):
    d = desc()

    def run(out=None, n=3, pairs=A, kc=A, vc=A, ko=A, vo=A, d=d):
        out = out or desc(dtype=pkv.F16, num_blocks=9)
        return lib.paged_kv4_expand(pairs, n, kc, vc, ctypes.byref(d), ko, vo, ctypes.byref(out), None)

    assert run(n=0) == 0
    assert run(n=-1) == 1
    for bad in (dict(pairs=None), dict(kc=None), dict(vc=None), dict(ko=None), dict(vo=None)):
        assert run(**bad) == 1
    assert run(ko=ODD) == 1 and run(kc=ODD) == 1
    assert run(out=desc(dtype=pkv.KV4)) == 2                 # the out pools are wide
    assert run(d=desc(dtype=pkv.F16)) == 2                   # the source is a 4-bit pool
    for other in (dict(block_size=8), dict(num_kv_heads=4), dict(head_dim=64)):
        assert run(out=desc(dtype=pkv.F16, **other)) == 1
        assert b"equal" in lib.paged_kv_last_error()


def test_binding_refuses_what_does_not_fit():
    k = torch.zeros(2, 4, 128)
    pool = torch.zeros((3, 4, 16, 80), dtype=torch.uint8)
    with pytest.raises(pkv.PagedKVError):                    # CPU tensors
        pkv.paged_kv4_append(k, k, torch.zeros(2, dtype=torch.int64), pool, pool)
    with pytest.raises(pkv.PagedKVError):
        pkv.paged_kv4_expand(torch.zeros((1, 2), dtype=torch.int64), pool, pool, torch.zeros(3, 4, 16, 128),
                             torch.zeros(3, 4, 16, 128))


def test_decode_checks(lib):
    d = desc()

    def run(d=d, q=A, q_dtype=pkv.BF16, kc=A, vc=A, tables=A, width=256, lens=A, S=4, Hq=32, L=4096, scale=0.1, out=A,
            out_dtype=pkv.BF16, ws=A, nbytes=1 << 30):
        return lib.paged_attention_decode_kv4(q, q_dtype, kc, vc, tables, width, lens, S, Hq, L, scale, out, out_dtype, ws,
                                              nbytes, ctypes.byref(d), None)

    assert run(S=0) == 0
    for bad in (dict(q=None), dict(kc=None), dict(vc=None), dict(tables=None), dict(lens=None), dict(out=None)):
        assert run(**bad) == 1
    for bad in (dict(q=ODD), dict(kc=ODD), dict(vc=ODD), dict(out=ODD)):
        assert run(**bad) == 1 and b"aligned" in lib.paged_kv_last_error()
    assert run(d=desc(dtype=pkv.BF16)) == 2
    assert run(Hq=8 * 17) == 2 and run(Hq=30) == 1 and run(Hq=0) == 1
    assert run(q_dtype=pkv.KV4) == 2 and run(q_dtype=7) == 2
    assert run(out_dtype=pkv.F16) == 2 and run(out_dtype=pkv.KV4) == 2
    assert run(S=-1) == 1 and run(S=65536) == 1 and run(L=-1) == 1
    assert run(width=255) == 1 and b"max_blocks_per_seq" in lib.paged_kv_last_error()
    assert run(scale=float("nan")) == 1 and run(scale=float("inf")) == 1
    need = lib.paged_attention_decode_kv4_workspace_bytes(4, 32, 4096, pkv.BF16, ctypes.byref(d))
    assert 0 < need < 32 << 20
    assert run(ws=None) == 3 and run(nbytes=need - 1) == 3 and run(ws=ctypes.c_void_p(0x10080)) == 1
    big = lib.paged_attention_decode_kv4_workspace_bytes(512, 32, 1 << 20, pkv.BF16, ctypes.byref(d))
    assert big == lib.paged_attention_decode_kv4_workspace_bytes(64, 32, 1 << 18, pkv.BF16, ctypes.byref(d)) < 32 << 20
    assert lib.paged_attention_decode_kv4_workspace_bytes(4, 32, 64, pkv.BF16, ctypes.byref(d)) == 0    # no split
    assert lib.paged_attention_decode_kv4_workspace_bytes(4, 32, 512, pkv.BF16, ctypes.byref(d)) == 0
    assert lib.paged_attention_decode_kv4_workspace_bytes(4, 32, 513, pkv.BF16, ctypes.byref(d)) > 0
    assert lib.paged_attention_decode_kv4_workspace_bytes(512, 32, 512, pkv.BF16, ctypes.byref(d)) > 0
    assert lib.paged_attention_decode_kv4_workspace_bytes(4, 30, 4096, pkv.BF16, ctypes.byref(d)) == 0  # invalid
    assert run(L=(1 << 30) + 1, width=1 << 30) == 2
    assert run(L=1 << 30, S=65535, d=desc(num_kv_heads=65535, head_dim=64, block_size=8), Hq=65535, width=1 << 30) == 2
