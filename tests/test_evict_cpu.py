"""Eviction without a GPU: the block manager's compaction against the plain-Python model, the
selection rule's model on hand-worked rows, and the calls' argument checks."""
import ctypes
import random

import pytest

import kv4_model as model
import paged_kv_cache_310_gb300 as pkv
from oracle.block_manager_model import BlockManagerModel, OutOfBlocks
from paged_kv_cache_310_gb300 import PagedKVError, _build
from paged_kv_cache_310_gb300.block_manager import BlockManager


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()


A = ctypes.c_void_p(0x10000)
B = ctypes.c_void_p(0x10000000)
ODD = ctypes.c_void_p(0x10008)


def desc(num_blocks=64, block_size=16, num_kv_heads=8, head_dim=128, dtype=pkv.BF16):
    return pkv.CacheDesc(num_blocks, block_size, num_kv_heads, head_dim, dtype)


def test_selection_rule_by_hand():
    nan, inf = float("nan"), float("inf")
    w = [3, 1, 3, 2, 0, 9]
    assert model.kept_rows(w, 6, 3, 0) == [0, 2, 5]
    assert model.kept_rows(w, 6, 3, 1) == [0, 2, 5]
    assert model.kept_rows(w, 6, 3, 2) == [0, 4, 5]          # ties: the lowest row
    assert model.kept_rows(w, 6, 3, 9) == [3, 4, 5]          # recent beyond keep
    assert model.kept_rows(w, 6, 0, 9) == [] and model.kept_rows(w, 0, 3, 1) == []
    assert model.kept_rows(w, 6, 10, 1) == list(range(6))
    assert model.kept_rows([nan, -inf, 0.0, -0.0, inf], 5, 3, 0) == [2, 3, 4]
    assert model.kept_rows([nan, -inf, nan], 3, 2, 0) == [0, 1]


def same_state(bm, ref):
    ids = sorted(ref.tables)
    if ids:
        mb = max(len(t) for t in ref.tables.values()) or 1
        tables, lens = bm.block_tables(ids, max_blocks=mb)
        for i, s in enumerate(ids):
            assert tables[i].tolist() == ref.tables[s] + [-1] * (mb - len(ref.tables[s]))
            assert int(lens[i]) == ref.lens[s]
    assert bm.stats() == ref.stats()


@pytest.mark.parametrize("seed", range(4))
def test_compact_matches_the_model(seed):
    rng = random.Random(310_950 + seed)
    bs, nb = rng.choice([1, 4, 16]), rng.randint(10, 60)
    bm, ref = BlockManager(nb, bs), BlockManagerModel(nb, bs)
    next_id = compacted = 0
    for _ in range(300):
        live = sorted(ref.tables)
        op = rng.random()
        if op < 0.25 or not live:
            n = rng.randint(0, 4 * bs)
            if -(-n // bs) <= len(ref.free):
                ref.add_sequence(next_id, n)
                bm.add_sequence(next_id, n)
                next_id += 1
        elif op < 0.4:
            parent = rng.choice(live)
            ref.fork(parent, next_id)
            bm.fork(parent, next_id)
            next_id += 1
        elif op < 0.55:
            s = rng.choice(live)
            ref.free_sequence(s)
            bm.free_sequence(s)
        else:
            ids = rng.sample(live, min(len(live), rng.randint(1, 3)))
            old = {b for s in ids for b in ref.tables[s]}
            lens = [rng.randint(0, ref.lens[s]) for s in ids]
            try:
                want = ref.compact(ids, lens)
            except OutOfBlocks:
                before = bm.stats()
                with pytest.raises(PagedKVError) as e:
                    bm.compact(ids, lens)
                assert e.value.status == 7 and bm.stats() == before
            else:
                got = bm.compact(ids, lens)
                # no fresh block is one that an eviction of these sequences reads
                assert got == want and not {b for x in got for b in x} & old
                compacted += 1
        same_state(bm, ref)
    assert compacted > 20


def test_compact_refusals():
    bm = BlockManager(8, 4)
    bm.add_sequence(1, 10)
    bm.add_sequence(2, 5)

    def state():
        return bm.stats(), [x.tolist() for x in bm.block_tables([1, 2])]

    before = state()
    for args in (([3], [1]), ([1], [11]), ([1], [-1]), ([1, 2], [4, 6]), ([2, 1, 2], [1, 1, 1]), ([1, 3], [1, 1]), ([1], [1, 1])):
        with pytest.raises(PagedKVError) as e:
            bm.compact(*args)
        assert e.value.status == 1 and state() == before
    with pytest.raises(PagedKVError) as e:
        bm.compact([1, 2], [9, 5])                            # five fresh blocks, three free
    assert e.value.status == 7 and state() == before
    lib, n = pkv.library(), ctypes.c_int32(0)
    out = (ctypes.c_int32 * 8)()
    ids, lens = (ctypes.c_int64 * 2)(1, 2), (ctypes.c_int64 * 2)(5, 4)
    assert lib.pkv_bm_compact(None, ids, lens, 2, out, 8, ctypes.byref(n)) == 1
    assert lib.pkv_bm_compact(bm._h, None, lens, 2, out, 8, ctypes.byref(n)) == 1
    assert lib.pkv_bm_compact(bm._h, ids, None, 2, out, 8, ctypes.byref(n)) == 1
    assert lib.pkv_bm_compact(bm._h, ids, lens, -1, out, 8, ctypes.byref(n)) == 1
    assert lib.pkv_bm_compact(bm._h, ids, lens, 2, out, 2, ctypes.byref(n)) == 1     # three blocks wanted
    assert lib.pkv_bm_compact(bm._h, ids, lens, 2, None, 8, ctypes.byref(n)) == 1
    assert lib.pkv_bm_compact(bm._h, ids, lens, 2, out, 8, None) == 1
    assert state() == before
    assert bm.compact([], []) == [] and state() == before
    none = (ctypes.c_int64 * 2)(0, 0)
    assert lib.pkv_bm_compact(bm._h, ids, none, 2, None, 0, ctypes.byref(n)) == 0 and n.value == 0
    assert bm.stats()["free_blocks"] == 8


def test_weights_checks():
    lib, d = pkv.library(), desc()

    def run(d=d, q=A, q_dtype=None, kc=A, tables=A, width=256, lens=A, tracked=None, S=4, Hq=32, L=4096, scale=0.1, w=A,
            out=A, wwidth=4096, ws=A, nbytes=1 << 40):
        return lib.paged_attention_weights(q, d.dtype if q_dtype is None else q_dtype, kc, tables, width, lens, tracked, S,
                                           Hq, L, scale, w, out, wwidth, ws, nbytes, ctypes.byref(d), None)

    assert run(S=0) == 0 and run(L=0) == 0
    for bad in (dict(q=None), dict(kc=None), dict(tables=None), dict(lens=None), dict(w=None), dict(out=None)):
        assert run(**bad) == 1
    assert run(q=ODD) == 1 and run(kc=ODD) == 1 and run(w=ctypes.c_void_p(0x10002)) == 1
    assert run(Hq=8 * 17) == 2 and run(Hq=30) == 1 and run(S=65536) == 1 and run(L=-1) == 1
    assert run(L=(1 << 30) + 1) == 2
    assert run(q_dtype=pkv.F16) == 1                          # not the cache's
    assert run(q_dtype=9) == 2 and run(d=desc(dtype=pkv.KV4), q_dtype=pkv.KV4) == 2
    assert run(width=255) == 1 and run(wwidth=4095) == 1 and run(scale=float("inf")) == 1
    size = 4 * 8 * 4096 * 4                                   # in place or apart, not in between
    for off in (4, size - 4):
        assert run(out=ctypes.c_void_p(0x10000 + off)) == 1 and b"overlap" in lib.paged_kv_last_error()
        assert run(w=ctypes.c_void_p(0x10000 + off)) == 1
    assert run(out=ctypes.c_void_p(0x10000 + size), ws=None) == 3
    need = lib.paged_attention_weights_workspace_bytes(4, 32, 4096, ctypes.byref(d))
    assert need >= 4 * 32 * 4096 * 4
    assert run(ws=None) == 3 and run(nbytes=need - 1) == 3 and run(ws=ctypes.c_void_p(0x10080)) == 1
    assert lib.paged_attention_weights_workspace_bytes(4, 30, 4096, ctypes.byref(d)) == 0


def test_evict_checks():
    lib, d = pkv.library(), desc()

    def run(d=d, w=A, out=B, wwidth=4096, tables=A, width=256, lens=A, keep=A, recent=0, new=A, new_width=64, S=4, L=4096,
            max_keep=1024, kept=A, kc=A, vc=A):
        return lib.paged_kv_evict(w, out, wwidth, tables, width, lens, keep, recent, new, new_width, S, L, max_keep, kept, kc,
                                  vc, ctypes.byref(d), None)

    assert run(S=0) == 0 and run(L=0) == 0
    for name in ("w", "out", "tables", "lens", "keep", "new", "kept", "kc", "vc"):
        assert run(**{name: None}) == 1
    assert run(kc=ODD) == 1 and run(vc=ODD) == 1
    assert run(out=A) == 1 and b"overlap" in lib.paged_kv_last_error()
    assert run(out=ctypes.c_void_p(0x10000 + 4 * 8 * 4096 * 4 - 4)) == 1
    assert run(recent=-1) == 1 and run(max_keep=-1) == 1 and run(L=-1) == 1 and run(S=65536) == 1
    assert run(wwidth=4095) == 1 and run(width=255) == 1 and run(new_width=63) == 1
    assert run(L=(1 << 30) + 1) == 2 and run(d=desc(dtype=7)) == 2 and run(d=desc(block_size=12)) == 2
