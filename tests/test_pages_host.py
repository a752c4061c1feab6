"""Forking sequences and compacting a pool: the host bookkeeping."""
import numpy as np
import pytest

pkv = pytest.importorskip("paged_kv_cache_159_gb300")


@pytest.fixture(scope="module", autouse=True)
def lib():
    from paged_kv_cache_159_gb300 import build
    build.build()
    return pkv.lib()


def _refs(p):
    return [p.refcount(i) for i in range(p.desc.num_blocks)]


@pytest.mark.parametrize("L,shared,copies", [(1, 0, 3), (15, 0, 3), (16, 1, 0), (17, 1, 3), (40, 2, 3), (48, 3, 0)])
def test_fork_shares_full_blocks_and_copies_the_partial_one(L, shared, copies):
    p = pkv.Pool(20, 1, 64, free_order=list(range(19, -1, -1)))
    row = p.build_block_tables([L], 5)[0]
    before = p.num_free()
    t, pairs = p.fork(row, L, 3)
    nb = -(-L // 16)
    assert t.shape == (3, 5) and (t[:, :shared] == row[:shared]).all() and (t[:, nb:] == -1).all()
    assert len(pairs) == copies and p.num_free() == before - copies
    for j in range(shared):
        assert p.refcount(int(row[j])) == 4
    if copies:
        assert (pairs[:, 0] == row[shared]).all() and pairs[:, 1].tolist() == t[:, shared].tolist()
        assert p.refcount(int(row[shared])) == 1 and [p.refcount(int(i)) for i in pairs[:, 1]] == [1, 1, 1]
        assert len(set(pairs[:, 1].tolist())) == 3
    # the forks append without a copy
    new = np.concatenate([row[None], t])
    if L % 16:
        again, more = p.cow_prepare(new, [L + 1] * 4)
        assert len(more) == 0 and np.array_equal(again, new)
    for r in new:
        p.free(r[r >= 0])
    assert p.num_free() == 20 and not any(_refs(p))


def test_fork_refusals_change_nothing():
    p = pkv.Pool(4, 1, 64)
    row = p.build_block_tables([40], 3)[0]
    refs = _refs(p)
    for args, st in (((row, 0, 1), pkv.ERR_INVALID), ((row, 49, 1), pkv.ERR_INVALID), ((row, 40, -1), None), ((row, 40, 2), pkv.ERR_OOM),
                     (([0, 1, 3], 40, 1), pkv.ERR_INVALID), (([0, -1, 2], 40, 1), pkv.ERR_INVALID), (([0, 1, 4], 40, 1), pkv.ERR_INVALID)):
        with pytest.raises((pkv.PkvError, ValueError)) as e:
            p.fork(*args)
        assert st is None or e.value.status == st
        assert _refs(p) == refs and p.num_free() == 1
    t, pairs = p.fork(row, 40, 0)
    assert t.shape == (0, 3) and len(pairs) == 0


def test_compact_by_hand():
    p = pkv.Pool(10, 1, 64)
    p.alloc(8)
    p.share([7, 2])
    p.free([1, 3, 4])                                   # live: 0 2 5 6 7, free list 8 9 1 3 4
    assert p.compact(1).tolist() == [[7, 1]]
    assert _refs(p) == [1, 2, 2, 0, 0, 1, 1, 0, 0, 0]
    assert p.compact().tolist() == [[6, 3], [5, 4]]
    assert _refs(p) == [1, 2, 2, 1, 1, 0, 0, 0, 0, 0]
    assert p.compact().tolist() == [] and p.compact(0).tolist() == []
    assert p.alloc(5).tolist() == [8, 9, 7, 6, 5]
    t = np.array([[0, 2, 7, -1], [6, 5, 8, 9]], np.int32)
    assert pkv.remap_tables(t, [[7, 1], [6, 3], [5, 4]]).tolist() == [[0, 2, 1, -1], [3, 4, 8, 9]]
    with pytest.raises(pkv.PkvError):
        pkv.remap_tables(t, [[5, 4], [7, 1]])           # not descending
    assert np.array_equal(pkv.remap_tables(t, np.zeros((0, 2), np.int32)), t)


@pytest.mark.parametrize("seed", range(6))
def test_compact_against_a_plain_model(seed):
    rng = np.random.default_rng(seed)
    n = int(rng.integers(1, 60))
    p = pkv.Pool(n, 2, 128, free_order=rng.permutation(n))
    held = p.alloc(int(rng.integers(0, n + 1))).tolist()
    drop = [i for i in held if rng.random() < 0.5]
    p.free(drop)
    live = sorted(set(held) - set(drop))
    free = [i for i in range(n) if i not in live]
    moves, limit = p.compact(), []
    while live and free and max(live) > min(free):
        s, d = max(live), min(free)
        limit.append([s, d])
        live.remove(s), free.remove(d)
        live.append(d), free.append(s)
    assert moves.tolist() == limit
    refs = _refs(p)
    assert refs == [1] * len(live) + [0] * (n - len(live)) and p.num_free() == n - len(live)
    got = p.alloc(p.num_free()).tolist()
    assert sorted(got) == list(range(len(live), n))


def test_cached_prefixes_follow_their_blocks():
    p = pkv.Pool(12, 1, 64, free_order=list(range(11, -1, -1)))
    toks = np.arange(64, dtype=np.int32)
    other = np.concatenate([toks[:32], 1000 + toks[:16]]).astype(np.int32)
    a = p.build_block_tables([64], 4)[0]                # blocks 11 10 9 8
    assert p.prefix_insert(toks, 5, a) == 4
    hit = p.prefix_lookup(other, 5)
    b = p.build_block_tables([48], 3, hit)[0]           # 11 10 7
    assert p.prefix_insert(other, 5, b) == 1
    p.free(a), p.free(b)
    assert p.prefix_cached_blocks() == 5 and p.num_free() == 7
    moves = p.compact()
    assert moves.tolist() == [[11, 0], [10, 1], [9, 2], [8, 3], [7, 4]]
    assert p.prefix_lookup(toks, 5).tolist() == [0, 1, 2, 3]
    assert p.prefix_lookup(other, 5).tolist() == [0, 1, 4]
    assert _refs(p) == [1] * 5 + [0] * 7
    p.prefix_lookup(toks, 5)                            # the other leaf is the least recently used
    assert p.prefix_evict(2).tolist() == [4, 3]
    assert p.prefix_insert(toks, 5, np.concatenate([p.prefix_lookup(toks, 5), p.alloc(1)])) == 1
    p.prefix_clear()
    assert p.prefix_cached_blocks() == 0


def test_null_and_negative_arguments():
    import ctypes
    L, P = pkv.lib(), ctypes.c_void_p
    p = pkv.Pool(4, 1, 64)
    n = ctypes.c_int32()
    buf = np.zeros(4, np.int32)
    b = buf.ctypes.data_as(P)
    assert L.pkv_pool_compact(None, 4, b, b, ctypes.byref(n)) == pkv.ERR_INVALID
    assert L.pkv_pool_compact(p.handle, -1, b, b, ctypes.byref(n)) == pkv.ERR_INVALID
    assert L.pkv_pool_compact(p.handle, 4, None, b, ctypes.byref(n)) == pkv.ERR_INVALID
    assert L.pkv_pool_compact(p.handle, 0, None, None, ctypes.byref(n)) == pkv.OK and n.value == 0
    assert L.pkv_remap_tables(b, -1, b, b, 0) == pkv.ERR_INVALID
    assert L.pkv_remap_tables(None, 4, None, None, 0) == pkv.ERR_INVALID
    assert L.pkv_fork_tables(p.handle, None, 4, 1, 2, b, b, b, ctypes.byref(n)) == pkv.ERR_INVALID
