"""Moving blocks on the device, and a pool's whole life over every type: prompts, prefill, decode
steps, forks, freeing, compaction."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import int4 as O
from tests import _int4 as I

pkv = pytest.importorskip("paged_kv_cache_159_gb300")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    pkv.lib()
    torch.cuda.set_device(0)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("kv,D,Hkv,layers,NB,moves", [(pkv.KV_BF16, 64, 1, 1, 4, 1), (pkv.KV_BF16, 128, 8, 3, 40, 17), (pkv.KV_FP8E4M3, 64, 3, 2, 9, 4),
                                                      (pkv.KV_INT4, 64, 1, 1, 3, 1), (pkv.KV_INT4, 64, 3, 5, 300, 150), (pkv.KV_INT4, 128, 8, 2, 64, 31)])
def test_moves_every_layer_and_the_tables(kv, D, Hkv, layers, NB, moves):
    rng = np.random.default_rng(NB)
    pool = pkv.Pool(NB, Hkv, D, kv, num_layers=layers)
    pool.attach_device(0)
    caches = [torch.from_numpy(rng.integers(0, 256, (layers, NB, Hkv * pool.tile_bytes())).astype(np.uint8)).cuda() for _ in range(2)]
    held = pool.alloc(NB)
    pool.free(rng.permutation(held)[:moves])
    live = [i for i in range(NB) if pool.refcount(i)]
    tables = rng.choice(live, (7, 13)).astype(np.int32)
    tables[rng.random(tables.shape) < 0.2] = -1
    tables[0, 0], tables[1, 1] = NB + 5, -9                # entries that name no block stay
    m = pool.compact()
    want = [c.clone() for c in caches]
    for s, d in m.tolist():
        for w in want:
            w[:, d] = w[:, s]
    bt = torch.from_numpy(tables).cuda()
    pkv.move_blocks(pool, *caches, _i32(m[:, 0]), _i32(m[:, 1]), bt)
    assert pool.get_device_error() == (pkv.OK, 0)
    assert all(torch.equal(a, b) for a, b in zip(caches, want))
    new = pkv.remap_tables(tables, m)
    assert np.array_equal(bt.cpu().numpy(), new)
    pkv.move_blocks(pool, *caches, _i32(m[:, 0]), _i32(m[:, 1]), bt)          # again: nothing changes
    assert all(torch.equal(a, b) for a, b in zip(caches, want)) and np.array_equal(bt.cpu().numpy(), new)
    pkv.move_blocks(pool, *caches, _i32([]), _i32([]), bt)
    pkv.move_blocks(pool, *caches, _i32(m[:, 0]), _i32(m[:, 1]))               # without tables
    assert all(torch.equal(a, b) for a, b in zip(caches, want))


def test_ids_outside_the_pool_are_flagged_and_skipped():
    pool = pkv.Pool(5, 1, 64)
    pool.attach_device(0)
    kc, vc = (torch.randn(5, 1, 16, 64, device="cuda").bfloat16() for _ in range(2))
    k0, v0 = kc.clone(), vc.clone()
    bt = _i32([[7, 4, 3, -1]])
    pkv.move_blocks(pool, kc, vc, _i32([7, 4, 3]), _i32([0, 1, -2]), bt)
    assert pool.get_device_error() == (pkv.ERR_DEVICE, pkv.DEVERR_BLOCK_ID)
    k0[1], v0[1] = k0[4], v0[4]
    assert torch.equal(kc, k0) and torch.equal(vc, v0) and bt.tolist() == [[7, 1, 3, -1]]


def test_move_refusals():
    pool = pkv.Pool(5, 1, 64)
    L, P = pkv.lib(), ctypes.c_void_p
    x = torch.zeros(5 * 1024, dtype=torch.bfloat16, device="cuda")
    ids = _i32([4, 3])
    ok = [pool.handle, P(x.data_ptr()), P(x.data_ptr()), P(ids.data_ptr()), P(ids.data_ptr()), 1, P(0), 0, P(0)]
    assert L.pkv_move_blocks(*ok) == pkv.ERR_INVALID                            # not attached
    pool.attach_device(0)
    for i, bad in ((0, None), (1, None), (1, P(x.data_ptr() + 2)), (2, P(x.data_ptr() + 8)), (3, None), (3, P(ids.data_ptr() + 2)), (4, None), (5, -1),
                   (7, 3), (7, -1)):
        args = list(ok)
        args[i] = bad
        assert L.pkv_move_blocks(*args) == pkv.ERR_INVALID, (i, bad)
    ok[5] = 0
    assert L.pkv_move_blocks(*ok) == pkv.OK


@pytest.mark.parametrize("kv", [pkv.KV_BF16, pkv.KV_FP8E4M3, pkv.KV_INT4])
def test_a_pools_life(kv):
    """Prompts, decode steps, a fork, a finished sequence, a compaction, more steps: the attention
    outputs are those of a pool that was never forked or compacted."""
    Hq, Hkv, D, NB, MB = 8, 2, 128, 40, 12
    scale = float(np.float32(1 / np.sqrt(D)))
    g = torch.Generator(device="cuda").manual_seed(kv)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    ks, vs = (1.0, 1.0) if kv == pkv.KV_BF16 else (0.02, 0.02)

    def new_pool(order):
        p = pkv.Pool(NB, Hkv, D, kv, ks, vs, free_order=order)
        p.attach_device(0)
        shape = (NB, Hkv, p.tile_bytes()) if kv == pkv.KV_INT4 else (NB, Hkv, 16, D)
        c = [torch.zeros(shape, dtype=torch.bfloat16 if kv == pkv.KV_BF16 else torch.uint8, device="cuda") for _ in range(2)]
        return p, c

    def step(p, c, tables, lens, q, k, v):
        out = torch.empty_like(q)
        bt, sl = _i32(tables), _i32(lens)
        ws = torch.zeros(pkv.decode_workspace_bytes(p, len(lens), Hq, MB), dtype=torch.uint8, device="cuda")
        pkv.decode_step(p, q, k, v, *c, bt, sl, scale, out, ws)
        assert p.get_device_error() == (pkv.OK, 0)
        return out

    lens = np.array([37, 50, 19], np.int32)
    p, c = new_pool(np.random.default_rng(1).permutation(NB))
    tables = p.build_block_tables(lens + 20, MB)            # room for the steps below
    k, v = rnd(int(lens.sum()), Hkv, D), rnd(int(lens.sum()), Hkv, D)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    slots = torch.from_numpy(pkv.slot_mapping_chunks(tables, lens, cu)).cuda()
    pkv.kv_append(p, k, v, slots, *c)
    q = rnd(int(lens.sum()), Hq, D)
    plan, grid = pkv.prefill_plan(p, cu, lens, Hq, MB)
    n = pkv.prefill_workspace_bytes(p, cu, lens, MB)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
    out = torch.empty_like(q)
    pkv.paged_prefill(p, q, *c, _i32(tables), scale, torch.from_numpy(plan).cuda(), grid, out, workspace=ws)
    assert p.get_device_error() == (pkv.OK, 0) and bool(torch.isfinite(out).all())
    # the same history in a second pool, which stays as it is: sequence 1 three times
    p2, c2 = new_pool(None)
    lens2 = np.array([37, 50, 50, 50], np.int32)
    tables2 = p2.build_block_tables(lens2 + 20, MB)
    for row, b in enumerate((0, 1, 1, 1)):
        s = pkv.slot_mapping_all(tables2[row:row + 1], lens2[row:row + 1])
        pkv.kv_append(p2, k[cu[b]:cu[b + 1]], v[cu[b]:cu[b + 1]], torch.from_numpy(s).cuda(), *c2)
    # sequence 1 forks twice: its first 3 blocks shared, the fourth (positions 48, 49) copied
    p.free(tables[1][tables[1] >= 0][4:])
    forks, pairs = p.fork(tables[1], int(lens[1]), 2)
    assert len(pairs) == 2
    pkv.copy_blocks(p, *c, _i32(pairs[:, 0]), _i32(pairs[:, 1]))
    rows = np.concatenate([tables[:2], forks])
    rows[1, 4:] = -1
    for r in (1, 2, 3):
        rows[r, 4] = p.alloc(1)[0]
    p.free(tables[2][tables[2] >= 0])                       # sequence 2 is done
    for i in range(6):
        L = lens2 + 1 + i
        qs, kn, vn = rnd(4, Hq, D), rnd(4, Hkv, D), rnd(4, Hkv, D)
        a = step(p, c, rows, L, qs, kn, vn)
        assert torch.equal(a, step(p2, c2, tables2, L, qs, kn, vn)), i
        if i == 2:                                          # in the middle: compact
            m = p.compact()
            assert len(m) > 0
            bt = _i32(rows)
            pkv.move_blocks(p, *c, _i32(m[:, 0]), _i32(m[:, 1]), bt)
            rows = pkv.remap_tables(rows, m)
            assert np.array_equal(bt.cpu().numpy(), rows)
            assert int(rows.max()) == NB - p.num_free() - 1
    # the rows read back are the same in both pools
    got = []
    for pp, cc, tt in ((p, c, rows), (p2, c2, tables2)):
        s = torch.from_numpy(pkv.slot_mapping_all(tt, lens2 + 6)).cuda()
        o = [torch.empty(s.numel(), Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        pkv.kv_gather(pp, s, *cc, *o)
        got.append(o)
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
