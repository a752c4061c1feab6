"""Attention of drafted tokens where rows, sequences and waits fail or hold nothing: what the other rows, sequences
and calls then get."""
import time

import numpy as np
import pytest
import torch

import paged_kv_cache_159_gb300 as pkv
from tests import _drafts as T

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    return pkv.lib()


def odd_queries(c, rows):
    """NaN, an infinity in one place and infinities in all places, in turn."""
    for i, r in enumerate(rows):
        if i % 3 == 1:
            c.q[r, :, 5] = float("inf")
        else:
            c.q[r] = float("nan") if i % 3 == 0 else -float("inf")


# (rows a KV head, and whether the tables make it a call of few tiles: units of 16 and 32 rows, and of 256)
UNITS = [(2, 3, 0), (8, 7, 0), (8, 30, 0), (8, 30, 1000), (32, 30, 1000), (18, 30, 1000)]


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int4"])
@pytest.mark.parametrize("Hq,new,width", UNITS)
def test_a_query_that_is_not_finite_and_sees_nothing_is_zero(kind, Hq, new, width):
    """A draft slot that is not in use: an empty mask, no context, and whatever q holds."""
    c = T.Case([0, 333], [new, 9], Hq, 2, 128, kind, seed=11, width=width)
    off = [1] if new == 3 else [1, 3, 6]
    c.drafts[0][off] = False
    c.see[0] = T.visible(0, new, 0, 0, c.drafts[0])
    odd_queries(c, off)
    seeing = new + 4
    c.q[seeing, 1] = float("nan")                                       # and one that sees its ancestors
    out = c.run()
    c.check(out)
    assert (out[off] == 0).all() and torch.isnan(out[seeing, 1].float()).all()


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int4"])
@pytest.mark.parametrize("Hq,new,width", UNITS)
@pytest.mark.parametrize("cached", [0, 40, 3000])
def test_a_query_that_is_not_finite_without_any_block_is_zero(kind, Hq, new, width, cached):
    """Every entry of a sequence's table is empty: flagged, and its rows are zeros whatever q holds, also where the
    unit is cut over several CTAs."""
    c = T.Case([cached, 100], [new, 4], Hq, 2, 128, kind, seed=12, width=width).attach()
    want = c.run()[new:c.T]
    odd_queries(c, range(new))
    c.qd.copy_(c.q)
    c.bt[0] = -1
    out = c.run(error=(pkv.ERR_DEVICE, pkv.DEVERR_BLOCK_ID))
    assert (out[:new] == 0).all() and torch.equal(out[new:c.T], want)


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int4"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new", [9, 20])
def test_a_wait_that_runs_out_behind_finished_units_ends_in_time(kind, D, new):
    """The last unit of every CTA's share gets no q, after units that did: the copies in flight are those that were
    issued, and the wait for them ends with them.  A wait gives up after 1 s.  All of a CTA's waits begin when it
    stands, some milliseconds after the launch, so that a warp that waits once more for what never comes would
    need 2 s."""
    c = T.Case(np.full(40, 1300), np.full(40, new), 64, 8, D, kind, tree=False, seed=new)       # 320 units, 152 CTAs
    want = c.run()
    assert torch.isfinite(want.float()).all()
    ws, out = c.workspace(), torch.empty_like(c.qd)
    pkv.test_expire_waits(pkv.TEST_EXPIRE_DECODE)
    try:
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        pkv.paged_attention_tree(c.pool, c.qd, c.kc, c.vc, c.bt, c.sl, c.cq, c.mk, c.max_q, c.scale, out, ws)
        assert c.pool.get_device_error() == (pkv.ERR_TIMEOUT, pkv.DEVERR_TIMEOUT)
        took = time.perf_counter() - t0
    finally:
        pkv.test_expire_waits(pkv.TEST_EXPIRE_NONE)
    assert 0.9 < took < 1.6
    assert torch.equal(c.run(ws), want)


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int4"])
@pytest.mark.parametrize("Hq,new,width", UNITS)
@pytest.mark.parametrize("cu,bad", [(lambda a, b, t: [0, a, b, t + 1], [2]), (lambda a, b, t: [-1, a, b, t], [0]),
                                    (lambda a, b, t: [0, a, b, 2 ** 31 - 1], [2]), (lambda a, b, t: [0, a, a - 1, a - 1], [1, 2]),
                                    (lambda a, b, t: [-2 ** 31, a, b, 2 ** 31 - 1], [0, 2])])
def test_a_sequence_whose_rows_are_out_of_range_is_left_alone(kind, Hq, new, width, cu, bad):
    """Rows of a sequence whose cu_q leaves 0 .. total_q, or descends, stay as they were; the others are right."""
    c = T.Case([100, 60, 700], [new, 4, 2], Hq, 2, 128, kind, seed=7, max_q=new + 4, width=width).attach()
    c.cq.copy_(torch.tensor(cu(int(c.cu[1]), int(c.cu[2]), c.T), dtype=torch.int32))
    out = c.run(error=(pkv.ERR_DEVICE, pkv.DEVERR_SEQ_LEN))
    c.check(out, skip=bad)
    for b in bad:
        assert torch.isnan(out[c.cu[b]:c.cu[b + 1]].float()).all()


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int4"])
@pytest.mark.parametrize("Hq,Hkv,most", [(2, 1, 6), (4, 2, 3), (8, 1, 21)])
@pytest.mark.parametrize("batch,active", [(4096, 1.0), (4096, 0.01), (2500, 0.5), (4095, 0.0)])
def test_batches_of_thousands(kind, Hq, Hkv, most, batch, active):
    """Several sequences a thread in the split of the work, and long runs of slots without rows, whose lengths mean
    nothing."""
    rng = np.random.default_rng(batch + most)
    new = np.where(rng.random(batch) < active, rng.integers(1, most + 1, batch), 0)
    cached = rng.integers(0, 40, batch) * (rng.random(batch) < 0.5)
    new[[7, batch - 1]], cached[[7, batch - 1]] = [most, 1], [900, 333]         # one long, and the last slot
    c = T.Case(cached, new, Hq, Hkv, 64, kind, seed=13, pad=5, max_q=most).attach()
    c.sl[torch.from_numpy(new == 0).cuda()] = -3
    out = c.run()
    c.check(out)
    assert torch.equal(c.run()[:c.T], out[:c.T])


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int4"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("group", [3, 5, 6, 7, 9, 10, 11, 12, 13, 14, 15])
def test_groups_whose_units_are_not_256_rows(kind, D, group):
    """Several units a KV head, with q-tiles that end inside a token's heads."""
    tokens = 256 // group // 8 * 8
    c = T.Case([130, 5, 40], [2 * tokens + 3, 128 // group + 1, tokens], 2 * group, 2, D, kind, seed=group, width=400, max_q=2 * tokens + 3)
    c.check(c.run())
