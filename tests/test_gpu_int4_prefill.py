"""Prefill attention over INT4 pools against the plain implementation in 64 bits."""
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


class Chunks(I.Case):
    """A Case whose sequences' last P_b positions are the query rows."""

    def __init__(self, P, C, Hq, Hkv, D, **kw):
        super().__init__([p + c for p, c in zip(P, C)], Hq, Hkv, D, **kw)
        self.cu = np.concatenate([[0], np.cumsum(P)]).astype(np.int32)
        self.rows = torch.randn(int(self.cu[-1]), Hq, D, generator=torch.Generator().manual_seed(99)).bfloat16()
        self.host_plan, self.grid = pkv.prefill_plan(self.pool, self.cu, self.lens, Hq, self.MB)
        self.plan = I.dev(self.host_plan)
        n = pkv.prefill_workspace_bytes(self.pool, self.cu, self.lens, self.MB)
        assert n > 0
        self.ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")       # bf16 NaN throughout

    def args(self, out, ws):
        return (self.pool, self.rows.cuda(), self.kc, self.vc, self.bt, self.scale, self.plan, self.grid, out, None, ws)

    def prefill(self):
        out = torch.full(self.rows.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
        pkv.paged_prefill(*self.args(out, self.ws))
        assert self.pool.get_device_error() == (pkv.OK, 0)
        return out

    def check_rows(self, out):
        ref, mag = O.prefill(I.bits(self.rows), self.kh, self.vh, self.tables, self.lens, self.cu, self.scale, self.k_scale, self.v_scale)
        got = out.float().cpu().double().numpy()
        # bf16 roundings of the output (2^-8 of it) and of p (2^-8 of sum p |v|, the expanded rows
        # being exact), and 2^-10 of it for the scores' and the sums' fp32 arithmetic: scores here
        # stay below 2^5, off by 2^-22 of at most 128 terms each
        tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -10) * mag
        assert np.isfinite(got).all() and (np.abs(got - ref) <= tol).all(), (np.abs(got - ref) / tol).max()


@pytest.mark.parametrize("Hq,Hkv,D", [(1, 1, 128), (2, 2, 64), (8, 2, 64), (8, 2, 128), (6, 2, 128), (7, 1, 128), (16, 1, 64), (24, 8, 128)])
def test_heads_and_head_dims(Hq, Hkv, D):
    c = Chunks([40, 1, 17], [37, 0, 16], Hq, Hkv, D, seed=Hq)
    c.check_rows(c.prefill())


@pytest.mark.parametrize("P,C", [(1, 0), (15, 0), (16, 0), (17, 0), (64, 0), (65, 63), (1, 64), (63, 1), (130, 200), (2, 1000), (257, 0)])
def test_edge_lengths(P, C):
    c = Chunks([P], [C], 8, 2, 128, seed=P)
    c.check_rows(c.prefill())


@pytest.mark.parametrize("D", [64, 128])
def test_sequences_without_rows_between_others(D):
    c = Chunks([0, 33, 0, 5, 0], [20, 7, 100, 50, 1], 4, 2, D, width=9)
    a = c.prefill()
    c.check_rows(a)
    assert torch.equal(a, c.prefill())                     # the workspace's old content does not matter


def test_prefill_row_agrees_with_decode():
    """The last row of every chunk is the decode query of its sequence."""
    c = Chunks([50, 3], [100, 400], 8, 2, 128, seed=4)
    out = c.prefill()
    c.q = c.rows[torch.from_numpy(c.cu[1:].astype(np.int64) - 1)]
    ref, mag, ds = O.decode(I.bits(c.q), c.kh, c.vh, c.tables, c.lens, c.scale, c.k_scale, c.v_scale)
    I.within(c.decode(), ref, mag, ds, c.lens[:, None, None], c.v_scale)
    last = out[torch.from_numpy(c.cu[1:].astype(np.int64) - 1).cuda()].float().cpu().double().numpy()
    assert (np.abs(last - ref) <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -10) * mag).all()


def test_captured_and_replayed_with_new_queries():
    c = Chunks([70, 20], [10, 300], 8, 2, 64)
    out, q = torch.zeros_like(c.rows, device="cuda"), c.rows.cuda()
    args = list(c.args(out, c.ws))
    args[1] = q
    pkv.paged_prefill(*args)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkv.paged_prefill(*args[:9], workspace=c.ws)
    c.rows = torch.randn(c.rows.shape, generator=torch.Generator().manual_seed(5)).bfloat16()
    q.copy_(c.rows)
    g.replay()
    torch.cuda.synchronize()
    c.check_rows(out)


def test_bad_entries_and_mismatched_plans_are_flagged():
    c = Chunks([20, 30], [0, 40], 4, 2, 64)
    ref, out = c.prefill(), torch.zeros_like(c.rows, device="cuda")
    c.bt[0, 0] = -7
    pkv.paged_prefill(*c.args(out, c.ws))
    assert c.pool.get_device_error() == (pkv.ERR_DEVICE, pkv.DEVERR_BLOCK_ID)
    assert torch.equal(out[20:], ref[20:])
    c.bt[0, 0] = int(c.tables[0, 0])
    # a workspace of one block less than the plan's sequences use
    block = 2 * 2 * 16 * 64 * 2
    pkv.paged_prefill(*c.args(out, c.ws[:c.ws.numel() - block]))
    assert c.pool.get_device_error() == (pkv.ERR_DEVICE, pkv.DEVERR_PLAN)
    assert torch.equal(c.prefill(), ref)


def test_a_plan_of_other_tables_is_flagged():
    # a plan made for wider tables than the call's: nothing is read past them or written
    c = Chunks([20, 30], [0, 40], 4, 2, 64)
    narrow = c.bt[:, :2].contiguous()
    out = torch.full_like(c.rows, 7.0, device="cuda")
    args = [narrow if x is c.bt else x for x in c.args(out, c.ws)]
    pkv.paged_prefill(*args)
    assert c.pool.get_device_error() == (pkv.ERR_DEVICE, pkv.DEVERR_PLAN)
    assert bool((out == 7.0).all())


def test_refusals():
    c = Chunks([20], [0], 4, 2, 64)
    out, L, P = torch.zeros_like(c.rows, device="cuda"), pkv.lib(), ctypes.c_void_p
    for ws in (None, c.ws[:256], c.ws[16:]):
        with pytest.raises(pkv.PkvError) as e:
            pkv.paged_prefill(*c.args(out, ws))
        assert e.value.status == pkv.ERR_INVALID
    q = c.rows.cuda()
    assert L.pkv_paged_prefill(c.pool.handle, P(q.data_ptr()), P(c.kc.data_ptr()), P(c.vc.data_ptr()), P(c.bt.data_ptr()), 1, 4, c.MB, 20,
                               c.scale, P(c.plan.data_ptr()), c.grid, P(out.data_ptr()), P(0)) == pkv.ERR_INVALID
    assert pkv.prefill_workspace_bytes(c.pool, [0, 21], [20], 2) == 0                # more rows than positions
    assert pkv.prefill_workspace_bytes(c.pool, [0, 5], [40], 2) == 0                 # more blocks than a row
    assert pkv.prefill_workspace_bytes(pkv.Pool(4, 2, 64), [0, 5], [20], 2) == 0     # a bf16 pool needs none
