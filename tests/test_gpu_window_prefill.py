"""Prefill and chunked prefill with a sliding window and sinks, against the definition in 64 bits."""
import numpy as np
import pytest
import torch

import paged_kv_cache_159_gb300 as pkv
from tests import _drafts as T

pytestmark = pytest.mark.gpu
P_BITS = {"bf16": 8, "fp8": 11, "int4": 11}


@pytest.fixture(scope="module", autouse=True)
def lib():
    return pkv.lib()


def prefill(c, error=(pkv.OK, 0), window=None, sinks=None, plan=None):
    c.attach()
    W, S = c.window if window is None else window, c.sinks if sinks is None else sinks
    plan, grid = plan or pkv.prefill_plan(c.pool, c.cu, c.L, c.Hq, c.MB, window=W, sinks=S)
    out = torch.full_like(c.qd, float("nan"))
    n = pkv.prefill_workspace_bytes(c.pool, c.cu, c.L, c.MB, window=W, sinks=S)
    assert (n > 0) == (c.kind == "int4")
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") if n else None
    pkv.paged_prefill(c.pool, c.qd, c.kc, c.vc, c.bt, c.scale, T.dev(plan), grid, out, workspace=ws)
    assert c.pool.get_device_error() == error
    return out


def case(cached, new, *args, **kw):
    return T.Case(cached, new, *args, tree=False, **kw)


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int4"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(2, 2), (8, 2), (14, 2), (16, 1)])
def test_heads_and_types(kind, D, Hq, Hkv):
    c = case([0, 333, 64, 900], [70, 40, 1, 130], Hq, Hkv, D, kind, window=100, sinks=4, seed=Hq)
    c.check(prefill(c), p_bits=P_BITS[kind])


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int4"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (15, 16), (16, 0), (17, 15), (63, 2), (64, 64), (65, 100), (128, 63), (129, 65), (300, 0), (1000, 200), (5000, 7), (50, 2 ** 31 - 1)])
def test_windows_and_sinks_at_block_and_tile_edges(kind, window, sinks):
    c = case([0, 63, 64, 65, 700], [200, 65, 64, 17, 150], 8, 2, 128, kind, window=window, sinks=sinks, seed=window)
    c.check(prefill(c), p_bits=P_BITS[kind])


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int4"])
@pytest.mark.parametrize("scale", [-0.09, 0.0])
def test_scales_of_any_sign(kind, scale):
    c = case([0, 300], [90, 70], 8, 2, 64, kind, window=50, sinks=3, scale=scale, seed=3)
    c.check(prefill(c), p_bits=P_BITS[kind])


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int4"])
def test_empty_chunks_and_long_contexts(kind):
    c = case([500, 3000, 0, 2000], [0, 33, 1, 0], 8, 2, 128, kind, window=600, sinks=20, seed=5)
    c.check(prefill(c), p_bits=P_BITS[kind])


@pytest.mark.parametrize("kind", ["bf16", "int4"])
def test_no_window_is_the_plain_prefill(kind):
    c = case([0, 333], [170, 40], 8, 2, 128, kind, seed=4)
    want = prefill(c, window=0)
    plain, grid = pkv.prefill_plan(c.pool, c.cu, c.L, c.Hq, c.MB)
    assert torch.equal(prefill(c, plan=(plain, grid)), want)
    assert torch.equal(prefill(c, window=373, sinks=9), want) and torch.equal(prefill(c, window=2 ** 31 - 1, sinks=2 ** 31 - 1), want)
    c.check(want, p_bits=P_BITS[kind])


def test_a_token_at_a_time_is_the_windowed_decode():
    c = case([100, 41, 0], [1, 1, 1], 8, 2, 128, "bf16", window=40, sinks=5, seed=6)
    a = prefill(c)
    b = torch.empty_like(a)
    ws = torch.empty(pkv.tree_workspace_bytes(c.pool, 3, 8), dtype=torch.uint8, device="cuda")
    pkv.paged_attention_window(c.pool, c.qd, c.kc, c.vc, c.bt, c.sl, c.scale, 40, 5, b, ws)
    c.check(a, p_bits=8), c.check(b)


def test_refusals_and_plans_that_do_not_match():
    c = case([100, 60], [30, 4], 8, 2, 128, "int4", window=20, sinks=2, free=False).attach()
    for kw in (dict(window=-1), dict(window=4, sinks=-1)):
        with pytest.raises(pkv.PkvError) as e:
            pkv.prefill_plan(c.pool, c.cu, c.L, c.Hq, c.MB, **kw)
        assert e.value.status == pkv.ERR_INVALID
        assert pkv.prefill_workspace_bytes(c.pool, c.cu, c.L, c.MB, **kw) == 0
    plan, grid = pkv.prefill_plan(c.pool, c.cu, c.L, c.Hq, c.MB, window=20, sinks=2)
    plain, flat = pkv.prefill_plan(c.pool, c.cu, c.L, c.Hq, c.MB)
    # the grid of one with the bytes of the other
    for pair in ((plan, grid & 0xFFFF), (plain, flat | (grid & ~0xFFFF))):
        prefill(c, plan=pair, window=0, error=(pkv.ERR_DEVICE, pkv.DEVERR_PLAN))
    # a plain plan in a window's workspace
    out, ws = torch.empty_like(c.qd), torch.empty(pkv.prefill_workspace_bytes(c.pool, c.cu, c.L, c.MB, window=20, sinks=2), dtype=torch.uint8, device="cuda")
    pkv.paged_prefill(c.pool, c.qd, c.kc, c.vc, c.bt, c.scale, T.dev(plain), flat, out, workspace=ws)
    assert c.pool.get_device_error() == (pkv.ERR_DEVICE, pkv.DEVERR_PLAN)
    c.check(prefill(c), p_bits=11)


def test_an_entry_that_is_needed_is_flagged():
    c = case([100, 60], [30, 4], 8, 2, 128, "bf16", window=40, sinks=2).attach()
    want = prefill(c)
    c.bt[0, 5] = -1
    out = prefill(c, error=(pkv.ERR_DEVICE, pkv.DEVERR_BLOCK_ID))
    assert torch.equal(out[30:], want[30:])


def test_the_whole_chunked_workload_in_a_window():
    rng = np.random.default_rng(7)
    c = case(rng.integers(0, 8192, 6), [512] * 6, 32, 8, 128, "bf16", window=1024, sinks=4, seed=8)
    out = prefill(c)
    keep = rng.choice(6 * 512, 40, replace=False)                # sampled rows
    q, got = c.q.double().numpy(), out.float().cpu().double().numpy()
    for r in keep:
        b, i = r // 512, r % 512
        pos = np.flatnonzero(c.see[b][i])
        k, v = c.pages.read(c.slots(b, pos))
        for h in range(0, 32, 5):
            s = c.scale * (k[:, h // 4] @ q[r, h])
            p = np.exp(s - s.max())
            p /= p.sum()
            ref, mag = p @ v[:, h // 4], p @ np.abs(v[:, h // 4])
            assert (np.abs(got[r, h] - ref) <= 2.0 ** -8 * np.abs(ref) + mag * (2.0 ** -8 + 2.0 ** -10)).all()
