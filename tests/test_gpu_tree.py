"""Attention of drafted tokens (trees, chains) over every pool type, against the definition in 64 bits."""
import numpy as np
import pytest
import torch

import paged_kv_cache_159_gb300 as pkv
from oracle import int4 as O
from tests import _drafts as T

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    return pkv.lib()


@pytest.fixture(autouse=True, params=["narrow tables", "wide tables"])
def width(request, monkeypatch):
    """With narrow tables a small case has few tiles, and takes units of 32 rows whatever its drafts."""
    monkeypatch.setattr(T, "WIDTH", 1500 if request.param == "wide tables" else 0)


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int4"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,new", [(2, 2, [1, 5, 16]), (8, 2, [3, 4, 1]), (8, 2, [8, 5, 0, 7]), (14, 2, [9, 2, 8]),
                                        (32, 2, [1, 2, 3]), (8, 1, [16, 13, 1]), (15, 3, [21, 40, 3])])
def test_trees(kind, D, Hq, Hkv, new):
    cached = [0, 333, 64, 15][:len(new)]
    c = T.Case(cached, new, Hq, Hkv, D, kind, seed=D + Hq)
    c.check(c.run())


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int4"])
@pytest.mark.parametrize("cached", [0, 1, 15, 16, 17, 47, 63, 64, 65, 127, 129, 255, 1023])
def test_context_lengths_at_block_and_tile_edges(kind, cached):
    c = T.Case([cached, cached + 1], [7, 12], 8, 2, 128, kind, seed=cached)
    c.check(c.run())


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int4"])
@pytest.mark.parametrize("new", [63, 64, 65, 128, 200, 256])
def test_large_trees(kind, new):
    c = T.Case([100, 37], [new, new // 3], 8, 2, 128 if new % 2 else 64, kind, seed=new)
    c.check(c.run())


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int4"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (15, 0), (16, 4), (17, 16), (40, 17), (64, 33), (200, 5), (2000, 3), (0, 0)])
def test_chains_with_windows_and_sinks(kind, window, sinks):
    c = T.Case([0, 5, 130, 421], [9, 3, 9, 1], 8, 2, 128, kind, tree=False, window=window, sinks=sinks, seed=window)
    c.check(c.run())


@pytest.mark.parametrize("kind", ["bf16", "int4"])
@pytest.mark.parametrize("window,sinks", [(11, 0), (16, 5), (33, 40), (64, 1), (500, 16)])
def test_trees_with_windows_and_sinks(kind, window, sinks):
    c = T.Case([0, 7, 64, 333, 1000], [11, 4, 8, 2, 10], 8, 2, 64, kind, window=window, sinks=sinks, seed=window)
    c.check(c.run())


@pytest.mark.parametrize("kind,new", [("bf16", 3), ("fp8", 6), ("int4", 2), ("bf16", 30)])
def test_units_cut_over_many_ctas(kind, new):
    c = T.Case([9000, 20, 4001], [new, 1, new], 4, 1, 128, kind, seed=new)
    c.check(c.run())


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int4"])
@pytest.mark.parametrize("Hq,new,most", [(16, 40, 2500), (32, 50, 700), (8, 18, 2500)])
def test_many_tiles_and_units_a_cta(kind, Hq, new, most):
    """Every CTA goes through many units and many times around its rings; units of one and two q-tiles in turn."""
    rng = np.random.default_rng(new)
    c = T.Case(rng.integers(0, most, 30), rng.integers(0, new + 1, 30), Hq, 8, 64, kind, seed=new, max_q=new)
    out = c.run()
    c.check(out)
    assert all(torch.equal(c.run()[:c.T], out[:c.T]) for _ in range(10))


def test_many_sequences_with_empty_ones_and_padding_rows():
    rng = np.random.default_rng(3)
    new = rng.integers(0, 6, 300)
    cached = rng.integers(0, 90, 300)
    c = T.Case(cached, new, 4, 2, 64, "bf16", pad=13, seed=4)
    c.check(c.run())


@pytest.mark.parametrize("Hq", [8, 32])
def test_every_length_of_a_sequence_without_rows_is_fine(Hq):
    c = T.Case([20, 30, 40], [2, 0, 3], 4, 2, 64).attach()
    c.sl[1] = -7
    out = c.run()
    c.sl[1] = 10 ** 9
    assert torch.equal(out[:c.T], c.run()[:c.T])
    c.check(out)


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int4"])
@pytest.mark.parametrize("Hq", [8, 32])
def test_a_row_that_sees_nothing_is_zero(kind, Hq):
    c = T.Case([0, 40], [6, 5], Hq, 2, 128, kind, seed=8)
    c.drafts[0][:] = False
    c.drafts[0][2, [2]] = True
    c.see[0] = T.visible(0, 6, 0, 0, c.drafts[0])
    out = c.run()
    c.check(out)
    assert (out[[0, 1, 3, 4, 5]] == 0).all() and (out[2] != 0).any()


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int4"])
@pytest.mark.parametrize("new", [4, 8, 13, 70])
@pytest.mark.parametrize("keys", [False, True])
def test_nan_and_infinity_stay_with_the_rows_that_see_them(kind, new, keys):
    """V (and K) of one drafted token in four is not finite in a column: rows below it are not finite there (with K,
    nowhere), all others as if it were not there."""
    c = T.Case([50, 3], [new, new], 8, 2, 128, kind, seed=new)
    clean = T.Case([50, 3], [new, new], 8, 2, 128, kind, seed=new)
    ref, mag, ds = clean.reference()
    for b in range(2):
        for j in range(1, new, 4):
            s = int(c.slots(b, [c.C[b] + j])[0])
            for is_key, x in zip((True, False), c.pages.caches):
                if is_key and not keys:
                    continue
                if kind == "bf16":
                    x[s // 16, :, s % 16, 5] = 0x7F80 if j % 8 == 1 and not is_key else 0x7FC1
                elif kind == "fp8":
                    x[s // 16, :, s % 16, 5] = 0xFF
                else:
                    x[s // 16, :, O.places(128, is_key)[2][s % 16, 5]] = 0x7F
    out = c.run()[:c.T].float().cpu().numpy()
    hit = np.concatenate([c.drafts[b][:, 1:new:4].any(1) for b in range(2)])
    assert hit.any() and not hit.all()
    cols = np.arange(128) < 32 if kind == "int4" else np.arange(128) == 5
    tol = 2.0 ** -8 * np.abs(ref) + mag * (2.0 ** -8 + 2 * ds[..., None] + 2.0 ** -10)
    fine = ~hit[:, None] | (~cols[None, :] if not keys else False)
    fine = np.broadcast_to(fine[:, None, :], ref.shape)
    assert (np.abs(out - ref) <= tol)[fine].all()
    assert not np.isfinite(out[hit][..., cols]).any()


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int4"])
@pytest.mark.parametrize("scale", [-0.09, 0.0, 3.0])
@pytest.mark.parametrize("Hq", [8, 32])
def test_scales_of_any_sign(kind, scale, Hq):
    c = T.Case([70, 200], [5, 9], Hq, 2, 128, kind, scale=float(np.float32(scale)), seed=6)
    c.check(c.run())


@pytest.mark.parametrize("kind", ["fp8", "int4"])
@pytest.mark.parametrize("gain", [1e-30, 1e-3, 1e4, 1e30])
@pytest.mark.parametrize("Hq", [8, 32])
def test_queries_of_any_size_over_quantised_pools(kind, gain, Hq):
    c = T.Case([70, 20], [5, 9], Hq, 2, 128, kind, q_gain=gain, scale=float(np.float32(0.09 / gain)), seed=6)
    c.check(c.run())


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int4"])
@pytest.mark.parametrize("Hq", [8, 32])
def test_placement_changes_no_bit_and_calls_repeat(kind, Hq):
    outs = []
    for order in (1, 2):
        c = T.Case([700, 33, 2100], [9, 4, 6], Hq, 2, 128, kind, seed=5, order_seed=order)
        ws = c.attach().workspace()
        outs += [c.run(ws), c.run(ws)]
    assert all(torch.equal(outs[0][:c.T], o[:c.T]) for o in outs)


@pytest.mark.parametrize("kind", ["bf16", "int4"])
@pytest.mark.parametrize("Hq", [8, 32])
def test_an_entry_outside_the_pool_is_flagged_and_not_seen(kind, Hq):
    c = T.Case([100, 60], [3, 4], Hq, 2, 128, kind, seed=7).attach()
    want = c.run()
    bt = c.bt.clone()
    c.bt[0, 2] = c.NB
    c.bt[0, 4] = -1
    out = c.run(error=(pkv.ERR_DEVICE, pkv.DEVERR_BLOCK_ID))
    assert torch.equal(out[3:7], want[3:7])
    c.see[0][:, 32:48] = c.see[0][:, 64:80] = False
    c.check(out)
    c.bt.copy_(bt)
    assert torch.equal(c.run()[:c.T], want[:c.T])


@pytest.mark.parametrize("Hq", [8, 32])
def test_bad_lengths_are_flagged_and_their_rows_zero(Hq):
    c = T.Case([100, 60, 30, 20], [3, 4, 2, 5], Hq, 2, 128, "bf16", seed=7, max_q=8).attach()
    good = c.sl.clone()
    for b, L in ((1, 3), (1, 0), (1, -4), (2, c.MB * 16 + 1), (3, 2 ** 31 - 1)):
        c.sl.copy_(good)
        c.sl[b] = L
        out = c.run(error=(pkv.ERR_DEVICE, pkv.DEVERR_SEQ_LEN))
        assert (out[c.cu[b]:c.cu[b + 1]] == 0).all()
        c.check(out, skip=[b])
    c.sl.copy_(good)
    c.max_q = 4                                                  # the last sequence has more rows than that
    ws = c.workspace()
    out = c.run(ws, error=(pkv.ERR_DEVICE, pkv.DEVERR_SEQ_LEN))
    assert (out[9:] == 0).all()
    c.check(out, skip=[3])


@pytest.mark.parametrize("Hq", [8, 32])
def test_cu_q_out_of_range_writes_nothing_for_that_sequence(Hq):
    c = T.Case([100, 60, 30], [3, 4, 2], Hq, 2, 128, "bf16", seed=7, max_q=8).attach()
    for cu in ([0, 3, 7, 10], [0, 3, 2, 9], [-1, 3, 7, 9], [0, 3, 7, 2 ** 31 - 1]):
        c.cq.copy_(torch.tensor(cu, dtype=torch.int32))
        out = c.run(error=(pkv.ERR_DEVICE, pkv.DEVERR_SEQ_LEN))
        assert not torch.isnan(out.float()).all()


def test_refusals():
    c = T.Case([100, 60], [3, 4], 8, 2, 128, "bf16").attach()
    ws = c.workspace()
    out = torch.empty_like(c.qd)

    def call(pool=c.pool, q=c.qd, mask=c.mk, max_q=c.max_q, scale=c.scale, ws=ws, o=out, **kw):
        pkv.paged_attention_tree(pool, q, c.kc, c.vc, c.bt, c.sl, c.cq, mask, max_q, scale, o, ws, **kw)

    call()
    for kw in (dict(max_q=0, mask=None), dict(max_q=257, mask=None), dict(scale=float("nan")), dict(scale=float("inf")), dict(window=-1),
               dict(sinks=-1), dict(window=3), dict(ws=ws[:1024]), dict(ws=ws[1:]), dict(pool=pkv.Pool(c.NB, 2, 128))):
        with pytest.raises(pkv.PkvError) as e:
            call(**kw)
        assert e.value.status == pkv.ERR_INVALID, kw
    call(window=4)
    call(window=3, mask=None)
    for kw in (dict(mask=c.mk[:-1]), dict(mask=c.mk.int()), dict(max_q=65), dict(o=out[:-1]), dict(q=c.qd.transpose(0, 1))):
        with pytest.raises(ValueError):
            call(**kw)
    with pytest.raises(ValueError):                                     # as many elements, other heads
        call(q=c.qd.view(7, 16, 64), o=out.view(7, 16, 64))
    both = torch.empty((8, 8, 128), dtype=torch.bfloat16, device="cuda")
    for q, o in ((both[:7], both[:7]), (both[:7], both[1:]), (both[1:], both[:7])):
        with pytest.raises(pkv.PkvError) as e:                          # out over q
            call(q=q, o=o)
        assert e.value.status == pkv.ERR_INVALID
    assert pkv.tree_workspace_bytes(c.pool, 0, 8, 4) == 0 and pkv.tree_workspace_bytes(c.pool, 1, 7, 4) == 0
    assert pkv.tree_workspace_bytes(c.pool, 4097, 8, 4) == 0 and pkv.tree_workspace_bytes(c.pool, 1, 66, 4) == 0
    assert c.pool.get_device_error() == (pkv.OK, 0)


@pytest.mark.parametrize("Hq", [8, 32])
def test_a_captured_call_follows_the_lengths_and_graphs_share_a_workspace(Hq):
    c = T.Case([100, 60, 333], [3, 8, 5], Hq, 2, 128, "bf16", seed=1, pad=4, max_q=8).attach()
    ws, out = c.workspace(), torch.full_like(c.qd, float("nan"))
    sl, cq, mk, bt = c.sl.clone(), c.cq.clone(), c.mk.clone(), c.bt.clone()

    def call():
        pkv.paged_attention_tree(c.pool, c.qd, c.kc, c.vc, bt, sl, cq, mk, 8, c.scale, out, ws)

    call()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        graphs.append(g)
    d = T.Case([17, 0, 40], [8, 8, 1], Hq, 2, 128, "bf16", seed=2, max_q=8, spare=30, width=c.MB)
    assert (d.NB, d.MB) == (c.NB, c.MB) and d.T < c.T + 4
    want_c, want_d = c.run(), d.run()
    for g in graphs:
        out.fill_(float("nan"))
        g.replay()
        assert torch.equal(out[:c.T], want_c[:c.T])
    # other lengths, rows, trees and tables in the same buffers
    c.kc.copy_(d.kc), c.vc.copy_(d.vc), bt.copy_(d.bt), sl.copy_(d.sl), cq.copy_(d.cq)
    c.qd[:d.T] = d.qd
    mk[:d.T] = d.mk
    for g in graphs:
        out.fill_(float("nan"))
        g.replay()
        assert torch.equal(out[:d.T], want_d) and torch.isnan(out[d.T:].float()).all()
    assert c.pool.get_device_error() == (pkv.OK, 0)


@pytest.mark.parametrize("Hq", [8, 32])
def test_another_stream(Hq):
    c = T.Case([100, 60, 333], [3, 8, 5], Hq, 2, 128, "fp8", seed=1)
    want = c.run()
    s, ws = torch.cuda.Stream(), c.workspace()
    out = torch.full_like(c.qd, float("nan"))
    s.wait_stream(torch.cuda.current_stream())
    pkv.paged_attention_tree(c.pool, c.qd, c.kc, c.vc, c.bt, c.sl, c.cq, c.mk, c.max_q, c.scale, out, ws, stream=s)
    s.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("Hq", [16, 128])
def test_offsets_past_32_bits(Hq):
    """Blocks at the end of a cache of more than 2^32 bytes, and of more than 2^31 elements."""
    NB, Hkv, D = 150_000, 8, 128
    c = T.Case([100, 60], [3, 4], Hq, Hkv, D, "bf16", seed=3).attach()
    far = torch.arange(NB - c.NB, NB, dtype=torch.int32, device="cuda")
    pool = pkv.Pool(NB, Hkv, D)
    pool.attach_device(torch.cuda.current_device())
    kc, vc = (torch.empty(NB, Hkv, 16, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kc[NB - c.NB:], vc[NB - c.NB:] = c.kc, c.vc
    out = torch.full_like(c.qd, float("nan"))
    bt = torch.where(c.bt >= 0, far[c.bt.clamp(min=0).long()], c.bt)
    pkv.paged_attention_tree(pool, c.qd, kc, vc, bt, c.sl, c.cq, c.mk, c.max_q, c.scale, out, c.workspace())
    assert pool.get_device_error() == (pkv.OK, 0)
    assert torch.equal(out, c.run())


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int4"])
@pytest.mark.parametrize("Hq", [8, 32])
def test_a_wait_that_runs_out_is_reported(kind, Hq):
    c = T.Case([500, 60], [3, 9], Hq, 2, 128, kind, seed=3)
    want = c.run()
    pkv.test_expire_waits(pkv.TEST_EXPIRE_DECODE)
    try:
        c.run(error=(pkv.ERR_TIMEOUT, pkv.DEVERR_TIMEOUT))
    finally:
        pkv.test_expire_waits(pkv.TEST_EXPIRE_NONE)
    assert torch.equal(c.run(), want)


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int4"])
@pytest.mark.parametrize("Hq,width", [(8, 0), (16, 1000), (32, 1000)])
def test_a_row_of_nans_stays_by_itself(kind, Hq, width):
    """A query of NaN: that row of that head is NaN, and the rows that share its unit and its tiles are not."""
    c = T.Case([700, 333], [30, 9], Hq, 2, 128, kind, seed=5, width=width)
    c.q[3, 1] = float("nan")
    c.q[35, 0, 17] = float("nan")
    out = c.run()
    c.check(out)
    assert torch.isnan(out[3, 1].float()).all() and int(torch.isnan(out[:c.T].float()).any(-1).sum()) == 2


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int4"])
def test_calls_on_two_streams_at_once(kind):
    """Two calls in flight, each with its own workspace: each as by itself."""
    cases = [T.Case([3000, 1200, 40], [20, 7, 64], 32, 4, 128, kind, seed=8).attach(), T.Case([2000] * 6, [3] * 6, 8, 2, 64, kind, seed=9).attach()]
    alone = [c.run() for c in cases]
    ws, outs = [c.workspace() for c in cases], [[torch.empty_like(o) for _ in range(20)] for o in alone]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for i in range(20):
        for c, w, o, s in zip(cases, ws, outs, streams):
            pkv.paged_attention_tree(c.pool, c.qd, c.kc, c.vc, c.bt, c.sl, c.cq, c.mk, c.max_q, c.scale, o[i], w, stream=s)
    torch.cuda.synchronize()
    for c, a, o in zip(cases, alone, outs):
        assert c.pool.get_device_error() == (pkv.OK, 0)
        for x in o:
            assert torch.equal(x[:c.T].view(torch.int16), a[:c.T].view(torch.int16))


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int4"])
def test_blocks_beyond_32_bit_offsets(kind):
    """The last blocks of a pool whose caches pass 2^32 bytes: attention, a windowed prefill and the accepted rows are
    those of a small pool, bit for bit."""
    c = T.Case([500, 90], [30, 5], 16, 2, 128, kind, seed=3, free=False).attach()
    few = T.Case([500, 90], [1, 2], 16, 2, 128, kind, seed=3, free=False).attach()
    prompt = T.Case([300, 0], [100, 70], 16, 2, 128, kind, tree=False, window=80, sinks=3, seed=4).attach()
    for x in (c, few, prompt):
        bits = torch.uint8 if kind != "bf16" else torch.int16
        off = 2 ** 32 // x.kc[0].nbytes + 1
        ks, vs = x.pages.scales
        pool = pkv.Pool(off + x.NB, x.Hkv, x.D, T.KINDS[kind], ks, vs)
        pool.attach_device(torch.cuda.current_device())
        big = [torch.zeros((off + x.NB,) + tuple(y.shape[1:]), dtype=y.dtype, device="cuda") for y in (x.kc, x.vc)]
        for y, z in zip(big, (x.kc, x.vc)):
            y.view(bits)[off:] = z.view(bits)
        bt = torch.where(x.bt >= 0, x.bt + off, x.bt).int()
        out = torch.empty_like(x.qd)
        if x is prompt:
            plan, grid = pkv.prefill_plan(pool, x.cu, x.L, x.Hq, x.MB, window=80, sinks=3)
            n = pkv.prefill_workspace_bytes(pool, x.cu, x.L, x.MB, window=80, sinks=3)
            ws = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
            small = torch.empty_like(out)
            pkv.paged_prefill(x.pool, x.qd, x.kc, x.vc, x.bt, x.scale, T.dev(plan), grid, small, workspace=ws)
            pkv.paged_prefill(pool, x.qd, *big, bt, x.scale, T.dev(plan), grid, out, workspace=ws)
        else:
            small = x.run()
            pkv.paged_attention_tree(pool, x.qd, *big, bt, x.sl, x.cq, x.mk, x.max_q, x.scale, out, x.workspace())
            path = torch.tensor([[0, 2, 7], [1, 3, 4]] if x is c else [[0], [1]], dtype=torch.int32, device="cuda")
            n, lens = torch.full((2,), path.shape[1], dtype=torch.int32, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda")
            pkv.accept_rows(x.pool, x.kc, x.vc, x.bt, x.sl, x.cq, path, n, lens)
            pkv.accept_rows(pool, *big, bt, x.sl, x.cq, path, n, lens)
            for y, z in zip(big, (x.kc, x.vc)):
                assert torch.equal(y.view(bits)[off:], z.view(bits))
        assert pool.get_device_error() == (pkv.OK, 0) and x.pool.get_device_error() == (pkv.OK, 0)
        assert torch.equal(out[:x.T].view(torch.int16), small[:x.T].view(torch.int16))
        del big
