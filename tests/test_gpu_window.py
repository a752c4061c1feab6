"""Decode with a sliding window and sinks, against the definition in 64 bits and the plain decode."""
import numpy as np
import pytest
import torch

import paged_kv_cache_159_gb300 as pkv
from tests import _drafts as T

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    return pkv.lib()


def decode(c, error=(pkv.OK, 0), window=None, sinks=None):
    c.attach()
    out = torch.full_like(c.qd, float("nan"))
    pkv.paged_attention_window(c.pool, c.qd, c.kc, c.vc, c.bt, c.sl, c.scale, c.window if window is None else window,
                               c.sinks if sinks is None else sinks, out, c.workspace())
    assert c.pool.get_device_error() == error
    return out


def case(lens, *args, **kw):
    return T.Case([n - 1 for n in lens], [1] * len(lens), *args, tree=False, **kw)


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int4"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(2, 2), (8, 2), (14, 2), (7, 1), (32, 2), (15, 5)])
def test_heads_and_types(kind, D, Hq, Hkv):
    c = case([1, 16, 17, 250, 1900], Hq, Hkv, D, kind, window=100, sinks=4, seed=Hq)
    c.check(decode(c))


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int4"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (2, 1), (15, 16), (16, 0), (17, 15), (63, 2), (64, 64), (65, 100), (128, 1), (5000, 7), (9, 2 ** 31 - 1)])
def test_windows_and_sinks_at_block_and_tile_edges(kind, window, sinks):
    c = case([1, 2, 15, 16, 17, 31, 64, 65, 129, 600], 8, 2, 128, kind, window=window, sinks=sinks, seed=window)
    c.check(decode(c))


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int4"])
def test_a_window_as_long_as_the_sequence_is_the_plain_decode(kind):
    c = case([333, 64, 1], 8, 2, 128, kind, window=0, seed=2)
    a, b, d = decode(c), decode(c, window=333), decode(c, window=2 ** 31 - 1, sinks=2 ** 31 - 1)
    c.check(a), c.check(b), c.check(d)
    ws = torch.zeros(pkv.decode_workspace_bytes(c.pool, 3, 8, c.MB), dtype=torch.uint8, device="cuda")
    e = torch.empty_like(c.qd)
    pkv.paged_attention_decode(c.pool, c.qd, c.kc, c.vc, c.bt, c.sl, c.scale, e, ws)
    assert (a.float() - e.float()).abs().max() <= 0.02


def test_a_long_window_is_cut_over_many_ctas():
    c = case([12000, 40], 4, 1, 128, "fp8", window=9000, sinks=20, seed=2)
    c.check(decode(c))


def test_bad_lengths_are_flagged_and_zero():
    c = case([100, 60, 30], 8, 2, 128, "int4", window=20, sinks=2, seed=7).attach()
    for L in (0, -1, c.MB * 16 + 1, 2 ** 31 - 1):
        c.sl[1] = L
        out = decode(c, error=(pkv.ERR_DEVICE, pkv.DEVERR_SEQ_LEN))
        assert (out[1] == 0).all()
        c.check(out, skip=[1])


def test_a_captured_window_slides():
    """One graph, replayed while the sequences grow and blocks behind the window leave the table."""
    c = case([200, 77], 8, 2, 128, "bf16", window=40, sinks=3, seed=9, free=False).attach()
    full = T.Case([199, 76], [1, 1], 8, 2, 128, "bf16", tree=False, seed=9, free=False)       # the same rows, all written
    full.attach()
    out, ws, sl, bt = torch.empty_like(c.qd), c.workspace(), full.sl.clone(), full.bt.clone()
    g = torch.cuda.CUDAGraph()
    call = lambda: pkv.paged_attention_window(full.pool, full.qd, full.kc, full.vc, bt, sl, full.scale, 40, 3, out, ws)  # noqa: E731
    call()
    with torch.cuda.graph(g):
        call()
    for lens in ([50, 20], [120, 60], [200, 77]):
        sl.copy_(torch.tensor(lens, dtype=torch.int32))
        for b, n in enumerate(lens):
            bt[b].copy_(full.bt[b])
            bt[b, 1:max(1, (n - 40) // 16)] = -1
        g.replay()
        for b, n in enumerate(lens):
            full.see[b] = T.visible(n - 1, 1, 40, 3)
        full.L = np.array(lens, np.int32)
        full.check(out)
    assert full.pool.get_device_error() == (pkv.OK, 0)


def test_refusals():
    c = case([100, 60], 8, 2, 128).attach()
    ws, out = c.workspace(), torch.empty_like(c.qd)
    good = dict(pool=c.pool, scale=c.scale, window=20, sinks=2, ws=ws, bt=c.bt, sl=c.sl)

    def call(**kw):
        a = {**good, **kw}
        pkv.paged_attention_window(a["pool"], c.qd, c.kc, c.vc, a["bt"], a["sl"], a["scale"], a["window"], a["sinks"], out, a["ws"])

    call()
    for kw in (dict(window=-1), dict(sinks=-2), dict(scale=float("inf")), dict(ws=ws[:-1]), dict(ws=ws[4:]), dict(pool=pkv.Pool(c.NB, 3, 128))):
        with pytest.raises(pkv.PkvError) as e:
            call(**kw)
        assert e.value.status == pkv.ERR_INVALID
    with pytest.raises(ValueError):
        pkv.paged_attention_window(c.pool, c.qd.view(2, 16, 64), c.kc, c.vc, c.bt, c.sl, c.scale, 20, 2, out.view(2, 16, 64), ws)
    with pytest.raises(pkv.PkvError):
        pkv.paged_attention_window(c.pool, c.qd, c.kc, c.vc, c.bt, c.sl, c.scale, 20, 2, c.qd, ws)
    for kw in (dict(sl=c.sl[:1]), dict(sl=c.sl.long()), dict(bt=c.bt[:1])):
        with pytest.raises(ValueError):
            call(**kw)
