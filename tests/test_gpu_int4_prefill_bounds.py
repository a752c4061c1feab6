"""Prefill over INT4 pools within the bound of exact elements and f16 weights, and at scores far
apart."""
import numpy as np
import pytest
import torch

from oracle import int4 as O
from tests import _int4 as I
from tests import _int4_bounds as B
from tests.test_gpu_int4_prefill import Chunks

pkv = pytest.importorskip("paged_kv_cache_159_gb300")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    pkv.lib()
    torch.cuda.set_device(0)


def _bound(c):
    return O.prefill_bound(I.bits(c.rows), c.kh, c.vh, c.tables, c.lens, c.cu, c.scale, c.k_scale, c.v_scale)


@pytest.mark.parametrize("v_gain,ks,vs", [(1.0, 0.0131, 0.0087), (1e3, 1.0, 1.0), (1e-3, 0.3, 1e-5)])
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 64), (8, 2, 128), (14, 2, 128)])
def test_prefill_bound(Hq, Hkv, D, v_gain, ks, vs):
    c = Chunks([130, 1, 64, 3], [270, 500, 0, 1200], Hq, Hkv, D, seed=Hq + D, v_gain=v_gain, k_scale=ks, v_scale=vs)
    B.check(c.prefill(), *_bound(c))


def test_many_equal_scores():
    # 4000 positions of about the same weight: small weights count in full
    c = Chunks([70], [4000], 4, 1, 128, seed=2)
    c.rows = (c.rows.float() * 2.0 ** -6).bfloat16()
    B.check(c.prefill(), *_bound(c))


@pytest.mark.parametrize("gain", [2.0 ** 12, 2.0 ** 30, 2.0 ** 60])
@pytest.mark.parametrize("D", [64, 128])
def test_large_scores(D, gain):
    # the outputs are means of visible rows of V, whatever the positions are that win
    c = Chunks([100, 3], [300, 700], 8, 2, D, seed=D)
    c.rows = (c.rows.float() * gain).bfloat16()
    got = c.prefill().float().cpu().double().numpy()
    assert np.isfinite(got).all()
    for b, L in enumerate(c.lens.tolist()):
        v = O.sequence(c.kh, c.vh, c.tables[b], L, c.k_scale, c.v_scale)[1]
        for h in range(8):
            x, o = v[:, h // 4], got[c.cu[b]:c.cu[b + 1], h]
            eps = np.abs(x).max(0) * 2.0 ** -7
            assert (o >= x.min(0) - eps).all() and (o <= x.max(0) + eps).all()
            assert (np.abs(o).max(-1) > np.abs(x).max() * 2.0 ** -10).all()       # and not zeros
