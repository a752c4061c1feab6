"""The query heads of a KV head are independent of each other in the INT4 decode: heads of
very different magnitude, and one that holds infinities or NaN."""
import numpy as np
import pytest
import torch

from oracle import int4 as O
from tests import _int4 as I
from tests import _int4_bounds as B

pkv = pytest.importorskip("paged_kv_cache_159_gb300")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    pkv.lib()
    torch.cuda.set_device(0)


SHAPES = [(8, 2, 64), (16, 2, 128), (14, 1, 64), (16, 1, 128)]          # groups 4, 8, 14, 16
LENS = [3000, 20, 333]                                                  # cut and whole units


def _grid():
    return torch.cuda.get_device_properties(0).multi_processor_count


@pytest.mark.parametrize("Hq,Hkv,D", SHAPES)
def test_heads_of_very_different_magnitude(Hq, Hkv, D):
    c = I.Case(LENS, Hq, Hkv, D, seed=Hq + D)
    gain = torch.tensor([1.0, 2.0 ** 30, 2.0 ** -30, 2.0 ** 100, 2.0 ** -100, 2.0 ** 12, 1.0])
    c.q = (c.q.float() * gain[torch.arange(Hq) % 7][:, None]).bfloat16()
    out = c.decode()
    B.check(out, *B.bound(c, _grid()))
    # scores of 2^30 and 2^100: the position with the largest, where it stands out by 2^-10 of itself
    # (scores are off by less than 2^-11 of it), returns its value
    q, got, seen = O.bf16_values(I.bits(c.q)).astype(np.float64), out.float().cpu().double().numpy(), 0
    for b, L in enumerate(c.lens.tolist()):
        k, v = O.sequence(c.kh, c.vh, c.tables[b], L, c.k_scale, c.v_scale)
        for h in (h for h in range(Hq) if h % 7 in (1, 3)):
            s = k[:, h // (Hq // Hkv)] @ q[b, h]
            top = np.argsort(s)[::-1]
            if s[top[0]] - s[top[1]] > 2.0 ** -10 * s[top[0]]:
                seen += 1
                ref = v[top[0], h // (Hq // Hkv)]
                # (two roundings of p scale to f16, the output's, one of the pool's scale)
                assert (np.abs(got[b, h] - ref) <= np.abs(ref) * (2.0 ** -8 + 2.0 ** -10 + 2.0 ** -16)).all()
    assert seen >= Hq // 7


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("Hq,Hkv,D", SHAPES)
def test_a_head_that_is_not_finite_leaves_the_others(Hq, Hkv, D, bad):
    c = I.Case(LENS, Hq, Hkv, D, seed=Hq)
    ref, tol = B.bound(c, _grid())
    c.q[0, Hq // Hkv - 1, 5] = bad
    c.q[1, 0, D - 1] = bad
    hit = np.zeros(c.q.shape[:2], bool)
    hit[0, Hq // Hkv - 1] = hit[1, 0] = True
    got = c.decode().float().cpu().double().numpy()
    assert (np.abs(got - ref) <= tol)[~hit].all()


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("opts", [None, {"grid_ctas": 1}, {"grid_ctas": 300}], ids=["default", "1", "300"])
@pytest.mark.parametrize("Hq,Hkv,D", SHAPES)
def test_a_head_that_is_not_finite_returns_nan(Hq, Hkv, D, opts, bad):
    # no finite answer of a head without one, whether its unit is cut or whole
    c = I.Case(LENS, Hq, Hkv, D, seed=Hq)
    c.q[:, Hq // Hkv - 1, 5] = bad
    out = c.decode(opts).float()
    assert bool(out[:, Hq // Hkv - 1].isnan().all())
    keep = [h for h in range(Hq) if h != Hq // Hkv - 1]
    assert bool(out[:, keep].isfinite().all())


@pytest.mark.parametrize("gain", [2.0 ** 12, 2.0 ** 30, 2.0 ** 60, 2.0 ** 120])
@pytest.mark.parametrize("Hq,Hkv,D", SHAPES)
def test_large_scores_over_many_pairs(Hq, Hkv, D, gain):
    # one warp (or a few) takes whole sequences, so that its reference is raised many times; the outputs
    # are means of rows of V, whatever the positions are that win
    c = I.Case([3000, 500, 1203], Hq, Hkv, D, seed=D)
    c.q = (c.q.float() * gain).bfloat16()
    for o in ({"grid_ctas": 1}, {"grid_ctas": 3}, None):
        got = c.decode(o).float().cpu().double().numpy()
        assert np.isfinite(got).all()
        for b, L in enumerate(c.lens.tolist()):
            v = O.sequence(c.kh, c.vh, c.tables[b], L, c.k_scale, c.v_scale)[1]
            for h in range(Hq):
                x = v[:, h // (Hq // Hkv)]
                # (the roundings of decode_bound's outputs, of the largest of a column)
                lo, hi, eps = x.min(0), x.max(0), np.abs(x).max(0) * 2.0 ** -7
                assert (got[b, h] >= lo - eps).all() and (got[b, h] <= hi + eps).all()
                assert (np.abs(got[b, h]) > np.abs(x).max() * 2.0 ** -10).any()       # and not zeros
