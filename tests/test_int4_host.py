"""INT4 pools without a GPU: the descriptor, sizes and refusals of the library, and the plain
implementation of the format against its definition."""
import numpy as np
import pytest
import torch

import workloads
from oracle import int4 as O

pkv = pytest.importorskip("paged_kv_cache_159_gb300")


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_159_gb300 import build
    build.build()
    return pkv.lib()


def test_pool_sizes_and_scales(lib):
    for D, tile in ((64, 544), (128, 1088)):
        p = pkv.Pool(10, 3, D, pkv.KV_INT4, num_layers=2)
        assert p.tile_bytes() == tile == O.tile_bytes(D) and p.layer_bytes() == 10 * 3 * tile
        assert p.get_desc().kv_dtype == pkv.KV_INT4
    assert pkv.Pool(10, 3, 64).tile_bytes() == 16 * 64 * 2
    assert pkv.Pool(10, 3, 64, pkv.KV_FP8E4M3).tile_bytes() == 16 * 64
    for bad in (dict(k_scale=0.0), dict(v_scale=-1.0), dict(k_scale=float("inf")), dict(v_scale=float("nan")), dict(kv_dtype=3)):
        kw = dict(num_blocks=4, num_kv_heads=1, head_dim=64, kv_dtype=pkv.KV_INT4)
        kw.update(bad)
        with pytest.raises(pkv.PkvError):
            pkv.Pool(**kw)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("is_key", [True, False])
def test_every_code_and_scale_has_its_own_place(D, is_key):
    at, sh, sc = O.places(D, is_key)
    assert sorted((at * 2 + sh // 4).ravel().tolist()) == list(range(16 * D))
    assert sorted(sc[:, ::32].ravel().tolist()) == list(range(8 * D, O.tile_bytes(D)))
    for t in range(16):                               # a token's bytes are its own
        assert not set(at[t]) & set(np.delete(at, t, 0).ravel())


def test_scale_encoder_is_round_to_nearest_even():
    x = np.concatenate([np.linspace(0, 2, 4001), np.exp2(np.linspace(-12, 8.8, 5000)), [448.0]]).astype(np.float32)
    ref = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(O.e4m3_encode(x), ref)
    assert O.e4m3_encode(np.float32([1e9, np.inf])).tolist() == [126, 126]


def test_quantised_rows_are_within_half_a_step():
    x = torch.randn(50, 3, 128, generator=torch.Generator().manual_seed(1)).bfloat16()
    b = workloads.bf16_bits(x)
    kc, vc = (np.zeros((5, 3, O.tile_bytes(128)), np.uint8) for _ in range(2))
    slots = np.random.default_rng(0).permutation(80)[:50]
    O.append(b, b, slots, kc, vc, 0.01, 0.02)
    amax = x.float().unflatten(-1, (-1, 32)).abs().amax(-1, keepdim=True).expand(-1, -1, -1, 32).flatten(-2).double().numpy()
    for cache, is_key, s in ((kc, True, 0.01), (vc, False, 0.02)):
        err = np.abs(O.rows(cache, slots, is_key, s) - x.double().numpy())
        # the scale lies within 2^-4 of amax / 7, half a step of rounding, 2^-20 of fp32 steps
        assert (err <= amax / 7 * 0.5 * (1 + 2.0 ** -4) * (1 + 2.0 ** -20)).all()


def test_attention_oracle_is_the_dense_formula():
    rng = np.random.default_rng(3)
    q, k, v = rng.standard_normal(64), rng.standard_normal((37, 64)), rng.standard_normal((37, 64))
    out, mag = O.attend(q, k, v, 0.125)
    w = torch.softmax(torch.from_numpy(k @ q) * 0.125, 0).numpy()
    assert np.allclose(out, w @ v, rtol=1e-12, atol=1e-14) and np.allclose(mag, w @ np.abs(v))
