"""INT4 decode within a bound taken from what the cache holds, at every shape, magnitude and scale,
and over long sequences in which every block of positions shows."""
import pytest
import torch

from tests import _int4 as I
from tests import _int4_bounds as B
from tests.test_gpu_int4 import SHAPES
from tests.test_int4_bounds import CASES

pkv = pytest.importorskip("paged_kv_cache_159_gb300")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    pkv.lib()
    torch.cuda.set_device(0)


def _grid(opts):
    return opts["grid_ctas"] if opts else torch.cuda.get_device_properties(0).multi_processor_count


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s[1:])) + "-%d" % len(s[0]))
def test_shapes_and_grids(shape):
    c = I.Case(*shape, seed=40 + shape[1])
    for o in (None, {"grid_ctas": 1}, {"grid_ctas": 37}):
        B.check(c.decode(o), *B.bound(c, _grid(o)))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("q_gain,v_gain,ks,vs,scale", [(1e-6, 1.0, 0.0131, 0.0087, 0.1), (3e4, 1.0, 0.0131, 0.0087, 0.1), (8.0, 1.0, 1.0, 1.0, 0.1),
                                                       (1.0, 1e4, 0.5, 40.0, 0.1), (1.0, 1.0, 1.0, 1.0, 0.0), (1.0, 1.0, 1.0, 1.0, -0.2)])
def test_magnitudes_and_scales(q_gain, v_gain, ks, vs, scale, D):
    c = I.Case([200, 9, 64, 3000], 8, 2, D, seed=5, q_gain=q_gain, v_gain=v_gain, k_scale=ks, v_scale=vs)
    c.scale = scale
    B.check(c.decode(), *B.bound(c, _grid(None)))


@pytest.mark.parametrize("case", CASES, ids=["128", "64"])
def test_every_block_of_long_sequences_counts(case):
    c = B.bands(*case, seed=len(case[0]))
    pool = pkv.Pool(c.NB, c.Hkv, c.D, pkv.KV_INT4, c.k_scale, c.v_scale)
    pool.attach_device(0)
    kc, vc, bt, sl, q = I.dev(c.kh), I.dev(c.vh), I.dev(c.tables), I.dev(c.lens), c.q.cuda()
    for o in (None, {"grid_ctas": 61}, {"grid_ctas": 300}):
        out = torch.full(c.q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
        ws = torch.zeros(pkv.decode_workspace_bytes(pool, len(c.lens), c.Hq, c.MB, o), dtype=torch.uint8, device="cuda")
        pkv.paged_attention_decode(pool, q, kc, vc, bt, sl, c.scale, out, ws, o)
        assert pool.get_device_error() == (pkv.OK, 0)
        B.check(out, *B.bound(c, _grid(o)))
