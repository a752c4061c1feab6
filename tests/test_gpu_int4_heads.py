"""The query heads of a KV head are independent of each other in the INT4 decode: one that
holds infinities or NaN leaves the others as they are."""
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
