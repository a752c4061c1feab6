"""What the INT4 decode's bound lets pass, on the plain implementation alone: a block of positions
left out anywhere in a long sequence has to show."""
import numpy as np
import pytest

from oracle import int4 as O
from tests import _int4 as I
from tests import _int4_bounds as B

CASES = [([20000], 8, 1, 128), ([5000, 333, 9000], 8, 2, 64)]


@pytest.mark.parametrize("lens,Hq,Hkv,D", CASES, ids=["128", "64"])
def test_a_block_left_out_is_outside_the_bound(lens, Hq, Hkv, D):
    c = B.bands(lens, Hq, Hkv, D, seed=len(lens))
    ref, tol = B.bound(c, 152)
    q = O.bf16_values(I.bits(c.q)).astype(np.float64)
    for b, L in enumerate(lens):
        k, v = O.sequence(c.kh, c.vh, c.tables[b], L, c.k_scale, c.v_scale)
        nb = -(-L // 16)
        for h in range(Hq):
            hk = h // (Hq // Hkv)
            s = (k[:, hk] @ q[b, h]) * float(np.float32(c.scale))
            p = np.exp(s - s.max())
            whole = p @ v[:, hk]
            assert np.allclose(whole / p.sum(), ref[b, h], rtol=1e-12)
            edges = np.arange(0, L, 16)
            pb = np.add.reduceat(p, edges)                                  # a block's mass and values
            vb = np.add.reduceat(p[:, None] * v[:, hk], edges, axis=0)
            without = (whole - vb) / (p.sum() - pb)[:, None]                # [blocks, D]
            shows = (np.abs(without - ref[b, h]) > tol[b, h]).any(-1)
            assert shows.all(), "%d of %d blocks could be lost" % ((~shows).sum(), nb)


def test_the_bound_leaves_no_room_for_zeros():
    c = B.bands(*CASES[0], seed=1)
    ref, tol = B.bound(c, 152)
    assert (tol < 2.0 ** -6 * np.abs(ref)).all()
