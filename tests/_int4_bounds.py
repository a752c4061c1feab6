"""INT4 decode against a bound taken from what the cache holds, and inputs in which every range of
positions shows in the output."""
import types

import numpy as np
import torch

from oracle import int4 as O
from tests import _int4 as I

BAND = 32                                     # positions: the least that a team of the decode takes


def bands(lens, Hq, Hkv, D, seed=0, k_scale=0.0131, v_scale=0.0087):
    """Host case: position t's value is 1 in column (t / BAND) % D and 0 elsewhere, so that an output
    column is the softmax mass of a few bands."""
    g = torch.Generator().manual_seed(seed)
    c = types.SimpleNamespace(lens=np.array(lens, np.int32), Hq=Hq, Hkv=Hkv, D=D, k_scale=k_scale, v_scale=v_scale,
                              scale=float(np.float32(1 / np.sqrt(D))))
    need = [-(-int(L) // 16) for L in lens]
    order = np.random.default_rng(seed).permutation(sum(need) + 2)
    c.NB, c.MB = sum(need) + 2, max(need)
    c.tables = np.full((len(lens), c.MB), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        c.tables[b, :n] = order[at:at + n]
        at += n
    T = int(c.lens.sum())
    c.k = torch.randn(T, Hkv, D, generator=g).bfloat16()
    c.v = torch.zeros(T, Hkv, D)
    pos = np.concatenate([np.arange(L) for L in lens])
    c.v[torch.arange(T), :, torch.from_numpy(pos // BAND % D)] = 1.0
    c.v = c.v.bfloat16()
    c.q = torch.randn(len(lens), Hq, D, generator=g).bfloat16()
    row = np.concatenate([np.full(L, b) for b, L in enumerate(lens)])
    c.slots = c.tables[row, pos // 16].astype(np.int64) * 16 + pos % 16
    c.kh, c.vh = (np.full((c.NB, Hkv, O.tile_bytes(D)), I.BAD_CODE, np.uint8) for _ in range(2))
    for x in (c.kh, c.vh):
        x[:, :, 8 * D:] = I.BAD_SCALE
    O.append(I.bits(c.k), I.bits(c.v), c.slots, c.kh, c.vh, k_scale, v_scale)
    return c


def partial_blocks(lens, Hq, Hkv, D, grid):
    """The most blocks that one partial state of the decode gathers: the (head group, block) tasks
    over the teams of the grid's warps, and no more than a sequence has."""
    nb = [-(-int(L) // 16) for L in lens]
    team = max(h for h in range(1, min(8, Hkv) + 1) if Hkv % h == 0)
    wide = Hq // Hkv > 8
    warps = {(128, False): 12, (128, True): 8, (64, False): 16, (64, True): 12}[D, wide]
    W = Hkv // team * sum(nb)
    teams = max(1, min((W + 1) // 2, grid * warps // team))
    return min(max(nb), -(-W // teams))


def bound(c, grid):
    return O.decode_bound(I.bits(c.q), c.kh, c.vh, c.tables, c.lens, c.scale, c.k_scale, c.v_scale,
                          partial_blocks(c.lens, c.Hq, c.Hkv, c.D, grid))


def check(out, ref, tol):
    got = out.float().cpu().double().numpy()
    assert np.isfinite(got).all()
    bad = np.abs(got - ref) > tol
    assert not bad.any(), "%d of %d outside; worst %.3g times its bound" % (bad.sum(), bad.size, (np.abs(got - ref) / tol).max())
