"""INT4 pool cases: seeded inputs, caches written by the plain implementation (oracle/int4.py),
unread positions poisoned, and the error bound of decode and prefill outputs."""
import numpy as np
import torch

import paged_kv_cache_159_gb300 as pkv
import workloads
from oracle import int4 as O

BAD_CODE, BAD_SCALE = 0xFF, 0x7F          # codes +7, scales NaN: what dead positions hold


def bits(x) -> np.ndarray:
    return workloads.bf16_bits(x)


def dev(x) -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


class Case:
    """Sequences of the given lengths over shuffled blocks of an INT4 pool: host and device
    copies of the caches holding seeded rows at every live position."""

    def __init__(self, lens, Hq, Hkv, D, seed=0, k_scale=0.0131, v_scale=0.0087, spare=3, q_gain=1.0, v_gain=1.0,
                 order_seed=None, width=0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.Hq, self.Hkv, self.D = np.array(lens, np.int32), Hq, Hkv, D
        self.k_scale, self.v_scale = k_scale, v_scale
        self.scale = float(np.float32(1 / np.sqrt(D)))
        need = [-(-int(L) // 16) for L in lens]
        self.NB, self.MB = sum(need) + spare, max(max(need), width)
        order = np.random.default_rng(seed if order_seed is None else order_seed).permutation(self.NB)
        self.tables = np.full((len(lens), self.MB), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.tables[b, :n] = order[at:at + n]
            at += n
        T = int(self.lens.sum())
        r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.k, self.v = r(T, Hkv, D).bfloat16(), (v_gain * r(T, Hkv, D)).bfloat16()
        self.q = (q_gain * r(len(lens), Hq, D)).bfloat16()
        self.slots = np.concatenate([self.row_slots(b, np.arange(L)) for b, L in enumerate(lens)])
        tb = O.tile_bytes(D)
        self.kh, self.vh = (np.full((self.NB, Hkv, tb), BAD_CODE, np.uint8) for _ in range(2))
        for x in (self.kh, self.vh):
            x[:, :, 8 * D:] = BAD_SCALE
        O.append(bits(self.k), bits(self.v), self.slots, self.kh, self.vh, k_scale, v_scale)
        self.kc, self.vc = dev(self.kh), dev(self.vh)
        self.bt, self.sl = dev(self.tables), dev(self.lens)
        self.pool = self.new_pool()

    def row_slots(self, b, pos):
        return self.tables[b, pos // 16].astype(np.int64) * 16 + pos % 16

    def new_pool(self, layers=1):
        p = pkv.Pool(self.NB, self.Hkv, self.D, pkv.KV_INT4, self.k_scale, self.v_scale, num_layers=layers)
        p.attach_device(torch.cuda.current_device())
        return p

    def workspace(self, opts=None, pool=None):
        n = pkv.decode_workspace_bytes(pool or self.pool, len(self.lens), self.Hq, self.MB, opts)
        assert n > 0
        return torch.zeros(n, dtype=torch.uint8, device="cuda")

    def decode(self, opts=None, ws=None):
        out = torch.full((len(self.lens), self.Hq, self.D), float("nan"), dtype=torch.bfloat16, device="cuda")
        ws = self.workspace(opts) if ws is None else ws
        pkv.paged_attention_decode(self.pool, self.q.cuda(), self.kc, self.vc, self.bt, self.sl, self.scale, out, ws, opts)
        assert self.pool.get_device_error() == (pkv.OK, 0)
        assert int(ws[:len(self.lens) * self.Hkv * 4].count_nonzero()) == 0
        return out

    def check(self, out, kh=None, vh=None):
        ref, mag, ds = O.decode(bits(self.q), self.kh if kh is None else kh, self.vh if vh is None else vh,
                                  self.tables, self.lens, self.scale, self.k_scale, self.v_scale)
        within(out, ref, mag, ds, self.lens[:, None, None], self.v_scale)


def within(out, ref, mag, ds, L, v_scale):
    """|out - ref| against the arithmetic's bound:
      output rounding             2^-8 |ref|
      p and p * scale in f16      2 * 2^-11 of sum p |v|
      scores                      off by ds (oracle/int4.py), which enters p and the normaliser
      exp2, sums                  2^-16
      f16 underflow               p 2^8 and p * scale each off by 2^-25 for every position, which
                                  is at most 7 * 448 * v_scale and 2^8 * 7 * v_scale of the
                                  largest p 2^8 >= 2^8
    """
    got = out.float().cpu().double().numpy()
    assert np.isfinite(got).all()
    tol = 2.0 ** -8 * np.abs(ref) + mag * (2.0 ** -10 + 2 * ds + 2.0 ** -16)
    tol = tol + L * 2.0 ** -25 * (7 * 448 + 7) * v_scale
    bad = np.abs(got - ref) > tol
    assert not bad.any(), "%d of %d outside; worst %.3g times its bound" % (
        bad.sum(), bad.size, (np.abs(got - ref) / tol).max())
