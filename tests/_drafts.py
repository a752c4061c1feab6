"""Cases for attention of drafted tokens and of windows: seeded caches of every pool type in which
every position that no row sees is NaN, trees, the definition in 64 bits and the bound of its outputs."""
import numpy as np
import torch

import paged_kv_cache_159_gb300 as pkv
from oracle import int4 as O

KINDS = {"bf16": pkv.KV_BF16, "fp8": pkv.KV_FP8E4M3, "int4": pkv.KV_INT4}
K_SCALE, V_SCALE = 0.0131, 0.0087
WIDTH = 0                                          # entries that a case's tables have at least: calls with few tiles take another kernel


def dev(x) -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def tree_parents(P, rng, roots=0.1, reach=6):
    """Parents of P drafted tokens (-1: the last cached token), children behind their parents."""
    return [-1] + [-1 if rng.random() < roots else int(rng.integers(max(0, i - reach), i)) for i in range(1, P)]


def ancestors(par):
    """sees [P, P]: token j is i or above it."""
    see = np.zeros((len(par), len(par)), bool)
    for i, up in enumerate(par):
        if up >= 0:
            see[i] = see[up]
        see[i, i] = True
    return see


def visible(C, P, window, sinks, drafts=None):
    """[P, C + P]: what each new row sees.  drafts [P, P]: a tree's rows (None: a chain)."""
    see = np.zeros((P, C + P), bool)
    for i in range(P):
        place = C + i if drafts is None else C + int(drafts[i].sum()) - 1
        for j in range(C + P):
            near = window == 0 or j > place - window or j < sinks
            if drafts is None:
                see[i, j] = j <= place and near
            else:
                see[i, j] = near if j < C else drafts[i, j - C]
    return see


class Pages:
    """Caches on the host by pool type: rows written, poisoned, and read in 64 bits."""

    def __init__(self, kind, NB, Hkv, D, layers=1):
        self.kind, self.D = kind, D
        self.scales = (1.0, 1.0) if kind == "bf16" else (float(np.float32(K_SCALE)), float(np.float32(V_SCALE)))
        shape = (NB, Hkv, O.tile_bytes(D)) if kind == "int4" else (NB, Hkv, 16, D)
        fill = {"bf16": 0x7FC0, "fp8": 0x7F, "int4": 0xFF}[kind]
        self.caches = [np.full(shape, fill, np.uint16 if kind == "bf16" else np.uint8) for _ in range(2)]
        if kind == "int4":
            for x in self.caches:
                x[:, :, 8 * D:] = 0x7F

    def write(self, slots, rows):
        """rows: (k, v) bf16 tensors [T, Hkv, D]."""
        s = np.asarray(slots)
        if self.kind == "int4":
            O.append(*[r.view(torch.int16).numpy().view(np.uint16) for r in rows], s, *self.caches, *self.scales)
            return
        for x, r, scale in zip(self.caches, rows, self.scales):
            if self.kind == "bf16":
                x[s // 16, :, s % 16] = r.view(torch.int16).numpy().view(np.uint16)
            else:
                x[s // 16, :, s % 16] = (r.float() / scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()

    def read(self, slots):
        """[(k), (v)] each [T, Hkv, D] in 64 bits."""
        s, out = np.asarray(slots), []
        for x, is_key, scale in zip(self.caches, (True, False), self.scales):
            if self.kind == "int4":
                n, sb = O.codes(x, s, is_key)
                out.append(n * sb * scale)
            elif self.kind == "bf16":
                out.append((x[s // 16, :, s % 16].astype(np.uint32) << 16).view(np.float32).astype(np.float64))
            else:
                out.append(O.e4m3_values()[x[s // 16, :, s % 16]] * scale)
        return out

    def device(self):
        return [torch.from_numpy(x.view(np.int16)).cuda().view(torch.bfloat16) if self.kind == "bf16" else dev(x) for x in self.caches]


class Case:
    def __init__(self, cached, new, Hq, Hkv, D, kind="bf16", tree=True, window=0, sinks=0, seed=0, spare=2, width=0, scale=None,
                 q_gain=1.0, free=True, order_seed=None, pad=0, max_q=None):
        rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        self.C, self.P = np.array(cached, np.int32), np.array(new, np.int32)
        self.L, self.Hq, self.Hkv, self.D, self.kind = self.C + self.P, Hq, Hkv, D, kind
        self.window, self.sinks, self.tree = window, sinks, tree
        self.scale = float(np.float32(1 / np.sqrt(D))) if scale is None else scale
        self.cu = np.concatenate([[0], np.cumsum(self.P)]).astype(np.int32)
        self.T = int(self.cu[-1])
        self.max_q = max(1, int(self.P.max())) if max_q is None else max_q
        self.drafts = [ancestors(tree_parents(int(p), rng)) if p else np.zeros((0, 0), bool) for p in self.P] if tree else [None] * len(self.P)
        self.see = [visible(int(c), int(p), window, sinks, d) for c, p, d in zip(self.C, self.P, self.drafts)]
        need = [-(-int(n) // 16) for n in self.L]
        self.NB, self.MB = sum(need) + spare, max(max(need), width, 1, WIDTH)
        order = np.random.default_rng(seed if order_seed is None else order_seed).permutation(self.NB)
        self.tables, at = np.full((len(need), self.MB), -1, np.int32), 0
        for b, n in enumerate(need):
            self.tables[b, :n] = order[at:at + n]
            at += n
        self.pages = Pages(kind, self.NB, Hkv, D)
        for b in range(len(need)):
            pos = np.flatnonzero(self.see[b].any(0))
            rows = [torch.randn(len(self.see[b][0]) if len(self.see[b]) else 0, Hkv, D, generator=g).bfloat16() for _ in range(2)]
            if len(pos):
                self.pages.write(self.slots(b, pos), [r[pos] for r in rows])
            if free:                                            # blocks that nobody sees are not in the table
                gone = np.setdiff1d(np.arange(need[b]), pos // 16)
                self.tables[b, gone] = -1
        self.q = (q_gain * torch.randn(self.T + pad, Hq, D, generator=g)).bfloat16()
        self.pool = None

    def slots(self, b, pos):
        pos = np.asarray(pos)
        return self.tables[b, pos // 16].astype(np.int64) * 16 + pos % 16

    def mask(self):
        """int64 [rows, words]."""
        words = -(-self.max_q // 64)
        out = np.zeros((self.q.shape[0], words), np.uint64)
        for b, d in enumerate(self.drafts):
            for i in range(len(d)):
                for j in np.flatnonzero(d[i]):
                    out[self.cu[b] + i, j // 64] |= np.uint64(1 << (int(j) % 64))
        return out.view(np.int64)

    def attach(self):
        if self.pool is None:
            ks, vs = self.pages.scales
            self.pool = pkv.Pool(self.NB, self.Hkv, self.D, KINDS[self.kind], ks, vs)
            self.pool.attach_device(torch.cuda.current_device())
            self.kc, self.vc = self.pages.device()
            self.bt, self.sl, self.cq, self.qd = dev(self.tables), dev(self.L), dev(self.cu), self.q.cuda()
            self.mk = dev(self.mask()) if self.tree else None
        return self

    def workspace(self):
        n = pkv.tree_workspace_bytes(self.pool, len(self.P), self.Hq, self.max_q)
        assert n > 0
        return torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")          # any content will do

    def run(self, ws=None, error=(pkv.OK, 0)):
        self.attach()
        out = torch.full(self.q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
        pkv.paged_attention_tree(self.pool, self.qd, self.kc, self.vc, self.bt, self.sl, self.cq, self.mk, self.max_q, self.scale,
                                 out, self.workspace() if ws is None else ws, window=self.window, sinks=self.sinks)
        assert self.pool.get_device_error() == error
        return out

    def reference(self):
        """(out, mag, ds) [T, Hq, D], [T, Hq, D], [T, Hq]: the definition in 64 bits, sum p |v|, and the bound of
        a score's error in the exponent's units."""
        out, mag, ds = np.zeros((self.T, self.Hq, self.D)), np.zeros((self.T, self.Hq, self.D)), np.zeros((self.T, self.Hq))
        g = self.Hq // self.Hkv
        for b in range(len(self.P)):
            pos = np.flatnonzero(self.see[b].any(0)) if self.P[b] else []
            if not len(pos):
                continue
            k, v = self.pages.read(self.slots(b, pos))
            see = self.see[b][:, pos]
            q = self.q[self.cu[b]:self.cu[b + 1]].double().numpy()
            for h in range(self.Hq):
                with np.errstate(all="ignore"):
                    s = np.where(see, self.scale * (q[:, h] @ k[:, h // g].T), -np.inf)
                    top = s.max(-1, keepdims=True)
                    e = np.exp(s - np.where(np.isfinite(top), top, 0))
                    e[~see] = 0
                    z = e.sum(-1, keepdims=True)
                    p = e / np.where(z > 0, z, 1)
                    vv = np.where(np.isfinite(v[:, h // g]), v[:, h // g], 0)
                    o = p @ vv
                    bad = p @ (~np.isfinite(v[:, h // g])).astype(float)          # weights on what is not finite
                    o[bad > 0] = np.nan
                    out[self.cu[b]:self.cu[b + 1], h] = o
                    mag[self.cu[b]:self.cu[b + 1], h] = p @ np.abs(vv)
                    a = abs(self.scale) * (np.abs(q[:, h]) @ np.abs(k[:, h // g]).T)
                    ds[self.cu[b]:self.cu[b + 1], h] = np.where(see, a, 0).max(-1) * (self.D * 2.0 ** -23 + 2.0 ** -22)
        return out, mag, ds

    def check(self, out, skip=(), p_bits=None):
        """Every output against the arithmetic's bound (p_bits: significant bits of P, whose largest is then at least 1):
          output rounding   2^-8 |ref|
          P in 8 bits (bf16 pools) or 11 (f16), relative 2^-8 or 2^-11 of sum p |v|; f16 below 2^-14 is off by
                            2^-25, where the largest P is 2^8 and sums are at least that: 2^-33 max |v| a position
          scores            products exact, D fp32 additions (each off by 2^-23 of sum |q k|: the tensor core
                            truncates), scale and exp2: ds, which enters P and the normaliser
          exp2, sums        2^-20, and 2^-23 for every position summed
        """
        ref, mag, ds = self.reference()
        got = out[:self.T].float().cpu().double().numpy()
        L = np.repeat(self.L, self.P)[:, None, None]
        p_err = 2.0 ** -p_bits if p_bits else 2.0 ** -8 if self.kind == "bf16" else 2.0 ** -11
        tol = 2.0 ** -8 * np.abs(ref) + mag * (p_err + 2 * ds[..., None] + 2.0 ** -20 + L * 2.0 ** -23)
        if self.kind != "bf16":
            tol = tol + L * (2.0 ** -25 if p_bits else 2.0 ** -33) * 7 * 448 * V_SCALE
        keep = np.ones(self.T, bool)
        for b in skip:
            keep[self.cu[b]:self.cu[b + 1]] = False
        want_nan = np.isnan(ref)
        assert np.array_equal(np.isnan(got) & keep[:, None, None], want_nan & keep[:, None, None])
        off = np.where(want_nan, 0, np.abs(got - np.where(want_nan, 0, ref)))[keep]
        bad = off > np.where(want_nan, 1, tol)[keep]
        with np.errstate(all="ignore"):
            assert not bad.any(), "%d of %d outside; worst %.3g times its bound" % (bad.sum(), bad.size, np.nanmax(off / tol[keep]))
        assert torch.isnan(out[self.T:].float()).all()                            # rows behind the last sequence
