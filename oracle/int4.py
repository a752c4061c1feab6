"""The INT4 pool format and attention over it, restated plainly in numpy: codes and scales by
the format's definition (fp32 where it says fp32), attention in 64 bits.  Shares no code with
the library; places are computed one (token, column) at a time."""
from __future__ import annotations

import functools

import numpy as np

BS = 16
GROUP = 32


def tile_bytes(D: int) -> int:
    return 8 * D + D // 2


@functools.lru_cache(None)
def e4m3_values():
    """Value of each E4M3 byte (bias 7; 0x7F and 0xFF are NaN)."""
    out = np.zeros(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        v = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        if e == 15 and m == 7:
            v = float("nan")
        out[b] = -v if b & 128 else v
    return out


def e4m3_encode(x) -> np.ndarray:
    """Bytes of non-negative fp32 values, nearest (ties to the even byte), saturating at 448."""
    table = e4m3_values()[:127]
    a = np.minimum(np.asarray(x, np.float64), 448.0)
    hi = np.clip(np.searchsorted(table, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    up, dn = table[hi] - a, a - table[lo]
    return np.where((dn < up) | ((dn == up) & (lo % 2 == 0)), lo, hi).astype(np.uint8)


@functools.lru_cache(None)
def places(D: int, is_key: bool):
    """(byte, shift, scale byte) of every (token, column) of a tile, each [16, D]."""
    at, sh, sc = (np.zeros((BS, D), np.int64) for _ in range(3))
    ng = D // GROUP
    for t in range(BS):
        for d in range(D):
            j, e = divmod(d, GROUP)
            if is_key:
                r = (t & 8) | (t & 3) << 1 | (t >> 2) & 1
                c, i = divmod(e, 8)
                bit = 32 * (c * ng + j) + 4 * i
                sc[t, d] = 8 * D + r * ng + j
            else:
                r = t
                c, i = divmod(e, 4)
                if D == 128 and t & 2:
                    c ^= 4
                bit = 16 * (c * ng + j) + 4 * i
                sc[t, d] = 8 * D + (t & 3) * (D // 8) + 4 * j + (t >> 2)
            at[t, d], sh[t, d] = r * (D // 2) + bit // 8, bit % 8
    return at, sh, sc


def bf16_values(bits) -> np.ndarray:
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32)


def quantise(bits, pool_scale: float):
    """Codes [..., D] and scale bytes [..., D / 32] of bf16 rows, in the format's fp32 steps."""
    x = bf16_values(bits)
    with np.errstate(all="ignore"):
        inv = np.float32(1) / np.float32(pool_scale)
        y = (x * inv).reshape(*x.shape[:-1], -1, GROUP)
        a = np.fmax.reduce(np.abs(y), axis=-1, initial=np.float32(0))
        sb = e4m3_encode(a * (np.float32(1) / np.float32(7)))
        s = e4m3_values()[sb].astype(np.float32)[..., None]
        n = np.rint(y * (np.float32(1) / s))
        n = np.where((s > 0) & ~np.isnan(y), np.clip(n, -7, 7), 0) + 8
    return n.reshape(x.shape).astype(np.uint8), sb


def append(k_bits, v_bits, slots, key_cache, value_cache, k_scale: float, v_scale: float):
    """Write rows [T, Hkv, D] into their slots of caches uint8 [NB, Hkv, tile bytes], in place."""
    D = k_bits.shape[-1]
    for bits, cache, is_key, scale in ((k_bits, key_cache, True, k_scale), (v_bits, value_cache, False, v_scale)):
        n, sb = quantise(bits, scale)
        at, sh, sc = places(D, is_key)
        for i, slot in enumerate(np.asarray(slots)):
            if slot < 0:
                continue
            t = int(slot) % BS
            tile = cache[int(slot) // BS]                       # [Hkv, bytes]
            for x in (0, 4):                                    # low and high nibbles never share a byte
                sel = sh[t] == x
                tile[:, at[t, sel]] = (tile[:, at[t, sel]] & (0xF0 >> x)) | (n[i][:, sel] << x)
            tile[:, sc[t, ::GROUP]] = sb[i]


def codes(cache, slots, is_key: bool):
    """What the slots hold: n - 8 and the scales' values, each [T, Hkv, D]."""
    D = cache.shape[-1] * 2 // 17
    at, sh, sc = places(D, is_key)
    slots = np.asarray(slots)
    tiles, t = cache[slots // BS], slots % BS                   # [T, Hkv, bytes]
    code = np.take_along_axis(tiles, np.broadcast_to(at[t][:, None], tiles.shape[:2] + (D,)), -1) >> sh[t][:, None]
    sb = np.take_along_axis(tiles, np.broadcast_to(sc[t][:, None], tiles.shape[:2] + (D,)), -1)
    return (code & 15).astype(np.int64) - 8, e4m3_values()[sb]


def rows(cache, slots, is_key: bool, pool_scale: float) -> np.ndarray:
    """The elements [T, Hkv, D] that the slots hold, in 64 bits."""
    n, s = codes(cache, slots, is_key)
    return n * s * float(np.float32(pool_scale))


def attend(q, k, v, scale: float):
    """One query head over k, v [L, D]: the output, and sum_t p_t |v_t| (for error bounds)."""
    s = (k @ q) * float(np.float32(scale))
    p = np.exp(s - s.max())
    p /= p.sum()
    return p @ v, p @ np.abs(v)


def sequence(key_cache, value_cache, table_row, L: int, k_scale: float, v_scale: float):
    pos = np.arange(L)
    slots = np.asarray(table_row)[pos // BS].astype(np.int64) * BS + pos % BS
    return rows(key_cache, slots, True, k_scale), rows(value_cache, slots, False, v_scale)


def decode(q_bits, key_cache, value_cache, tables, seq_lens, scale, k_scale, v_scale):
    """q [B, Hq, D] -> (out, sum p |v|, score error), each [B, Hq, D] in 64 bits.  The score error of
    (b, head) bounds how far a score may be off that is formed from f16 products of q with the codes
    and fp32 sums: with ks_tj = k scale * scale of token t and group j,
      |scale| * max_t sum_j ks_tj (7 * 32 * 2^-24 max|q| + 2^-16 sum_{d in j} |q_d|):
    an element of q is off by at most 2^-24 of the largest, times |n - 8| <= 7 for 32 columns; a
    group's sum starts at -8 sum q and takes two products of codes up to 15, each taken to be off by
    2^-21 of the largest of these, at most 15 sum |q|, and its joining the score rounds four times
    by 2^-24: in all about 2^-16 of sum |q|.  (An estimate: decode_bound has what the products can
    be off by at most.)"""
    q = bf16_values(q_bits).astype(np.float64)
    B, Hq, D = q.shape
    Hkv = key_cache.shape[1]
    out, mag, ds = np.zeros_like(q), np.zeros_like(q), np.zeros_like(q)
    sc = places(D, True)[2]
    for b in range(B):
        L = int(seq_lens[b])
        k, v = sequence(key_cache, value_cache, tables[b], L, k_scale, v_scale)
        pos = np.arange(L)
        blk = np.asarray(tables[b])[pos // BS]
        for h in range(Hq):
            hk = h // (Hq // Hkv)
            out[b, h], mag[b, h] = attend(q[b, h], k[:, hk], v[:, hk], scale)
            sb = key_cache[blk[:, None], hk, sc[pos % BS][:, ::GROUP]]
            ks = e4m3_values()[sb] * float(np.float32(k_scale))
            aq = np.abs(q[b, h])
            ds[b, h] = abs(scale) * (ks @ (224 * 2.0 ** -24 * aq.max() + 2.0 ** -16 * aq.reshape(-1, GROUP).sum(-1))).max()
    return out, mag, ds


def decode_bound(q_bits, key_cache, value_cache, tables, seq_lens, scale, k_scale, v_scale, blocks):
    """q [B, Hq, D] -> (out, bound), each [B, Hq, D] in 64 bits: how far a decode may be off that
    takes codes to a tensor core as f16 subnormals, by what the cache holds.

    The tensor core aligns a product's 16 terms and its accumulator to the largest exponent among
    them and cuts each 25 bits below it (17 cuts, so less than 2^-20 of that exponent), and a
    subnormal counts with the smallest normal's exponent, 2^-14, whatever its value: a code n 2^-24 (the
    even nibbles) stands 2^10 below it, n 2^-20 (the odd ones) 2^6.

    Scores are off by ds = |scale| max_t sum_j ks_tj (...), with ks_tj = k scale * scale of token t and
    group j (of 32 columns), of
      products    two a group of q with the codes, 2 * 2^-20 * 2^10 = 2^-9 of max_{d in j} |q_d| (their
                  accumulator, at most 15 sum |q| <= 480 max |q| code units, is below 2^10 max |q|)
      q in f16    2^-24 of the head's largest, times 7, for 32 columns
      sums        five roundings of 2^-24 as group sums join the reference and each other, each of at
                  most 2 * 7 sum |q|: below 2^-17 of sum_{d in j} |q_d|.
    With p_t = exp(s_t - max s), Z = sum p, e the scale of a V element and a = |n - 8|, an output by
      output rounding           2^-8 |out|
      p and p e in f16          2 * 2^-11 of sum p |v| / Z
      scores                    ds in p and in the normaliser, e^(2 ds) - 1 of the same
      exp2, sums, the merge     2^-16 and 2^-22 a block (the normaliser's additions) of the same
      products                  two a block (the offset's, the codes'), each 2^-20 of the accumulator, at
                                most sum p e (a + 8) code units, and of 2^10 (2^6 for odd nibbles) times
                                the block's largest p e; `blocks` the most blocks that a partial state
                                gathers
      f16 underflow             p and p e are held as p 2^8 and p e (the largest p at 2^8 or more) and
                                off by 2^-25 each where they are subnormal: a (e 2^-8 + 1) 2^-25
                                a position, of a normaliser of 2^8 Z at least, and 2^8 times larger
                                once the scale's 2^-8 is taken back."""
    q = bf16_values(q_bits).astype(np.float64)
    B, Hq, D = q.shape
    Hkv = key_cache.shape[1]
    vs, sc = float(np.float32(v_scale)), places(D, True)[2]
    cut = np.where(np.arange(D) % 2 == 0, 2.0 ** -9, 2.0 ** -13)
    out, tol = np.zeros_like(q), np.zeros_like(q)
    for b, L in enumerate(np.asarray(seq_lens).tolist()):
        pos = np.arange(L)
        slots = np.asarray(tables[b])[pos // BS].astype(np.int64) * BS + pos % BS
        k = rows(key_cache, slots, True, k_scale)
        n, e = codes(value_cache, slots, False)
        a, edges = np.abs(n), np.arange(0, L, BS)
        for h in range(Hq):
            hk = h // (Hq // Hkv)
            s = (k[:, hk] @ q[b, h]) * float(np.float32(scale))
            p = np.exp(s - s.max())
            Z = p.sum()
            out[b, h] = p @ (n[:, hk] * e[:, hk]) / Z * vs
            mag = p @ (a[:, hk] * e[:, hk]) / Z * vs
            ks = e4m3_values()[key_cache[(slots // BS)[:, None], hk, sc[pos % BS][:, ::GROUP]]] * float(np.float32(k_scale))
            aq = np.abs(q[b, h]).reshape(-1, GROUP)
            ds = abs(scale) * (ks @ (2.0 ** -9 * aq.max(-1) + 224 * 2.0 ** -24 * aq.max() + 2.0 ** -17 * aq.sum(-1))).max()
            pe = p[:, None] * e[:, hk]
            if ds > 30:                                 # scores too large to tell one position from another
                tol[b, h] = np.inf
                continue
            tol[b, h] = (2.0 ** -8 * np.abs(out[b, h]) + mag * (2.0 ** -10 + 2.0 ** -16 + blocks * 2.0 ** -22 + np.expm1(2 * ds))
                         + vs / Z * (blocks * 2.0 ** -19 * (pe * (a[:, hk] + 8)).sum(0)
                                     + cut * np.maximum.reduceat(pe, edges, axis=0).sum(0)
                                     + 2.0 ** -25 * (a[:, hk] * (e[:, hk] * 2.0 ** -8 + 1)).sum(0)))
    return out, tol


def prefill(q_bits, key_cache, value_cache, tables, seq_lens, cu_q, scale, k_scale, v_scale):
    """q [T, Hq, D]: row cu_q[b] + i attends over positions 0 .. L_b - P_b + i of sequence b; (out,
    sum p |v|) in 64 bits."""
    q = bf16_values(q_bits).astype(np.float64)
    Hq, Hkv = q.shape[1], key_cache.shape[1]
    out, mag = np.zeros_like(q), np.zeros_like(q)
    for b, L in enumerate(np.asarray(seq_lens).tolist()):
        r0, r1 = int(cu_q[b]), int(cu_q[b + 1])
        if r1 == r0:
            continue
        k, v = sequence(key_cache, value_cache, tables[b], L, k_scale, v_scale)
        for h in range(Hq):
            hk = h // (Hq // Hkv)
            s = q[r0:r1, h] @ k[:, hk].T * float(np.float32(scale))
            s[np.arange(L)[None, :] > np.arange(L - (r1 - r0), L)[:, None]] = -np.inf
            p = np.exp(s - s.max(-1, keepdims=True))
            p /= p.sum(-1, keepdims=True)
            out[r0:r1, h], mag[r0:r1, h] = p @ v[:, hk], p @ np.abs(v[:, hk])
    return out, mag


def prefill_bound(q_bits, key_cache, value_cache, tables, seq_lens, cu_q, scale, k_scale, v_scale):
    """q [T, Hq, D] -> (out, bound) in 64 bits: how far a prefill may be off that multiplies exact
    elements with f16 weights.  With p, Z, mag = sum p |v| / Z and D / 16 (or L / 16) tensor-core products
    in a sum, each off by at most 2^-20 of the magnitudes that it adds (decode_bound):
      output rounding    2^-8 |out|
      p in f16           2^-11 of mag, and 2^-25 |v| / Z a position where p is subnormal (the largest is 1 or more)
      scores             ds = |scale| D / 16 2^-20 max_t sum |q| |k|, which enters p and Z: e^(2 ds) - 1 of mag
      products, sums     (L / 16) 2^-20, and 2^-16 for exp2 and the normaliser, of mag."""
    q = bf16_values(q_bits).astype(np.float64)
    D, Hq, Hkv = q.shape[2], q.shape[1], key_cache.shape[1]
    out, tol = np.zeros_like(q), np.zeros_like(q)
    for b, L in enumerate(np.asarray(seq_lens).tolist()):
        r0, r1 = int(cu_q[b]), int(cu_q[b + 1])
        if r1 == r0:
            continue
        k, v = sequence(key_cache, value_cache, tables[b], L, k_scale, v_scale)
        late = np.arange(L)[None, :] > np.arange(L - (r1 - r0), L)[:, None]
        for h in range(Hq):
            hk = h // (Hq // Hkv)
            s = q[r0:r1, h] @ k[:, hk].T * float(np.float32(scale))
            s[late] = -np.inf
            p = np.exp(s - s.max(-1, keepdims=True))
            Z = p.sum(-1, keepdims=True)
            av = np.abs(v[:, hk])
            out[r0:r1, h], mag = p @ v[:, hk] / Z, p @ av / Z
            ds = abs(scale) * D / 16 * 2.0 ** -20 * (np.abs(q[r0:r1, h]) @ np.abs(k[:, hk]).T).max(-1, keepdims=True)
            tol[r0:r1, h] = (2.0 ** -8 * np.abs(out[r0:r1, h]) + mag * (2.0 ** -11 + L / 16 * 2.0 ** -20 + 2.0 ** -16 + np.expm1(2 * ds))
                             + 2.0 ** -25 * (~late @ av) / Z)
    return out, tol
