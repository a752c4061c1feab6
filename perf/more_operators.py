"""Drafted tokens, sliding windows and page bookkeeping on the GPU, as operators to be measured.

Five operators over the paged K/V pools (bf16, FP8 E4M3, INT4) that belong to one loop: block tables
and slots extended on the GPU from lengths, attention for trees of drafted tokens behind a cached
context, single-token and chunk attention with a sliding window and sink tokens, and the rows of the
accepted path moved to where they belong.

Row i of a sequence with C cached and P new positions, whose keys are at positions 0 .. C + P - 1:

  chunk or chain: the row is position p = C + i and sees j <= p with j > p - window or j < sinks;
  tree: bit j of the row's mask words says whether it sees new position C + j; with n such bits it
  counts as position p = C + n - 1 and sees the cached j < C with j > p - window or j < sinks.

window 0 is no window.  A row that sees nothing gives zeros.

`own` False: each operator in elementary torch operations in 32 bits.  `own` True: the library.
"""
import math

import numpy as np
import torch

own = False

BS = 16                                       # tokens per block
K_SCALE, V_SCALE = 0.0131, 0.0087             # the FP8 and INT4 pools' scales


# ------------------------------------------------------------------------------ cases
def listed():
    return [
        # one conversation of the Llama-3-8B layout, a small tree of drafts: latency counts
        dict(name="tree of 13, one sequence", op="tree", kind="bf16", batch=1, heads=32, kv_heads=8, dim=128, lens="fixed", length=333, new=13, ragged=False, tree=True, window=0, sinks=0, lens_seed=1),
        # the repository's headline batch, verifying eight drafts a sequence
        dict(name="tree 64 x 2048, 8 drafts", op="tree", kind="bf16", batch=64, heads=32, kv_heads=8, dim=128, lens="fixed", length=2048, new=8, ragged=False, tree=True, window=0, sinks=0, lens_seed=2),
        # an uneven batch of the Qwen2.5-7B layout over an INT4 pool, trees of different sizes
        dict(name="tree 37 ragged, INT4", op="tree", kind="int4", batch=37, heads=28, kv_heads=4, dim=128, lens="uniform", length=4096, new=25, ragged=True, tree=True, window=0, sinks=0, lens_seed=3),
        # large trees of the Llama-3-70B layout over an FP8 pool: bound by the products
        dict(name="tree 16 x 61 drafts, FP8", op="tree", kind="fp8", batch=16, heads=64, kv_heads=8, dim=128, lens="uniform", length=8192, new=61, ragged=False, tree=True, window=0, sinks=0, lens_seed=4),
        # three conversations of a small model with a short window
        dict(name="window 3 x 1900, FP8", op="window", kind="fp8", batch=3, heads=14, kv_heads=2, dim=64, lens="uniform", length=1900, window=250, sinks=3, lens_seed=5),
        # a ragged serving batch far beyond its window: what left the window is no longer in the pool
        dict(name="window 256 ragged", op="window", kind="bf16", batch=256, heads=32, kv_heads=8, dim=128, lens="uniform", length=16384, window=1024, sinks=4, lens_seed=6),
        # three short chunks that cross their window
        dict(name="chunks 3 short, FP8", op="chunk", kind="fp8", batch=3, heads=8, kv_heads=2, dim=64, lens="uniform", length=137, new=40, ragged=True, window=50, sinks=4, lens_seed=7),
        # the repository's chunked prefill with a window
        dict(name="chunks 16 x 512", op="chunk", kind="bf16", batch=16, heads=32, kv_heads=8, dim=128, lens="uniform", length=8192, new=512, ragged=False, window=1024, sinks=4, lens_seed=8),
        # a step's tables and slots: 64 sequences gain their drafts
        dict(name="extend 64 by 8", op="extend", batch=64, lens="uniform", length=2048, new=8, ragged=False, lens_seed=9),
        # a batch of whole prompts
        dict(name="extend 512 prompts", op="extend", batch=512, lens="empty", length=0, new=2000, ragged=True, lens_seed=10),
        # a small model's accepted rows, one layer
        dict(name="accept 5 trees, FP8", op="accept", kind="fp8", layers=1, batch=5, kv_heads=2, dim=64, lens="uniform", length=90, new=9, ragged=True, lens_seed=11),
        # eight layers of the headline layout, large trees
        dict(name="accept 64 trees, 8 layers", op="accept", kind="bf16", layers=8, batch=64, kv_heads=8, dim=128, lens="uniform", length=100, new=61, ragged=False, lens_seed=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "window", "window", "chunk", "chunk", "extend", "accept"])
    kv_heads, group = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 2, 3, 4, 7, 8, 16])
    dim, seed, kind = rng.choice([64, 128, 128]), rng.randrange(1 << 30), rng.choice(["bf16", "fp8", "int4"])
    shape = dict(kind=kind, heads=kv_heads * group, kv_heads=kv_heads, dim=dim)
    if op == "tree":
        new = _log(rng, 1, 130)
        batch = _log(rng, 1, 64)
        most = max(16, min(16384, 160_000 // batch, 250_000_000 // (batch * new * kv_heads * group)))
        return dict(op=op, **shape, batch=batch, lens=rng.choice(["fixed", "uniform", "lognormal"]), length=_log(rng, 1, most), new=new, ragged=rng.random() < 0.6,
                    tree=rng.random() < 0.8, window=rng.choice([0, max(new, _log(rng, 16, 4096))]), sinks=rng.randint(0, 40), lens_seed=seed)
    if op == "window":
        batch = _log(rng, 1, 256)
        return dict(op=op, **shape, batch=batch, lens=rng.choice(["fixed", "uniform", "lognormal"]), length=_log(rng, 1, 30000),
                    window=_log(rng, 1, max(16, 200_000 // batch)) if batch > 24 else _log(rng, 1, 8000), sinks=rng.randint(0, 40), lens_seed=seed)
    if op == "chunk":
        new, length, window = _log(rng, 1, 500), _log(rng, 1, 8000), _log(rng, 1, 2000)
        batch = _log(rng, 1, max(1, min(16, (1 << 29) // (new * (new + window) * kv_heads * group))))
        return dict(op=op, **shape, batch=batch, lens="uniform", length=length, new=new, ragged=rng.random() < 0.7, window=window, sinks=rng.randint(0, 40), lens_seed=seed)
    if op == "extend":
        batch = _log(rng, 1, 512)
        return dict(op=op, batch=batch, lens=rng.choice(["empty", "uniform"]), length=_log(rng, 1, 8000), new=_log(rng, 1, 500_000 // batch), ragged=rng.random() < 0.7, lens_seed=seed)
    return dict(op=op, kind=kind, layers=rng.choice([1, 2, 5]), batch=_log(rng, 1, 64), kv_heads=kv_heads, dim=dim, lens="uniform", length=_log(rng, 1, 100),
                new=_log(rng, 1, 130), ragged=rng.random() < 0.7, lens_seed=seed)


# ------------------------------------------------------------------------------ sizes of a case
def _blocks(n):
    return -(-np.asarray(n) // BS)


def _lengths(c):
    """(cached, new) positions of every sequence."""
    r = np.random.Generator(np.random.PCG64(c["lens_seed"]))
    n = c["batch"]
    if c["lens"] == "fixed":
        C = np.full(n, c["length"])
    elif c["lens"] == "empty":
        C = np.zeros(n)
    elif c["lens"] == "uniform":
        C = r.integers(0, c["length"], size=n, endpoint=True)
    else:
        C = np.clip(np.rint(np.exp(r.normal(math.log(0.35 * c["length"] + 1), 0.6, size=n))), 1, c["length"])
    P = np.ones(n) if c["op"] == "window" else r.integers(1, c["new"], size=n, endpoint=True) if c.get("ragged") else np.full(n, c["new"])
    return C.astype(np.int32), P.astype(np.int32)


def _parents(c, P):
    """The parent of every drafted token among its sequence's (-1: the last cached token), children behind parents."""
    r = np.random.Generator(np.random.PCG64(c["lens_seed"] + 1))
    return [np.array([-1] + [int(r.integers(max(0, i - 7), i)) if r.random() < 0.95 else -1 for i in range(1, p)], np.int64) for p in P]


def _mask_words(parents, words):
    """Mask words [rows, words]: bit j of a row where drafted token j is the row itself or above it."""
    out = np.zeros((sum(len(p) for p in parents), words), np.uint64)
    at = 0
    for par in parents:
        for i, up in enumerate(par):
            if up >= 0:
                out[at + i] = out[at + up]
            out[at + i, i // 64] |= np.uint64(1 << (i % 64))
        at += len(par)
    return out.view(np.int64)


def _paths(c, P):
    """The accepted path of every sequence, from a root down, padded with -1, and how long it is."""
    r = np.random.Generator(np.random.PCG64(c["lens_seed"] + 2))
    path, count = np.full((len(P), int(P.max())), -1, np.int32), np.zeros(len(P), np.int32)
    for b, par in enumerate(_parents(c, P)):
        i, up = int(r.integers(0, len(par))), []
        while i >= 0:
            up.append(i)
            i = int(par[i])
        count[b] = int(r.integers(0, len(up), endpoint=True))
        path[b, : len(up)] = up[::-1]
    return path, count


def _row_bytes(c):
    return c["kv_heads"] * c["dim"] * {"bf16": 32, "fp8": 16, "int4": 8.5}[c["kind"]] / 16


def _seen_by(c, C, P):
    """For every sequence, pairs (row, position) that are seen, and positions that some row sees."""
    pairs, union = 0, 0
    W, S = c["window"], c["sinks"]
    for n, p in zip(C.tolist(), P.tolist()):
        i = np.arange(p, dtype=np.int64)
        if c.get("tree"):
            pairs += p * (min(n, W + min(S, max(0, n - W))) if W else n) + p * (p + 1) // 4      # about: depths differ
        else:
            pos = n + i
            pairs += int((np.minimum(pos + 1, W) + np.minimum(S, np.maximum(0, pos + 1 - W))).sum() if W else (pos + 1).sum())
        lo = max(0, n - W) if W else 0
        union += n + p - lo + min(S, lo)
    return pairs, union


def work(c):
    C, P = _lengths(c)
    rows = int(P.sum())
    if c["op"] in ("tree", "window", "chunk"):
        pairs, union = _seen_by(c, C, P)
        return {"bytes": 2 * union * _row_bytes(c) + 2 * rows * c["heads"] * c["dim"] * 2 + union // BS * 4 + 8 * c["batch"], "flops": 4 * pairs * c["heads"] * c["dim"]}
    if c["op"] == "extend":                                                        # lengths in and out, an entry a new block, a slot and a position a row
        return {"bytes": 12 * c["batch"] + 8 * int((_blocks(C + P) - _blocks(C)).sum()) + 12 * rows, "flops": 2 * rows}
    path, count = _paths(c, P)
    moved = sum(int((path[b, :n] != np.arange(n)).sum()) for b, n in enumerate(count))
    return {"bytes": 4 * c["layers"] * moved * _row_bytes(c) + 4 * int(count.sum()) + 16 * c["batch"], "flops": 0}


# ------------------------------------------------------------------------------ the pools' elements
def _int4_places(D, device="cuda"):
    """For K, then V: the nibble's place of element (token, column) of an INT4 tile, and the byte of its scale."""
    t, d = torch.arange(BS, device=device)[:, None], torch.arange(D, device=device)[None, :]
    ng, j = D // 32, d // 32
    r = (t & 8) | (t & 3) << 1 | (t >> 2) & 1
    k = (r * (D // 8) + d % 32 // 8 * ng + j) * 8 + d % 8
    c = d % 32 // 4
    c = c ^ ((t & 2) << 1) if D == 128 else c
    v = (t * (D // 4) + c * ng + j) * 4 + d % 4
    return (k, 8 * D + r * ng + j), (v, 8 * D + (t & 3) * (D // 8) + 4 * j + (t >> 2))


def _values(tiles, kind, places, scale):
    """Elements [..., 16, D] of tiles in 32 bits."""
    if kind == "bf16":
        return tiles.float()
    if kind == "fp8":
        return tiles.view(torch.float8_e4m3fn).float() * scale
    nib, sc = places
    n = (tiles[..., nib // 2] >> (nib % 2 * 4).byte() & 15).float() - 8
    return n * (tiles[..., sc].view(torch.float8_e4m3fn).float() * scale)


# ------------------------------------------------------------------------------ inputs
def _cache(g, kind, shape, D, scale, gains):
    """One cache tensor [*shape, tile] of blocks that were all written."""
    if kind == "int4":
        n = (torch.randn(*shape, 16 * D, generator=g, device="cuda") * 3).round_().clamp_(-7, 7).add_(8).byte()
        n = n[..., 0::2] | n[..., 1::2] << 4
        s = ((2 + torch.rand(*shape, D // 2, generator=g, device="cuda")) / (7 * scale)).to(torch.float8_e4m3fn)
        return torch.cat([n, s.view(torch.uint8)], -1)
    x = torch.randn(*shape, BS, D, generator=g, device="cuda")
    if gains:                                                                      # keys have a few channels larger than the rest
        x *= torch.where(torch.rand(D, generator=g, device="cuda") < 0.03, 3.0, 1.0)
    return x.bfloat16() if kind == "bf16" else (x / scale).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _tables(g, C, P, blocks, window, sinks):
    """Block tables over shuffled physical blocks: -1 where a row needs no more, and where no row of the sequence sees a block."""
    nb = _blocks(C + P)
    col = np.arange(int(nb.max()))[None, :]
    used = col < nb[:, None]
    if window:
        used &= (col * BS < sinks) | (col >= np.maximum(0, C - window)[:, None] // BS)
    used = torch.from_numpy(used).cuda()
    t = torch.full(used.shape, -1, dtype=torch.int32, device="cuda")
    n = int(used.sum())
    t[used] = torch.randperm(n if blocks is None else blocks, generator=g, device="cuda")[:n].int()
    return t, n


def _pool(c, blocks, layers=1):
    import paged_kv_cache_159_gb300 as pkv
    kind = {"bf16": pkv.KV_BF16, "fp8": pkv.KV_FP8E4M3, "int4": pkv.KV_INT4}[c.get("kind", "bf16")]
    scales = {} if kind == pkv.KV_BF16 else dict(k_scale=K_SCALE, v_scale=V_SCALE)
    p = pkv.Pool(blocks, c.get("kv_heads", 1), c.get("dim", 64), kv_dtype=kind, num_layers=layers, **scales)
    p.attach_device(torch.cuda.current_device())
    return p


def prepare(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    C, P = _lengths(c)
    B, rows, L = c["batch"], int(P.sum()), C + P
    cu = np.concatenate([[0], np.cumsum(P)]).astype(np.int32)
    s = dict(case=c, P=torch.from_numpy(P).cuda(), cu=torch.from_numpy(cu).cuda())
    if c["op"] == "extend":
        fresh = int((_blocks(L) - _blocks(C)).sum())
        blocks, MB = int(_blocks(L).sum()), int(_blocks(L).max())
        ids = torch.randperm(blocks, generator=g, device="cuda").int()
        s["reserve"] = ids[: fresh + 5].contiguous() if blocks >= fresh + 5 else ids
        held = torch.arange(MB, device="cuda") < torch.from_numpy(_blocks(C)).cuda()[:, None]
        s["tables"] = torch.full((B, MB), -1, dtype=torch.int32, device="cuda")
        s["tables"][held] = ids[blocks - int(held.sum()):]
        s["lens"], s["cursor"] = torch.from_numpy(C).cuda(), torch.zeros(2, dtype=torch.int32, device="cuda")
        s["new_lens"] = torch.empty(B, dtype=torch.int32, device="cuda")
        s["slots"], s["positions"] = torch.empty(rows, dtype=torch.int64, device="cuda"), torch.empty(rows, dtype=torch.int32, device="cuda")
        if own:
            s["pool"] = _pool(c, blocks)
        return s
    Hkv, D, kind = c["kv_heads"], c["dim"], c["kind"]
    layers = c.get("layers", 1)
    s["tables"], blocks = _tables(g, C, P, None, c.get("window", 0), c.get("sinks", 0))
    shape = (blocks, Hkv) if layers == 1 else (layers, blocks, Hkv)
    s["kc"], s["vc"] = _cache(g, kind, shape, D, K_SCALE, True), _cache(g, kind, shape, D, V_SCALE, False)
    s["lens"], s["places"] = torch.from_numpy(L).cuda(), _int4_places(D)
    if own:
        s["pool"] = _pool(c, blocks, layers)
    if c["op"] == "accept":
        path, count = _paths(c, P)
        s["path"], s["count"] = torch.from_numpy(path).cuda(), torch.from_numpy(count).cuda()
        s["new_lens"] = torch.empty(B, dtype=torch.int32, device="cuda")
        if kind == "int4":
            pos = np.concatenate([np.arange(a, b) for a, b in zip(C, L)])
            row = np.repeat(np.arange(B), P)
            t = s["tables"].long()[torch.from_numpy(row).cuda(), torch.from_numpy(pos // BS).cuda()]
            s["slots"] = t * BS + torch.from_numpy(pos % BS).cuda()
            s["k"], s["v"] = (torch.empty(layers, rows, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        return s
    s["q"] = torch.randn(rows, c["heads"], D, generator=g, device="cuda").bfloat16()
    s["out"] = torch.empty_like(s["q"])
    s["scale"] = float(np.float32(1 / math.sqrt(D)))
    s["mask"] = None
    if c.get("tree"):
        s["mask"] = torch.from_numpy(_mask_words(_parents(c, P), -(-c["new"] // 64))).cuda()
    if own:
        import paged_kv_cache_159_gb300 as pkv
        if c["op"] == "chunk":
            MB = s["tables"].shape[1]
            plan, s["grid"] = pkv.prefill_plan(s["pool"], cu, L, c["heads"], MB, window=c["window"], sinks=c["sinks"])
            s["plan"] = torch.from_numpy(plan).cuda()
            n = pkv.prefill_workspace_bytes(s["pool"], cu, L, MB, window=c["window"], sinks=c["sinks"])
        else:
            n = pkv.tree_workspace_bytes(s["pool"], B, c["heads"], c.get("new", 1))
        s["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------------------ one pass
def _attend(s):
    """Masked attention of every sequence's rows, padded to the most rows, over the blocks that some row sees."""
    c, lens, P = s["case"], s["lens"].long(), s["P"].long()
    W, S, B = c["window"], c["sinks"], c["batch"]
    g, D, n = c["heads"] // c["kv_heads"], c["dim"], int(c.get("new", 1))
    MB, C = s["tables"].shape[1], lens - P
    if W:                                                                          # blocks of the sinks, then those from the window's first on
        sb = min(MB, -(-S // BS))
        first = ((C - W).clamp(min=0) // BS).clamp(min=sb)
        blk = torch.cat([torch.arange(sb, device="cuda").expand(B, sb), first[:, None] + torch.arange(min(MB, (W + n) // BS + 2), device="cuda")], 1)
    else:
        blk = torch.arange(MB, device="cuda").expand(B, MB)
    ids = s["tables"].gather(1, blk.clamp(max=MB - 1)).clamp(min=0).long()
    k = _values(s["kc"][ids], c["kind"], s["places"][0], K_SCALE).transpose(1, 2).flatten(2, 3)
    v = _values(s["vc"][ids], c["kind"], s["places"][1], V_SCALE).transpose(1, 2).flatten(2, 3)
    j = (blk[:, :, None] * BS + torch.arange(BS, device="cuda")).flatten(1)[:, None, :]      # [B, 1, N]
    i = torch.arange(n, device="cuda")
    real = i < P[:, None]
    ctx, end = C[:, None, None], lens[:, None, None]
    if s["mask"] is None:
        p = ctx + i[:, None]
        seen = (j <= p) & (j < end)
    else:
        m = torch.zeros(B, n, s["mask"].shape[1], dtype=torch.int64, device="cuda")
        m[real] = s["mask"]
        d = torch.arange(n, device="cuda")
        p = ctx - 1 + (m[:, :, d // 64] >> (d % 64) & (d < P[:, None, None])).sum(-1, keepdim=True)
        e = (j - ctx).clamp(0, 64 * m.shape[2] - 1).expand(B, n, -1)
        seen = (j < ctx) | ((j < end) & (m.gather(2, e // 64) >> (e % 64) & 1).bool())
    if W:
        seen = seen & ((j >= ctx) & (s["mask"] is not None) | (j > p - W) | (j < S))
    q = torch.zeros(B, n, c["heads"], D, device="cuda")
    q[real] = s["q"].float()
    q = q.unflatten(2, (c["kv_heads"], g)).permute(0, 2, 3, 1, 4).flatten(2, 3)              # [B, Hkv, g * n, D]
    seen = seen[:, None, None].expand(-1, 1, g, -1, -1).flatten(2, 3)
    x = (q @ k.transpose(-1, -2)).mul_(s["scale"]).masked_fill_(~seen, -math.inf)
    x = x.sub_(x.amax(-1, keepdim=True).clamp(min=-1e30)).exp_()
    z = x.sum(-1, keepdim=True)
    out = ((x @ v) / torch.where(z > 0, z, 1.0)).unflatten(2, (g, n)).permute(0, 3, 1, 2, 4).flatten(2, 3)
    return out[real].bfloat16()


def _extend(s):
    """Empty entries of the blocks that gain positions filled from the reserve, in the sequences' order; every new position's slot."""
    B, MB = s["tables"].shape
    L = s["lens"].long()
    end = L + s["P"]
    col = torch.arange(MB, device="cuda")
    t = s["tables"]
    empty = (col >= (L // BS)[:, None]) & (col < ((end + BS - 1) // BS)[:, None]) & (t < 0)
    nth = empty.flatten().cumsum(0) - 1 + s["cursor"][0]
    t.copy_(torch.where(empty, s["reserve"][nth.clamp(0, s["reserve"].numel() - 1)].view(B, MB), t))
    s["cursor"][0] += empty.sum()
    row = torch.arange(B, device="cuda").repeat_interleave(s["P"].long(), output_size=s["slots"].numel())
    pos = torch.arange(s["slots"].numel(), device="cuda") - s["cu"].long()[row] + L[row]
    s["slots"].copy_(t[row, pos // BS].long() * BS + pos % BS)
    s["positions"].copy_(pos)
    s["new_lens"].copy_(end)
    return t, s["cursor"][:1], s["new_lens"], s["slots"], s["positions"]


def _slots_of(s, pos):
    return s["tables"].long().gather(1, pos // BS) * BS + pos % BS


def _accept(s):
    c = s["case"]
    C = (s["lens"] - s["P"]).long()[:, None]
    i = torch.arange(s["path"].shape[1], device="cuda")
    take = i < s["count"][:, None]
    src, dst = (torch.where(take, _slots_of(s, x), 0)[take] for x in (torch.where(take, C + s["path"], 0), torch.where(take, C + i, 0)))
    s["new_lens"].copy_(C[:, 0] + s["count"])
    D, got = c["dim"], []
    for cache, (nib, sc) in ((s["kc"], s["places"][0]), (s["vc"], s["places"][1])):
        x = cache if c["layers"] > 1 else cache[None]
        if c["kind"] != "int4":
            x[:, dst // BS, :, dst % BS] = x[:, src // BS, :, src % BS]
            got.append(cache if c["kind"] == "bf16" else cache.view(torch.float8_e4m3fn))
            continue
        # a token's codes and scales have bytes of their own in a tile: those of the one token to those of the other
        byte = torch.cat([nib.sort(-1).values[:, 0::2] // 2, sc[:, ::32]], 1)
        code = x[:, src // BS][..., :8 * D].view(c["layers"], -1, c["kv_heads"], 8 * D)
        n = (code.gather(3, (nib // 2)[src % BS][None, :, None].expand(c["layers"], -1, c["kv_heads"], -1)) >> (nib % 2 * 4).byte()[src % BS][:, None]) & 15
        back = nib.argsort(-1)[dst % BS][None, :, None].expand(n.shape)
        n = n.gather(3, back)
        e = x[:, src // BS].gather(3, sc[:, ::32][src % BS][None, :, None].expand(c["layers"], -1, c["kv_heads"], -1))
        at = byte[dst % BS][None, :, None].expand(c["layers"], -1, c["kv_heads"], -1)
        start = (torch.arange(c["layers"], device="cuda")[:, None, None] * x.stride(0) + (dst // BS)[:, None] * x.stride(1) + torch.arange(c["kv_heads"], device="cuda") * x.stride(2))[..., None]
        x.view(-1)[start + at] = torch.cat([n[..., 0::2] | n[..., 1::2] << 4, e], -1)
    if c["kind"] == "int4":
        for cache, places, scale in ((s["kc"], s["places"][0], K_SCALE), (s["vc"], s["places"][1], V_SCALE)):
            x = cache if c["layers"] > 1 else cache[None]
            rows = _values(x[:, s["slots"] // BS], "int4", places, scale)
            got.append(rows[:, torch.arange(rows.shape[1], device="cuda"), :, s["slots"] % BS].transpose(0, 1).bfloat16())
    return (*got, s["new_lens"])


def run(s):
    c = s["case"]
    if own:
        import paged_kv_cache_159_gb300 as pkv
        p = s["pool"]
        if c["op"] == "tree":
            pkv.paged_attention_tree(p, s["q"], s["kc"], s["vc"], s["tables"], s["lens"], s["cu"], s["mask"], c["new"], s["scale"], s["out"], s["ws"], window=c["window"], sinks=c["sinks"])
            return s["out"]
        if c["op"] == "window":
            pkv.paged_attention_window(p, s["q"], s["kc"], s["vc"], s["tables"], s["lens"], s["scale"], c["window"], c["sinks"], s["out"], s["ws"])
            return s["out"]
        if c["op"] == "chunk":
            pkv.paged_prefill(p, s["q"], s["kc"], s["vc"], s["tables"], s["scale"], s["plan"], s["grid"], s["out"], workspace=s["ws"])
            return s["out"]
        if c["op"] == "extend":
            pkv.extend_tables(p, s["lens"], s["cu"], s["tables"], s["reserve"], s["cursor"], s["new_lens"], s["slots"], s["positions"])
            return s["tables"], s["cursor"][:1], s["new_lens"], s["slots"], s["positions"]
        pkv.accept_rows(p, s["kc"], s["vc"], s["tables"], s["lens"], s["cu"], s["path"], s["count"], s["new_lens"])
        if c["kind"] == "int4":
            pkv.kv_gather_layers(p, s["slots"], s["kc"], s["vc"], s["k"], s["v"])
            return s["k"], s["v"], s["new_lens"]
        got = (s["kc"], s["vc"]) if c["kind"] == "bf16" else (s["kc"].view(torch.float8_e4m3fn), s["vc"].view(torch.float8_e4m3fn))
        return (*got, s["new_lens"])
    return _extend(s) if c["op"] == "extend" else _accept(s) if c["op"] == "accept" else _attend(s)


# ------------------------------------------------------------------------------ the definition in 64 bits
def _e4m3_values():
    x = []
    for b in range(256):
        e, m = b >> 3 & 15, b & 7
        v = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        x.append(-v if b > 127 else v)
    return torch.tensor(x, dtype=torch.float64, device="cuda")


def _tile_bits(D, key):
    """For (token, column) of an INT4 tile the byte and shift of its code and the byte of its scale, by the format's words."""
    at, sh, sc = (np.zeros((BS, D), np.int64) for _ in range(3))
    ng = D // 32
    for t in range(BS):
        for d in range(D):
            j, e = divmod(d, 32)
            if key:
                r = 8 * (t // 8) + 2 * (t % 4) + t // 4 % 2
                bit = r * 4 * D + 32 * (e // 8 * ng + j) + 4 * (e % 8)
                sc[t, d] = 8 * D + r * ng + j
            else:
                word = e // 4 if D == 64 or t // 2 % 2 == 0 else (e // 4 + 4) % 8
                bit = t * 4 * D + 16 * (word * ng + j) + 4 * (e % 4)
                sc[t, d] = 8 * D + t % 4 * 4 * ng + 4 * j + t // 4
            at[t, d], sh[t, d] = bit // 8, bit % 8
    return [torch.from_numpy(x).cuda() for x in (at, sh, sc)]


def _rows64(cache, kind, blk, t, key, bits):
    """Rows (block, token) of a cache [NB, Hkv, ...] in 64 bits: [n, Hkv, D]."""
    scale = K_SCALE if key else V_SCALE
    if kind == "bf16":
        return cache[blk, :, t].double()
    e = _e4m3_values()
    if kind == "fp8":
        return e[cache[blk, :, t].long()] * float(np.float32(scale))
    at, sh, sc = (x[t][:, None, :].expand(-1, cache.shape[1], -1) for x in bits)
    tiles = cache[blk]
    return ((tiles.gather(2, at) >> sh.byte() & 15).double() - 8) * e[tiles.gather(2, sc).long()] * float(np.float32(scale))


def exact(c, seed):
    s = prepare(c, seed)
    C, P = _lengths(c)
    if c["op"] == "extend":
        t, left, slots, positions = s["tables"].tolist(), s["reserve"].tolist()[::-1], [], []
        start = len(left)
        for b, (n, p) in enumerate(zip(C.tolist(), P.tolist())):
            for pos in range(n, n + p):
                if t[b][pos // BS] < 0:
                    t[b][pos // BS] = left.pop()
                slots.append(t[b][pos // BS] * BS + pos % BS)
                positions.append(pos)
        return [torch.tensor(x) for x in (t, [start - len(left)], (C + P).tolist(), slots, positions)]
    D, kind = c["dim"], c["kind"]
    bits = [_tile_bits(D, True), _tile_bits(D, False)] if kind == "int4" else [None, None]
    if c["op"] == "accept":
        path, count = _paths(c, P)
        tables = s["tables"].tolist()
        slot = lambda b, pos: (tables[b][pos // BS], pos % BS)  # noqa: E731
        got = []
        for cache, key in ((s["kc"], True), (s["vc"], False)):
            x = cache if c["layers"] > 1 else cache[None]
            if kind == "int4":                                                     # the rows that the slots then stand for
                after = []
                for b in range(c["batch"]):
                    order = list(range(int(P[b])))
                    for j in range(int(count[b])):
                        order[j] = int(path[b, j])
                    after += [slot(b, int(C[b]) + i) for i in order]
                blk, t = (torch.tensor(v, device="cuda") for v in zip(*after))
                got.append(torch.stack([_rows64(y, kind, blk, t, key, bits[0 if key else 1]) for y in x]))
                continue
            x = x.double() if kind == "bf16" else _e4m3_values()[x.long()]
            for b in range(c["batch"]):
                for j in range(int(count[b])):
                    (a, u), (z, w) = slot(b, int(C[b]) + int(path[b, j])), slot(b, int(C[b]) + j)
                    x[:, z, :, w] = x[:, a, :, u]
            got.append(x if c["layers"] > 1 else x[0])
        return (*got, torch.from_numpy(C + count))
    W, S, group = c["window"], c["sinks"], c["heads"] // c["kv_heads"]
    above = _parents(c, P) if c.get("tree") else None
    out, row = [], 0
    for b in range(c["batch"]):
        n, p = int(C[b]), int(P[b])
        see = np.zeros((p, n + p), bool)
        for i in range(p):
            if above is None:
                see[i, : n + i + 1] = True
                if W:
                    see[i, S : max(S, n + i + 1 - W)] = False
                continue
            chain, at = [], i
            while at >= 0:
                chain.append(at)
                at = int(above[b][at])
            see[i, :n] = True
            if W:
                see[i, S : max(S, min(n, n + len(chain) - W))] = False
            see[i, [n + x for x in chain]] = True
        pos = torch.from_numpy(np.flatnonzero(see.any(0))).cuda()
        see = torch.from_numpy(see).cuda()[:, pos]
        blk = s["tables"][b].long()[pos // BS]
        k, v = _rows64(s["kc"], kind, blk, pos % BS, True, bits[0]), _rows64(s["vc"], kind, blk, pos % BS, False, bits[1])
        q = s["q"][row : row + p].double()
        o = torch.empty_like(q)
        for h in range(c["heads"]):
            w = (q[:, h] @ k[:, h // group].T * s["scale"]).masked_fill(~see, -math.inf)
            o[:, h] = torch.softmax(w, -1) @ v[:, h // group]
        out.append(o)
        row += p
    return torch.cat(out)
