"""Block tables and slots extended on the GPU, and the rows of an accepted draft path, against plain models."""
import numpy as np
import pytest
import torch

import paged_kv_cache_159_gb300 as pkv
from tests import _drafts as T

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    return pkv.lib()


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


class Step:
    """extend_tables on device copies, and the same in plain Python."""

    def __init__(self, lens, new, MB, held=None, spare=4, pad=0, seed=0, NB=None):
        rng = np.random.default_rng(seed)
        self.lens, self.new, self.MB = np.array(lens, np.int32), np.array(new, np.int32), MB
        self.cu = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)
        held = -(-self.lens // 16) if held is None else np.array(held)
        want = np.maximum(0, -(-(self.lens + self.new) // 16) - held)
        self.NB = int(held.sum() + want.sum()) + spare if NB is None else NB
        ids = rng.permutation(self.NB).astype(np.int32)
        self.tables = np.full((len(lens), MB), -1, np.int32)
        at = 0
        for b, n in enumerate(held):
            self.tables[b, :n] = ids[at:at + n]
            at += n
        self.reserve = ids[at:]
        self.total = int(self.cu[-1]) + pad
        self.pool = pkv.Pool(self.NB, 2, 64)
        self.pool.attach_device(torch.cuda.current_device())
        self.reset()

    def reset(self):
        self.d = dict(lens=i32(self.lens), cu=i32(self.cu), tables=i32(self.tables), reserve=i32(self.reserve), state=i32([0, 0]),
                      new_lens=torch.full((len(self.lens),), -9, dtype=torch.int32, device="cuda"),
                      slots=torch.full((self.total,), -9, dtype=torch.int64, device="cuda"),
                      positions=torch.full((self.total,), -9, dtype=torch.int32, device="cuda"))

    def run(self, error=(pkv.OK, 0), **kw):
        a = {**self.d, **kw}
        pkv.extend_tables(self.pool, a["lens"], a["cu"], a["tables"], a["reserve"], a["state"], a["new_lens"], a["slots"], a["positions"])
        assert self.pool.get_device_error() == error

    def plain(self):
        t, used, slots, pos, filled = self.tables.copy(), 0, [], [], set()
        for b, (n, p) in enumerate(zip(self.lens.tolist(), self.new.tolist())):
            for x in range(n, n + p):
                if t[b, x // 16] < 0 and (b, x // 16) not in filled:
                    filled.add((b, x // 16))
                    t[b, x // 16] = self.reserve[used]
                    used += 1
                slots.append(int(t[b, x // 16]) * 16 + x % 16)
                pos.append(x)
        pad = self.total - len(slots)
        return t, used, self.lens + self.new, slots + [-1] * pad, pos + [0] * pad

    def check(self):
        t, used, lens, slots, pos = self.plain()
        d = self.d
        assert np.array_equal(d["tables"].cpu().numpy(), t) and d["state"].tolist() == [used, 0]
        assert d["new_lens"].tolist() == lens.tolist() and d["slots"].tolist() == slots and d["positions"].tolist() == pos

    def unchanged(self):
        d = self.d
        assert np.array_equal(d["tables"].cpu().numpy(), self.tables) and d["state"][0] == 0
        assert d["new_lens"].tolist() == self.lens.tolist() and (d["slots"] == -1).all() and (d["positions"] == 0).all()


@pytest.mark.parametrize("lens,new", [([0], [1]), ([15], [1]), ([16], [1]), ([17, 0, 31, 32], [1, 33, 2, 0]), ([0, 0], [0, 0]),
                                      ([5] * 40, [8] * 40), ([0, 700, 3], [900, 1, 16])])
@pytest.mark.parametrize("pad", [0, 7])
def test_extend(lens, new, pad):
    s = Step(lens, new, 70, pad=pad)
    s.run()
    s.check()
    s.run()                                        # the same step again: every entry is there already
    s.check()


@pytest.mark.parametrize("batch", [1, 31, 1023, 1024, 1025, 4096])
def test_extend_batches(batch):
    rng = np.random.default_rng(batch)
    s = Step(rng.integers(0, 50, batch), rng.integers(0, 20, batch), 6, seed=batch, pad=3)
    s.run()
    s.check()


@pytest.mark.parametrize("total", [8191, 8192, 8193, 60000])
def test_extend_many_rows(total):
    rng = np.random.default_rng(total)
    cut = np.sort(rng.integers(0, total + 1, 6))
    s = Step([0, 3, 16, 17, 0, 40, 0], np.diff(np.concatenate([[0], cut, [total]])), 4000, seed=total, pad=total % 5)
    s.run()
    s.check()


def test_extend_fills_only_what_is_empty():
    # blocks that a refused draft left behind are used before the reserve; freed ones in front stay empty
    s = Step([20, 64, 31], [40, 20, 1], 8, held=[3, 6, 2])
    s.tables[1, :3] = -1
    s.reset()
    s.run()
    s.check()


def test_extend_matches_the_host_allocator():
    lens, new = [3, 0, 50, 16], [14, 5, 30, 1]
    pool = pkv.Pool(40, 2, 64)
    pool.attach_device(torch.cuda.current_device())
    tables = pool.build_block_tables([max(1, n) for n in lens], 8)
    tables[1] = -1
    s = Step(lens, new, 8, NB=40)
    s.tables, s.reserve, s.pool = tables, pool.alloc(12), pool
    s.reset()
    s.run()
    got = s.d["tables"].cpu().numpy()
    end = np.array(lens) + np.array(new)
    assert s.d["slots"].tolist() == pkv.slot_mapping_chunks(got, end, s.cu).tolist()
    used = [x for r, t in zip(got, tables) for x, y in zip(r, t) if y < 0 and x >= 0]
    assert used == s.reserve[:len(used)].tolist() and s.d["state"][0] == len(used)


def test_extend_in_place_and_captured():
    s = Step([3, 0, 30], [5, 5, 5], 40, NB=90)
    lens, state, tables, slots = s.d["lens"], s.d["state"], s.d["tables"], s.d["slots"]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkv.extend_tables(s.pool, lens, s.d["cu"], tables, s.d["reserve"], state, lens, slots, None)
    for step in range(20):
        g.replay()
        s.lens = np.array([3, 0, 30], np.int32) + 5 * step
        t, used, end, want, _ = s.plain()
        assert slots.tolist() == want and lens.tolist() == end.tolist()
        s.tables, s.reserve = t, s.reserve[used:]
    assert np.array_equal(tables.cpu().numpy(), s.tables)
    assert state[0] == sum(-(-(n + 100) // 16) - -(-n // 16) for n in (3, 0, 30))
    assert s.pool.get_device_error() == (pkv.OK, 0)


@pytest.mark.parametrize("many", [False, True])
def test_extend_refuses_as_a_whole(many):
    rows = 9000 if many else 40
    for lens, new, MB, cu, bit in (([0, 5], [rows, 20], 600, None, "reserve"), ([0, 600 * 16 - 3], [rows, 4], 600, None, "len"),
                                   ([0, -1], [rows, 4], 600, None, "len"), ([0, 5], [rows, 4], 600, [0, 9, 8], "len"),
                                   ([0, 5], [rows, 4], 600, [1, 9, 10], "len"), ([0, 5], [rows, 4], 600, [0, 9, 10 ** 6], "len"),
                                   ([2 ** 31 - 1, 5], [rows, 4], 600, None, "len")):
        s = Step([0, 5], new, MB, seed=3)
        s.lens = np.array(lens, np.int64).astype(np.int32)
        if bit == "reserve":
            s.reserve = s.reserve[:-(-rows // 16)]
        s.reset()
        if cu:
            s.d["cu"] = i32(cu)
        s.run(error=(pkv.ERR_DEVICE, pkv.DEVERR_RESERVE if bit == "reserve" else pkv.DEVERR_SEQ_LEN))
        s.unchanged()
        assert s.d["state"][1] == 1
    s = Step([0, 5], new, 600)
    s.d["state"] = i32([-1, 0])                    # a cursor that is none
    s.run(error=(pkv.ERR_DEVICE, pkv.DEVERR_RESERVE))
    assert (s.d["slots"] == -1).all() and s.d["state"][0] == -1


def test_extend_flags_ids_outside_the_pool():
    s = Step([0, 5], [40, 20], 6)
    s.reserve[1] = s.NB
    s.reserve[2] = -5
    s.reset()
    s.run(error=(pkv.ERR_DEVICE, pkv.DEVERR_BLOCK_ID))
    t, used, _, slots, _ = s.plain()
    t[0, 1:3] = -1
    assert np.array_equal(s.d["tables"].cpu().numpy(), t)
    assert s.d["slots"].tolist() == slots[:16] + [-1] * 24 + slots[40:]


def test_extend_refusals():
    s = Step([0, 5], [40, 20], 6)
    d = s.d
    bad = pkv.Pool(s.NB, 2, 64)
    with pytest.raises(pkv.PkvError) as e:
        pkv.extend_tables(bad, d["lens"], d["cu"], d["tables"], d["reserve"], d["state"], d["new_lens"], d["slots"])
    assert e.value.status == pkv.ERR_INVALID
    big = Step([0] * 4097, [1] * 4097, 1)
    with pytest.raises(pkv.PkvError):
        big.run()
    for kw in (dict(lens=d["lens"][:1]), dict(cu=d["cu"][:2]), dict(cu=d["cu"].long()), dict(new_lens=d["new_lens"][:1]), dict(state=d["state"][:1]),
               dict(slots=d["slots"].int()), dict(positions=d["positions"][1:]), dict(tables=d["tables"].t())):
        with pytest.raises(ValueError):
            s.run(**kw)
    s.run()
    s.check()


# ------------------------------------------------------------------------------ accepted rows
class Accept:
    def __init__(self, kind, cached, new, Hkv, D, layers=1, seed=0, every=False):
        rng = np.random.default_rng(seed)
        self.c = T.Case(cached, new, Hkv, Hkv, D, kind, seed=seed, free=False)
        c = self.c
        self.layers = layers
        pages = [T.Pages(kind, c.NB, Hkv, D) for _ in range(layers)]
        g = torch.Generator().manual_seed(seed + 1)
        live = np.concatenate([c.slots(b, np.arange(n)) for b, n in enumerate(c.L)])
        for p in pages:
            p.write(live, [torch.randn(len(live), Hkv, D, generator=g).bfloat16() for _ in range(2)])
        self.pages = pages
        most = max(1, int(c.P.max()))
        self.path, self.n = np.full((len(c.P), most), -1, np.int32), np.zeros(len(c.P), np.int32)
        for b, P in enumerate(c.P.tolist()):
            k = P if every else int(rng.integers(0, P + 1))
            self.path[b, :k] = np.sort(rng.permutation(P)[:k])
            self.n[b] = k
        ks, vs = pages[0].scales
        self.pool = pkv.Pool(c.NB, Hkv, D, T.KINDS[kind], ks, vs, num_layers=layers)
        self.pool.attach_device(torch.cuda.current_device())
        self.reset()

    def reset(self):
        both = [torch.stack(x) for x in zip(*[p.device() for p in self.pages])]
        self.kc, self.vc = both if self.layers > 1 else [x[0] for x in both]
        c = self.c
        self.d = dict(tables=i32(c.tables), lens=i32(c.L), cu=i32(c.cu), path=i32(self.path), n=i32(self.n),
                      out=torch.full((len(c.P),), -9, dtype=torch.int32, device="cuda"))

    def run(self, error=(pkv.OK, 0), **kw):
        a = {**self.d, **kw}
        pkv.accept_rows(self.pool, self.kc, self.vc, a["tables"], a["lens"], a["cu"], a["path"], a["n"], a["out"])
        assert self.pool.get_device_error() == error

    def bits(self):
        return [x.view(torch.int16 if x.dtype == torch.bfloat16 else torch.uint8).cpu() for x in (self.kc, self.vc)]

    def check(self, skip=()):
        c = self.c
        for l in range(self.layers):
            want = T.Pages(c.kind, c.NB, c.pages.caches[0].shape[1], c.D)
            got = T.Pages(c.kind, c.NB, c.pages.caches[0].shape[1], c.D)
            want.caches = self.pages[l].caches
            got.caches = [(x[l] if self.layers > 1 else x).numpy().view(w.dtype) for x, w in zip(self.bits(), want.caches)]
            src, dst, rest = [], [], []
            for b, (C, L) in enumerate(zip(c.C.tolist(), c.L.tolist())):
                n = 0 if b in skip else int(self.n[b])
                src += list(c.slots(b, [C + int(x) for x in self.path[b, :n]])) if n else []
                dst += list(c.slots(b, [C + j for j in range(n)])) if n else []
                rest += list(c.slots(b, list(range(C)) + list(range(C + n, L)))) if C + n < L or C else []
            for a, z in ((src, dst), (rest, rest)):              # moved rows, and all others as they were
                if len(a):
                    for x, y in zip(want.read(np.array(a)), got.read(np.array(z))):
                        assert np.array_equal(x, y)
        lens = [-9 if b in skip else int(c.C[b] + self.n[b]) for b in range(len(c.P))]
        assert self.d["out"].tolist() == lens


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int4"])
@pytest.mark.parametrize("D,Hkv,layers", [(64, 1, 1), (64, 3, 2), (128, 2, 1), (128, 8, 3)])
def test_accept(kind, D, Hkv, layers):
    a = Accept(kind, [0, 5, 15, 16, 33, 100], [1, 9, 17, 40, 0, 8], Hkv, D, layers, seed=D + Hkv)
    a.run()
    a.check()


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int4"])
def test_accept_of_long_paths(kind):
    a = Accept(kind, [7, 30, 0], [256, 130, 64], 2, 128, seed=5)
    a.run()
    a.check()


@pytest.mark.parametrize("kind", ["bf16", "int4"])
def test_accept_of_everything_changes_nothing(kind):
    a = Accept(kind, [7, 30], [20, 64], 2, 128, seed=5, every=True)
    before = a.bits()
    a.run()
    a.check()
    assert all(torch.equal(x, y) for x, y in zip(before, a.bits()))


@pytest.mark.parametrize("bad", ["descending", "twice", "range", "negative", "count", "negative count", "more than drafts", "length", "entry"])
def test_accept_leaves_a_bad_sequence_as_it_was(bad):
    a = Accept("bf16", [7, 30, 40], [20, 64, 10], 2, 64, seed=5)
    a.path[1, :4], a.n[1] = [1, 5, 9, 60], 4
    bit = pkv.DEVERR_PATH
    if bad == "descending":
        a.path[1, :4] = [1, 9, 5, 60]
    elif bad == "twice":
        a.path[1, :4] = [1, 5, 5, 60]
    elif bad == "range":
        a.path[1, 3] = 64
    elif bad == "negative":
        a.path[1, 0] = -1
    elif bad == "count":
        a.n[1] = 65
    elif bad == "negative count":
        a.n[1] = -1
    elif bad == "more than drafts":
        a.path[2, :12], a.n[2] = np.arange(12), 12
    elif bad == "length":
        bit = pkv.DEVERR_SEQ_LEN
    elif bad == "entry":
        bit = pkv.DEVERR_BLOCK_ID
    a.reset()
    skip = [2] if bad == "more than drafts" else [1]
    if bad == "length":
        a.d["lens"][1] = 63
    if bad == "entry":
        a.d["tables"][1, (30 + 60) // 16] = -1
    a.run(error=(pkv.ERR_DEVICE, bit))
    a.check(skip=skip)


def test_accept_refusals():
    a = Accept("fp8", [7, 30], [20, 64], 2, 64)
    d = a.d
    for kw in (dict(out=d["lens"]), dict(out=d["n"]), dict(out=d["cu"][1:]), dict(out=d["path"].view(-1)[3:5]), dict(out=d["tables"].view(-1)[1:3])):
        with pytest.raises(pkv.PkvError) as e:
            a.run(**kw)
        assert e.value.status == pkv.ERR_INVALID
    for kw in (dict(lens=d["lens"][:1]), dict(cu=d["cu"][:2]), dict(n=d["n"].long()), dict(out=d["out"][:1]), dict(path=d["path"][:1]),
               dict(path=d["path"].t())):
        with pytest.raises(ValueError):
            a.run(**kw)
    a.run()
    a.check()


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int4"])
def test_a_drafting_loop_on_the_gpu(kind):
    """Extend, append, attend, accept, captured once and replayed: every step's outputs and the cache at the
    end are those of the definition on the tokens that were kept."""
    Hq, Hkv, D, B, P, MB, NB = 8, 2, 64, 3, 6, 12, 40
    rng = np.random.default_rng(1)
    g = torch.Generator().manual_seed(1)
    scale = float(np.float32(1 / np.sqrt(D)))
    pages = T.Pages(kind, NB, Hkv, D)
    ks, vs = pages.scales
    pool = pkv.Pool(NB, Hkv, D, T.KINDS[kind], ks, vs)
    pool.attach_device(torch.cuda.current_device())
    kc, vc = pages.device()
    tables, lens, total = torch.full((B, MB), -1, dtype=torch.int32, device="cuda"), i32([0] * B), i32([0] * B)
    cu, reserve, state = i32([0] * (B + 1)), i32(pool.alloc(NB)), i32([0, 0])
    T_ = B * P
    slots = torch.empty(T_, dtype=torch.int64, device="cuda")
    q, out = (torch.zeros(T_, Hq, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k, v = (torch.zeros(T_, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    mask, path, n = torch.zeros(T_, 1, dtype=torch.int64, device="cuda"), torch.zeros(B, P, dtype=torch.int32, device="cuda"), i32([0] * B)
    ws = torch.empty(pkv.tree_workspace_bytes(pool, B, Hq, P), dtype=torch.uint8, device="cuda")

    def step():
        pkv.extend_tables(pool, lens, cu, tables, reserve, state, total, slots)
        pkv.kv_append(pool, k, v, slots, kc, vc)
        pkv.paged_attention_tree(pool, q, kc, vc, tables, total, cu, mask, P, scale, out, ws)
        pkv.accept_rows(pool, kc, vc, tables, total, cu, path, n, lens)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    assert lens.tolist() == [0] * B and state[0] == 0
    kept = [[torch.zeros(0, Hkv, D).bfloat16() for _ in range(2)] for _ in range(B)]
    for it in range(12):
        new = rng.integers(0, P + 1, B)
        drafts = [T.ancestors(T.tree_parents(int(p), rng)) if p else np.zeros((0, 0), bool) for p in new]
        c = T.Case([x[0].shape[0] for x in kept], new, Hq, Hkv, D, kind, seed=100 + it, scale=scale, free=False)
        c.drafts, c.see = drafts, [T.visible(int(a), int(p), 0, 0, d) for a, p, d in zip(c.C, c.P, drafts)]
        rows = [[torch.randn(int(p), Hkv, D, generator=g).bfloat16() for _ in range(2)] for p in new]
        for b in range(B):                             # the definition on contiguous copies
            if c.L[b]:
                c.pages.write(c.slots(b, np.arange(c.L[b])), [torch.cat([x, y]) for x, y in zip(kept[b], rows[b])])
        accepted = []
        for b, p in enumerate(new.tolist()):
            i = int(rng.integers(0, p)) if p else -1
            line = np.flatnonzero(drafts[b][i]) if p else np.zeros(0, int)
            accepted.append(line[:int(rng.integers(0, len(line) + 1))])
        m = c.mask() if c.T else np.zeros((0, 1), np.int64)
        cu.copy_(i32(c.cu))
        if c.T:
            q[:c.T], mask[:c.T] = c.q.cuda(), T.dev(m)
            k[:c.T], v[:c.T] = (torch.cat([r[x] for r in rows]).cuda() for x in (0, 1))
        path.fill_(-1)
        for b, a in enumerate(accepted):
            path[b, :len(a)] = i32(a)
        n.copy_(i32([len(a) for a in accepted]))
        out.fill_(float("nan"))
        graph.replay()
        c.check(out)
        kept = [[torch.cat([x, y[a]]) for x, y in zip(kept[b], rows[b])] for b, a in enumerate(accepted)]
        assert lens.tolist() == [x[0].shape[0] for x in kept]
    assert pool.get_device_error() == (pkv.OK, 0)
    bt = tables.cpu().numpy()
    for b in range(B):
        L = kept[b][0].shape[0]
        assert L > 0
        pos = np.arange(L)
        s = bt[b, pos // 16].astype(np.int64) * 16 + pos % 16
        ref = T.Pages(kind, -(-L // 16), Hkv, D)
        ref.write(pos, kept[b])
        got = T.Pages(kind, NB, Hkv, D)
        got.caches = [x.view(torch.int16 if kind == "bf16" else torch.uint8).cpu().numpy().view(w.dtype) for x, w in zip((kc, vc), got.caches)]
        for x, y in zip(ref.read(pos), got.read(s)):
            assert np.array_equal(x, y)
