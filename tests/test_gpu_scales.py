"""Attention at every finite scale -- positive, zero, negative, too small to tell apart -- over every
pool type: prefill and decode against the formula in 64 bits on the rows that the pool gives back."""
import numpy as np
import pytest
import torch

pkv = pytest.importorskip("paged_kv_cache_159_gb300")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    pkv.lib()
    torch.cuda.set_device(0)


P, C = [40, 1, 130, 64], [37, 0, 100, 0]              # a chunk's rows, and the positions before them
S = 2.0 ** -6                                         # a power of two: the rows come back exactly


def _run(kv, D, scale, Hq=8, Hkv=2):
    """(lengths, first rows, q, k, v as the pool gives them back, prefill output, decode output of the last rows)"""
    lens = np.array([p + c for p, c in zip(P, C)], np.int32)
    cu = np.concatenate([[0], np.cumsum(P)]).astype(np.int32)
    g = torch.Generator(device="cuda").manual_seed(D + kv)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    MB = -(-int(lens.max()) // 16)
    ps = 1.0 if kv == pkv.KV_BF16 else S
    pool = pkv.Pool(int(sum(-(-lens // 16))) + 2, Hkv, D, kv, ps, ps)
    pool.attach_device(0)
    tables = pool.build_block_tables(lens, MB)
    NB = pool.desc.num_blocks
    shape = (NB, Hkv, pool.tile_bytes()) if kv == pkv.KV_INT4 else (NB, Hkv, 16, D)
    kc, vc = (torch.zeros(shape, dtype=torch.bfloat16 if kv == pkv.KV_BF16 else torch.uint8, device="cuda") for _ in range(2))
    slots = torch.from_numpy(pkv.slot_mapping_all(tables, lens)).cuda()
    T = int(lens.sum())
    pkv.kv_append(pool, rnd(T, Hkv, D), rnd(T, Hkv, D), slots, kc, vc)
    k, v = (torch.empty(T, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pkv.kv_gather(pool, slots, kc, vc, k, v)
    q = rnd(int(cu[-1]), Hq, D)
    bt, sl = torch.from_numpy(tables).cuda(), torch.from_numpy(lens).cuda()
    plan, grid = pkv.prefill_plan(pool, cu, lens, Hq, MB)
    n = pkv.prefill_workspace_bytes(pool, cu, lens, MB)
    out = torch.full_like(q, float("nan"))
    pkv.paged_prefill(pool, q, kc, vc, bt, scale, torch.from_numpy(plan).cuda(), grid, out,
                      workspace=torch.empty(n, dtype=torch.uint8, device="cuda") if n else None)
    last = torch.from_numpy(cu[1:].astype(np.int64) - 1).cuda()
    dout = torch.full((len(P), Hq, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(pkv.decode_workspace_bytes(pool, len(P), Hq, MB), dtype=torch.uint8, device="cuda")
    pkv.paged_attention_decode(pool, q[last], kc, vc, bt, sl, scale, dout, ws)
    assert pool.get_device_error() == (pkv.OK, 0)
    return lens, cu, q, k, v, out, dout


@pytest.mark.parametrize("scale", [0.125, 0.0, -0.0, -0.125, 1e-40, -1e-40])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kv", [pkv.KV_BF16, pkv.KV_FP8E4M3, pkv.KV_INT4])
def test_prefill_and_decode(kv, D, scale):
    Hq, Hkv = 8, 2
    lens, cu, q, k, v, out, dout = _run(kv, D, scale)
    at = 0
    for b, L in enumerate(lens.tolist()):
        kb, vb = (x[at:at + L].double().repeat_interleave(Hq // Hkv, 1) for x in (k, v))
        at += L
        s = torch.einsum("rhd,thd->hrt", q[cu[b]:cu[b + 1]].double(), kb) * float(np.float32(scale))
        late = torch.arange(L, device="cuda")[None, :] > torch.arange(L - P[b], L, device="cuda")[:, None]
        w = torch.softmax(s.masked_fill(late, float("-inf")), -1)
        ref, mag = (torch.einsum("hrt,thd->rhd", w, x) for x in (vb, vb.abs()))
        # bf16 roundings of the output and of p (2^-8 each), 2^-10 for scores and sums: scores stay
        # below 2^4, off by 2^-22 of at most 128 terms each, and by 2^-17 of |k| a term where q is taken to f16
        tol = 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -10) * mag
        got = out[cu[b]:cu[b + 1]].double()
        assert bool(((got - ref).abs() <= tol).all()), ("prefill", b, ((got - ref).abs() / tol).max())
        assert bool(((dout[b].double() - ref[-1]).abs() <= tol[-1]).all()), ("decode", b)


@pytest.mark.parametrize("scale", [1e30, -1e30])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kv", [pkv.KV_BF16, pkv.KV_FP8E4M3, pkv.KV_INT4])
def test_scales_at_the_end_of_the_range(kv, D, scale):
    # one position takes all the weight: the largest score, where it stands out by 2^-8 of the largest
    # magnitude (scores are off by less than 2^-9 of it); everywhere the outputs are visible values' means
    lens, cu, q, k, v, out, dout = _run(kv, D, scale / (1.0 if kv == pkv.KV_BF16 else S))
    at = seen = 0
    for b, L in enumerate(lens.tolist()):
        kb, vb = (x[at:at + L].double().repeat_interleave(4, 1) for x in (k, v))
        at += L
        s = torch.einsum("rhd,thd->hrt", q[cu[b]:cu[b + 1]].double(), kb) * (1.0 if scale > 0 else -1.0)
        big = s.abs().amax(-1)
        late = torch.arange(L, device="cuda")[None, :] > torch.arange(L - P[b], L, device="cuda")[:, None]
        s = s.masked_fill(late, float("-inf"))
        top = s.topk(min(2, L), -1)
        clear = (top.values[..., 0] - top.values[..., 1] > 2.0 ** -8 * big) if L > 1 else torch.ones_like(big, dtype=torch.bool)
        ref = vb.permute(1, 0, 2).gather(1, top.indices[..., :1].expand(-1, -1, D)).permute(1, 0, 2)         # [rows, heads, D]
        got = out[cu[b]:cu[b + 1]].double()
        eps = vb.abs().amax() * 2.0 ** -7
        for o, r, c in ((got, ref, clear.T), (dout[b:b + 1].double(), ref[-1:], clear.T[-1:])):
            assert bool(o.isfinite().all())
            assert bool((o >= vb.amin(0) - eps).all()) and bool((o <= vb.amax(0) + eps).all())
            # (f16 roundings of p and p scale, the output's)
            assert bool(((o - r).abs() <= r.abs() * (2.0 ** -8 + 2.0 ** -9) + 2.0 ** -20)[c].all())
            seen += int(c.sum())
    assert seen > 0
