"""INT4 pools on the GPU: the append and gather bit for bit against the plain implementation
(oracle/int4.py), decode within the bound of its arithmetic, at the sizes where it can go wrong."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import int4 as O
from tests import _int4 as I

pkv = pytest.importorskip("paged_kv_cache_159_gb300")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    pkv.lib()
    torch.cuda.set_device(0)


def _pool(NB, Hkv, D, layers=1, ks=0.0131, vs=0.0087, kv=None):
    p = pkv.Pool(NB, Hkv, D, pkv.KV_INT4 if kv is None else kv, ks, vs, num_layers=layers)
    p.attach_device(0)
    return p


# ------------------------------------------------------------------ append and gather
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,Hkv", [(1, 1), (3, 3), (17, 2), (16, 8), (333, 5)])
def test_append_and_gather_bit_for_bit(T, Hkv, D):
    rng = np.random.default_rng(T * 131 + Hkv)
    NB = -(-T // 16) + 4
    slots = rng.permutation(NB * 16)[:T].astype(np.int64)
    if T > 4:
        slots[2] = -1                                   # padding rows are skipped
    k, v = (torch.from_numpy(rng.standard_normal((T, Hkv, D)).astype(np.float32) * s).bfloat16() for s in (1.0, 3e-3))
    kh, vh = (rng.integers(0, 256, (NB, Hkv, O.tile_bytes(D))).astype(np.uint8) for _ in range(2))
    pool, kc, vc = _pool(NB, Hkv, D), I.dev(kh), I.dev(vh)
    assert pool.tile_bytes() == O.tile_bytes(D) and pool.layer_bytes() == kc.numel()
    pkv.kv_append(pool, k.cuda(), v.cuda(), I.dev(slots), kc, vc)
    O.append(I.bits(k), I.bits(v), slots, kh, vh, 0.0131, 0.0087)
    assert np.array_equal(kc.cpu().numpy(), kh) and np.array_equal(vc.cpu().numpy(), vh)
    ko, vo = (torch.full((T, Hkv, D), -5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pkv.kv_gather(pool, I.dev(slots), kc, vc, ko, vo)
    assert pool.get_device_error() == (pkv.OK, 0)
    for out, cache, is_key, s in ((ko, kh, True, 0.0131), (vo, vh, False, 0.0087)):
        ref = torch.full((T, Hkv, D), -5.0, dtype=torch.bfloat16)
        w = slots >= 0
        # (n - 8) times the fp32 product of the scales, in fp32, then bf16
        n, e = O.codes(cache, slots[w], is_key)
        x = n.astype(np.float32) * (e.astype(np.float32) * np.float32(s))
        ref[torch.from_numpy(w)] = torch.from_numpy(x).bfloat16()
        assert np.array_equal(I.bits(out), I.bits(ref))


@pytest.mark.parametrize("D", [64, 128])
def test_append_of_every_kind_of_value(D):
    """Groups of zeros, subnormals, one huge element, infinities and NaN, scale bytes from zero
    through subnormal to saturated."""
    special = [0x0000, 0x8000, 0x0001, 0x0080, 0x7F7F, 0xFF7F, 0x7F80, 0xFF80, 0x7FC0, 0xFFC1]
    T, Hkv = 64, 2
    rng = np.random.default_rng(D)
    x = torch.from_numpy((rng.standard_normal((T, Hkv, D)) * np.exp2(rng.integers(-20, 20, (T, Hkv, 1)))).astype(np.float32)).bfloat16()
    b = I.bits(x).copy()
    b[0] = 0
    for i, s in enumerate(special):
        b[1 + i, 0, 5::32] = s
        b[1 + i, 1, :] = s
    x = torch.from_numpy(b.view(np.int16)).view(torch.bfloat16)
    slots = rng.permutation(T).astype(np.int64)
    kh, vh = (np.zeros((T // 16, Hkv, O.tile_bytes(D)), np.uint8) for _ in range(2))
    pool, kc, vc = _pool(T // 16, Hkv, D, ks=1.0, vs=0.25), I.dev(kh), I.dev(vh)
    pkv.kv_append(pool, x.cuda(), x.cuda(), I.dev(slots), kc, vc)
    O.append(b, b, slots, kh, vh, 1.0, 0.25)
    assert np.array_equal(kc.cpu().numpy(), kh) and np.array_equal(vc.cpu().numpy(), vh)
    assert not np.isnan(O.rows(kh, slots, True, 1.0)).any()


@pytest.mark.parametrize("kv", [pkv.KV_BF16, pkv.KV_FP8E4M3, pkv.KV_INT4])
@pytest.mark.parametrize("D", [64, 128])
def test_gather_of_every_pool_type_and_layer(kv, D):
    layers, NB, Hkv, T = 3, 5, 3, 29
    rng = np.random.default_rng(kv * 7 + D)
    pool = _pool(NB, Hkv, D, layers, 0.5, 0.25, kv)
    shape = (layers, NB, Hkv, 16, D) if kv != pkv.KV_INT4 else (layers, NB, Hkv, pool.tile_bytes())
    dt = torch.bfloat16 if kv == pkv.KV_BF16 else torch.uint8
    kc, vc = (torch.zeros(shape, dtype=dt, device="cuda") for _ in range(2))
    k, v = (torch.from_numpy(rng.standard_normal((layers, T, Hkv, D)).astype(np.float32)).bfloat16().cuda() for _ in range(2))
    slots = I.dev(rng.permutation(NB * 16)[:T].astype(np.int64))
    pkv.kv_append_layers(pool, k, v, slots, kc, vc)
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    pkv.kv_gather_layers(pool, slots, kc, vc, ko, vo)
    assert pool.get_device_error() == (pkv.OK, 0)
    for src, out, cache, s in ((k, ko, kc, 0.5), (v, vo, vc, 0.25)):
        if kv == pkv.KV_BF16:
            assert torch.equal(src, out)
        elif kv == pkv.KV_FP8E4M3:
            assert torch.equal(out, ((src.float() / s).to(torch.float8_e4m3fn).float() * s).bfloat16())
        else:
            # a power-of-two pool scale leaves one rounding, of a product of 7 significant bits: none
            for l in range(layers):
                ref = O.rows(cache[l].cpu().numpy(), slots.cpu().numpy(), cache is kc, s)
                assert np.array_equal(out[l].float().cpu().double().numpy(), ref)
            step = (src.float().unflatten(-1, (-1, 32)).abs().amax(-1, keepdim=True) / 7).expand(-1, -1, -1, -1, 32).flatten(-2)
            # half a step, the scale rounded by at most 2^-4, and clamping to 7 steps
            assert bool(((src.float() - out.float()).abs() <= step * 0.5 * (1 + 2.0 ** -4) * (1 + 2.0 ** -20)).all())
    # single layers, rows repeated
    rep = slots[torch.tensor([0, 0, 5, 3])]
    ko1, vo1 = torch.empty(4, Hkv, D, dtype=torch.bfloat16, device="cuda"), torch.empty(4, Hkv, D, dtype=torch.bfloat16, device="cuda")
    pkv.kv_gather(pool, rep, kc[1], vc[1], ko1, vo1)
    assert torch.equal(ko1, ko[1][[0, 0, 5, 3]]) and torch.equal(vo1, vo[1][[0, 0, 5, 3]])


@pytest.mark.parametrize("T,Hkv,layers,D", [(4100, 3, 1, 64), (4100, 3, 1, 128), (8193, 1, 1, 128), (1400, 2, 3, 64), (1400, 2, 3, 128)])
def test_many_rows_of_every_kind_of_value(T, Hkv, layers, D):
    # enough rows for a quarter of a row a thread; padding, slots beyond the pool, special values
    rng = np.random.default_rng(T + D)
    NB = -(-T // 16) + 2
    slots = rng.permutation(NB * 16)[:T].astype(np.int64)
    slots[[1, 700, T - 1]] = -1
    slots[[2, 31, T - 2]] = [NB * 16, 1 << 40, NB * 16 + 5]
    x = (rng.standard_normal((2, layers, T, Hkv, D)) * np.exp2(rng.integers(-16, 16, (2, layers, T, Hkv, 1)))).astype(np.float32)
    x = torch.from_numpy(x).bfloat16()
    b = I.bits(x).copy()
    at = rng.random(b.shape) < 2e-4
    b[at] = rng.choice(np.array([0x0000, 0x0001, 0x7F7F, 0x7F80, 0xFF80, 0x7FC0], np.uint16), int(at.sum())).view(b.dtype)
    k, v = torch.from_numpy(b.view(np.int16)).view(torch.bfloat16)
    kh, vh = (rng.integers(0, 256, (layers, NB, Hkv, O.tile_bytes(D))).astype(np.uint8) for _ in range(2))
    pool, kc, vc, sl = _pool(NB, Hkv, D, layers, 0.5, 0.25), I.dev(kh), I.dev(vh), I.dev(slots)
    pkv.kv_append_layers(pool, k.cuda(), v.cuda(), sl, kc, vc)
    assert pool.get_device_error() == (pkv.ERR_DEVICE, pkv.DEVERR_SLOT)
    ok = (slots >= 0) & (slots < NB * 16)
    for l in range(layers):
        O.append(b[0, l], b[1, l], np.where(ok, slots, -1), kh[l], vh[l], 0.5, 0.25)
    assert np.array_equal(kc.cpu().numpy(), kh) and np.array_equal(vc.cpu().numpy(), vh)
    ko, vo = (torch.full((layers, T, Hkv, D), -5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pkv.kv_gather_layers(pool, sl, kc, vc, ko, vo)
    assert pool.get_device_error() == (pkv.ERR_DEVICE, pkv.DEVERR_SLOT)
    for out, cache, is_key, s in ((ko, kh, True, 0.5), (vo, vh, False, 0.25)):
        got = out.float().cpu().double().numpy()
        for l in range(layers):                      # (a power-of-two pool scale: no rounding)
            assert np.array_equal(got[l][ok], O.rows(cache[l], slots[ok], is_key, s))
        assert (got[:, ~ok] == -5).all()


def test_slots_beyond_the_pool_are_flagged_and_skipped():
    pool = _pool(2, 1, 64)
    kc, vc = (torch.zeros(2, 1, 544, dtype=torch.uint8, device="cuda") for _ in range(2))
    x = torch.ones(3, 1, 64, dtype=torch.bfloat16, device="cuda")
    slots = torch.tensor([32, 5, -1], device="cuda")
    pkv.kv_append(pool, x, x, slots, kc, vc)
    assert pool.get_device_error() == (pkv.ERR_DEVICE, pkv.DEVERR_SLOT)
    ko, vo = torch.full_like(x, 9.0), torch.full_like(x, 9.0)
    pkv.kv_gather(pool, slots, kc, vc, ko, vo)
    assert pool.get_device_error() == (pkv.ERR_DEVICE, pkv.DEVERR_SLOT)
    assert (ko[[0, 2]] == 9).all() and (vo[[0, 2]] == 9).all() and (ko[1] != 9).all()
    assert int(kc[1].count_nonzero()) == 0


# ------------------------------------------------------------------ decode
SHAPES = [  # lens, Hq, Hkv, D
    ([1], 1, 1, 128),
    ([1, 2, 15, 16, 17], 4, 2, 64),
    ([31, 32, 33, 47, 48, 49, 1], 8, 2, 128),
    ([129, 5, 255], 7, 1, 128),
    ([100, 16, 700], 24, 3, 64),
    ([513, 31], 9, 1, 128),
    ([77, 1300], 32, 2, 64),
    ([64, 1000, 3], 16, 1, 128),
    ([300] * 12, 12, 3, 128),
    ([2500], 32, 8, 128),
    ([70, 33, 1], 24, 12, 64),             # more KV heads than a team: 6 of 12
    ([40, 130], 22, 11, 128),              # 11 teams of one
    ([90, 17], 32, 16, 64),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s[1:])) + "-%d" % len(s[0]))
def test_decode_shapes_and_grids(shape):
    c = I.Case(*shape, seed=len(shape[0]) + shape[1])
    outs = [c.decode(o) for o in (None, {"grid_ctas": 1}, {"grid_ctas": 5}, {"grid_ctas": 37}, {"grid_ctas": 200})]
    for out in outs:
        c.check(out)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("q_gain,v_gain,ks,vs", [(1e-6, 1.0, 0.0131, 0.0087), (3e4, 1.0, 0.0131, 0.0087), (8.0, 1.0, 1.0, 1.0),
                                                 (1.0, 1e-5, 0.0131, 4e-9), (1.0, 1e4, 0.5, 40.0)])
def test_decode_over_magnitudes(q_gain, v_gain, ks, vs, D):
    c = I.Case([200, 9, 64], 8, 2, D, seed=3, q_gain=q_gain, v_gain=v_gain, k_scale=ks, v_scale=vs)
    c.check(c.decode())


@pytest.mark.parametrize("scale", [0.0, -0.25, 2.0])
def test_any_finite_scale(scale):
    c = I.Case([100, 7, 33], 8, 2, 128, seed=8)
    c.scale = scale
    c.check(c.decode())


def test_one_position_returns_its_value():
    c = I.Case([1, 1], 4, 2, 128, v_scale=0.25)
    ref = O.rows(c.vh, c.slots, False, 0.25)
    got = c.decode().float().cpu().double().numpy()
    assert np.array_equal(got, np.repeat(ref, 2, axis=1))   # 7 significant bits: exact in bf16


def test_physical_placement_and_repeats_do_not_change_a_bit():
    lens = [700, 3, 1025, 64]
    outs = []
    for order in (1, 2, 3):
        c = I.Case(lens, 16, 4, 128, seed=5, order_seed=order)
        outs += [c.decode({"grid_ctas": 61}), c.decode({"grid_ctas": 61})]
    assert all(torch.equal(outs[0], o) for o in outs[1:])


@pytest.mark.parametrize("B,Hq,Hkv,D", [(700, 4, 2, 64), (4096, 1, 1, 128)])
def test_large_batches_of_short_sequences(B, Hq, Hkv, D):
    lens = np.random.default_rng(B).integers(1, 40, B)
    lens[5] = 300
    c = I.Case(lens.tolist(), Hq, Hkv, D, seed=B)
    c.check(c.decode())


def test_offsets_past_32_bits():
    """The same rows at the far end of a pool of 4.5 GB a cache: same codes, rows and outputs."""
    c = I.Case([40, 1000], 16, 8, 128, seed=21)
    NB, shift = 520_000, 520_000 - c.NB
    pool = pkv.Pool(NB, 8, 128, pkv.KV_INT4, c.k_scale, c.v_scale)
    pool.attach_device(0)
    kc, vc = (torch.zeros(NB, 8, 1088, dtype=torch.uint8, device="cuda") for _ in range(2))
    slots = I.dev(c.slots + 16 * shift)
    pkv.kv_append(pool, c.k.cuda(), c.v.cuda(), slots, kc, vc)
    ko, vo, kr, vr = (torch.zeros_like(c.k, device="cuda") for _ in range(4))
    pkv.kv_gather(pool, slots, kc, vc, ko, vo)
    pkv.kv_gather(c.pool, I.dev(c.slots), c.kc, c.vc, kr, vr)
    assert torch.equal(ko, kr) and torch.equal(vo, vr) and int(kr.count_nonzero()) > 0
    bt = torch.where(c.bt >= 0, c.bt + shift, c.bt)
    out = torch.zeros_like(c.q, device="cuda")
    pkv.paged_attention_decode(pool, c.q.cuda(), kc, vc, bt, c.sl, c.scale, out, c.workspace())
    assert pool.get_device_error() == (pkv.OK, 0) and torch.equal(out, c.decode())
    m = torch.arange(NB - 1, NB - 4, -1, dtype=torch.int32, device="cuda")
    want = [x[m.long()] for x in (kc, vc)]
    pkv.move_blocks(pool, kc, vc, m, torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda"), bt)
    assert torch.equal(kc[:3], want[0]) and torch.equal(vc[:3], want[1])
    pkv.paged_attention_decode(pool, c.q.cuda(), kc, vc, bt, c.sl, c.scale, out, c.workspace())
    assert torch.equal(out, c.decode())


def test_long_sequence_over_many_ctas():
    c = I.Case([20000], 8, 1, 128, seed=9)
    c.check(c.decode())


@pytest.mark.parametrize("shape", [([1, 16, 17, 33, 400], 8, 2, 64), ([2, 15, 48, 1111, 500], 28, 4, 128)], ids=["d64", "d128"])
def test_step_equals_append_then_decode(shape):
    c = I.Case(*shape, seed=11)
    new = [torch.randn(len(c.lens), c.Hkv, c.D, generator=torch.Generator().manual_seed(s)).bfloat16() for s in (1, 2)]
    slots = np.array([c.row_slots(b, L - 1) for b, L in enumerate(c.lens)], np.int64)
    O.append(I.bits(new[0]), I.bits(new[1]), slots, c.kh, c.vh, c.k_scale, c.v_scale)
    out, ws = torch.empty_like(c.q, device="cuda"), c.workspace()
    ka, va = c.kc.clone(), c.vc.clone()
    pkv.decode_step(c.pool, c.q.cuda(), new[0].cuda(), new[1].cuda(), c.kc, c.vc, c.bt, c.sl, c.scale, out, ws)
    assert c.pool.get_device_error() == (pkv.OK, 0)
    assert np.array_equal(c.kc.cpu().numpy(), c.kh) and np.array_equal(c.vc.cpu().numpy(), c.vh)
    c.check(out)
    pkv.kv_append(c.pool, new[0].cuda(), new[1].cuda(), I.dev(slots), ka, va)
    assert torch.equal(ka, c.kc) and torch.equal(va, c.vc) and torch.equal(out, c.decode(ws=ws))
    # the same step from host memory, and without a workspace
    host = dict(q=c.q.pin_memory(), k_new=new[0].pin_memory(), v_new=new[1].pin_memory(), block_tables=torch.from_numpy(c.tables).pin_memory(),
                seq_lens=torch.from_numpy(c.lens).pin_memory(), out=torch.empty_like(c.q).pin_memory())
    d = {k: torch.empty_like(t, device="cuda") for k, t in host.items()}
    pkv.decode_step_host(c.pool, host, d, c.kc, c.vc, c.scale, ws)
    torch.cuda.synchronize()
    assert torch.equal(host["out"], out.cpu())
    out2 = torch.empty_like(out)
    pkv.paged_attention_decode_noalloc(c.pool, c.q.cuda(), c.kc, c.vc, c.bt, c.sl, c.scale, out2)
    assert c.pool.get_device_error() == (pkv.OK, 0)
    c.check(out2)                                     # (a smaller grid where the scratch asks for it)


@pytest.mark.parametrize("append", [False, True])
def test_every_layer_in_one_launch(append):
    c = [I.Case([33, 500, 16, 1], 8, 2, 128, seed=s, order_seed=4) for s in range(3)]
    pool = c[0].new_pool(3)
    q, kc, vc = (torch.stack([getattr(x, n).cuda() for x in c]) for n in ("q", "kc", "vc"))
    kn, vn = (torch.randn(3, 4, 2, 128, generator=torch.Generator().manual_seed(s)).bfloat16() for s in (1, 2))
    out = torch.empty_like(q)
    n = pkv.decode_workspace_bytes(pool, 4, 8, c[0].MB)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    new = (kn.cuda(), vn.cuda()) if append else (None, None)
    pkv.decode_step_layers(pool, q, *new, kc, vc, c[0].bt, c[0].sl, c[0].scale, out, ws)
    assert pool.get_device_error() == (pkv.OK, 0)
    for l, x in enumerate(c):
        if append:
            slots = np.array([x.row_slots(b, L - 1) for b, L in enumerate(x.lens)], np.int64)
            O.append(I.bits(kn[l]), I.bits(vn[l]), slots, x.kh, x.vh, x.k_scale, x.v_scale)
        assert np.array_equal(kc[l].cpu().numpy(), x.kh) and np.array_equal(vc[l].cpu().numpy(), x.vh)
        x.check(out[l])


def test_bad_lengths_and_tables_are_flagged():
    c = I.Case([40, 20, 30], 4, 2, 64)
    ref = c.decode()
    c.sl[1] = 0
    out, ws = torch.full_like(ref, float("nan")), c.workspace()
    args = (c.pool, c.q.cuda(), c.kc, c.vc, c.bt, c.sl, c.scale, out, ws)
    pkv.paged_attention_decode(*args)
    assert c.pool.get_device_error() == (pkv.ERR_DEVICE, pkv.DEVERR_SEQ_LEN)
    assert int(out[1].count_nonzero()) == 0 and torch.equal(out[[0, 2]], ref[[0, 2]])
    c.sl[1] = 20
    c.bt[2, 0] = c.NB
    ws.zero_()
    pkv.paged_attention_decode(*args)
    assert c.pool.get_device_error() == (pkv.ERR_DEVICE, pkv.DEVERR_BLOCK_ID)
    assert torch.equal(out[:2], ref[:2])


def test_decode_captured_replayed_and_on_another_stream():
    c = I.Case([65, 1000, 7], 16, 4, 128, seed=2)
    ref = c.decode()
    out, ws, q = torch.zeros_like(ref), c.workspace(), c.q.cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        ko, vo = torch.zeros_like(c.k, device="cuda"), torch.zeros_like(c.v, device="cuda")
        slots = I.dev(c.slots)
        pkv.kv_gather(c.pool, slots, c.kc, c.vc, ko, vo, stream=side)
        pkv.paged_attention_decode(c.pool, q, c.kc, c.vc, c.bt, c.sl, c.scale, out, ws, stream=side)
    side.synchronize()
    assert torch.equal(out, ref)
    with torch.cuda.graph(g):
        pkv.paged_attention_decode(c.pool, q, c.kc, c.vc, c.bt, c.sl, c.scale, out, ws)
    for n in ([65, 1000, 7], [1, 33, 2]):
        out.zero_()
        c.sl.copy_(torch.tensor(n, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        c.lens = np.array(n, np.int32)
        c.check(out)


def test_decodes_captured_behind_copies_and_joined_streams():
    # the decode's launches may start early: their inputs come from a copy, from another stream's
    # append and from a decode just before, all within one capture, replayed back to back
    c = I.Case([65, 1000, 7, 300], 16, 4, 128, seed=8)
    want = c.decode()
    c.sl.fill_(1)
    q, q0, lens = c.q.cuda(), torch.zeros_like(c.q, device="cuda"), torch.from_numpy(c.lens).cuda()
    outs, ws, side = [torch.zeros_like(want) for _ in range(3)], [c.workspace(), c.workspace()], torch.cuda.Stream()
    kc, vc = torch.zeros_like(c.kc), torch.zeros_like(c.vc)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        main = torch.cuda.current_stream()
        q0.copy_(q)
        side.wait_stream(main)
        with torch.cuda.stream(side):
            kc.copy_(c.kc)
            pkv.paged_attention_decode(c.pool, q0, c.kc, c.vc, c.bt, lens, c.scale, outs[2], ws[1], stream=side)
            vc.copy_(c.vc)
        c.sl.copy_(lens)
        main.wait_stream(side)
        pkv.paged_attention_decode(c.pool, q0, kc, vc, c.bt, c.sl, c.scale, outs[0], ws[0])
        pkv.paged_attention_decode(c.pool, outs[0], kc, vc, c.bt, c.sl, c.scale, outs[1], ws[0])
        q0.zero_()
        c.sl.fill_(1)
        kc.zero_()
    twice = torch.zeros_like(want)
    pkv.paged_attention_decode(c.pool, want, c.kc, c.vc, c.bt, lens, c.scale, twice, c.workspace())
    for _ in range(5):
        for o in outs:
            o.zero_()
        g.replay()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want) and torch.equal(outs[2], want) and torch.equal(outs[1], twice)
    assert c.pool.get_device_error() == (pkv.OK, 0)


def test_copy_blocks_moves_whole_tiles():
    layers, NB, Hkv, D = 2, 6, 3, 64
    pool = _pool(NB, Hkv, D, layers)
    kc, vc = (torch.randint(0, 256, (layers, NB, Hkv, 544), dtype=torch.uint8, device="cuda") for _ in range(2))
    want = [x.clone() for x in (kc, vc)]
    for x in want:
        x[:, [4, 0]] = x[:, [1, 5]]
    pkv.copy_blocks(pool, kc, vc, torch.tensor([1, 5], dtype=torch.int32, device="cuda"), torch.tensor([4, 0], dtype=torch.int32, device="cuda"))
    assert torch.equal(kc, want[0]) and torch.equal(vc, want[1])


def test_refusals():
    c = I.Case([40, 20], 8, 2, 64)
    q, out = c.q.cuda(), torch.empty_like(c.q, device="cuda")
    for opts in ({"variant": 3}, {"variant": 1}, {"heads_per_copy": 2}, {"shared_prefix_blocks": 2}, {"stages": 3}, {"warps_per_cta": 4}, {"unit_cost": 3},
                 {"grid_ctas": -1}):
        assert pkv.decode_workspace_bytes(c.pool, 2, 8, c.MB, opts) == 0
        with pytest.raises(pkv.PkvError) as e:
            pkv.paged_attention_decode(c.pool, q, c.kc, c.vc, c.bt, c.sl, c.scale, out, c.workspace(), opts)
        assert e.value.status == pkv.ERR_INVALID
    L, P, s = pkv.lib(), ctypes.c_void_p, ctypes.c_void_p(0)
    sl = I.dev(c.slots)
    ok = [c.pool.handle, P(sl.data_ptr()), 4, P(c.kc.data_ptr()), P(c.vc.data_ptr()), P(q.data_ptr()), P(out.data_ptr()), s]
    for i, bad in ((0, None), (1, None), (1, P(sl.data_ptr() + 4)), (2, -1), (3, None), (3, P(c.kc.data_ptr() + 8)), (4, None), (5, None),
                   (5, P(q.data_ptr() + 2)), (6, None), (6, P(out.data_ptr() + 8))):
        args = list(ok)
        args[i] = bad
        assert L.pkv_kv_gather(*args) == pkv.ERR_INVALID, (i, bad)
    ok[2] = 0
    assert L.pkv_kv_gather(*ok) == pkv.OK
    fresh = pkv.Pool(4, 2, 64, pkv.KV_INT4)
    assert L.pkv_kv_gather(fresh.handle, *ok[1:]) == pkv.ERR_INVALID                 # not attached
