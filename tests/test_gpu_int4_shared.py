"""INT4 pools where sequences share blocks, prefill over more blocks than the expansion has CTAs, and
the decode without a workspace at the groups whose partial states need a smaller grid."""
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


def _shared(P, C, Hq, Hkv, D, own=1):
    """Sequences of C[b] + P[b] positions, the last P[b] of them rows, that share all but their last
    `own` blocks with the longest."""
    lens = [p + c for p, c in zip(P, C)]
    nb = [-(-L // 16) for L in lens]
    first = int(np.argmax(lens))
    private = [0 if b == first else min(own, n) for b, n in enumerate(nb)]
    # one sequence over every block, then the tables cut out of it
    c = I.Case([16 * (nb[first] + sum(private))], Hq, Hkv, D, seed=Hq)
    pool = c.tables[0]
    tables, at = np.full((len(P), nb[first]), -1, np.int32), nb[first]
    for b, n in enumerate(nb):
        tables[b, :n] = pool[:n]
        tables[b, n - private[b]:n] = pool[at:at + private[b]]
        at += private[b]
    c.lens, c.tables, c.MB = np.array(lens, np.int32), tables, nb[first]
    c.bt, c.sl = I.dev(tables), I.dev(c.lens)
    c.cu = np.concatenate([[0], np.cumsum(P)]).astype(np.int32)
    g = torch.Generator().manual_seed(3)
    c.rows = torch.randn(int(c.cu[-1]), Hq, D, generator=g).bfloat16()
    c.q = torch.randn(len(P), Hq, D, generator=g).bfloat16()
    return c


def _check_prefill(c):
    plan, grid = pkv.prefill_plan(c.pool, c.cu, c.lens, c.Hq, c.MB)
    n = pkv.prefill_workspace_bytes(c.pool, c.cu, c.lens, c.MB)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")            # bf16 NaN throughout
    out = torch.full(c.rows.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    pkv.paged_prefill(c.pool, c.rows.cuda(), c.kc, c.vc, c.bt, c.scale, torch.from_numpy(plan).cuda(), grid, out, workspace=ws)
    assert c.pool.get_device_error() == (pkv.OK, 0)
    ref, mag = O.prefill(I.bits(c.rows), c.kh, c.vh, c.tables, c.lens, c.cu, c.scale, c.k_scale, c.v_scale)
    got = out.float().cpu().double().numpy()
    # bf16 roundings of the output and of p, 2^-10 for scores (below 2^5, off by 2^-22 of at most 128
    # terms each) and sums
    assert (np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -10) * mag).all()
    return got


@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 64), (8, 2, 128)])
def test_sequences_that_share_blocks(Hq, Hkv, D):
    c = _shared([40, 5, 0, 17, 1], [300, 300, 200, 64, 0], Hq, Hkv, D)
    _check_prefill(c)
    B.check(c.decode(), *B.bound(c, 1))


@pytest.mark.parametrize("D", [64, 128])
def test_more_expanded_blocks_than_ctas(D):
    # the expansion walks its blocks with 32 CTAs an SM: every sequence's last ones lie beyond them
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    C = 16 * (32 * sms // 7)
    P = [2, 1, 0, 3, 1, 1, 2, 1, 1, 2]
    c = _shared(P, [C, C - 5, C, C - 16, C - 1, 33, C, C - 40, C - 3, C], 2, 1, D, own=40)
    assert sum(-(-int(L) // 16) for L, p in zip(c.lens, P) if p) > 32 * sms
    _check_prefill(c)


@pytest.mark.parametrize("Hq,Hkv,D", [(7, 1, 128), (16, 2, 128), (14, 1, 128), (32, 2, 128), (16, 1, 64), (48, 3, 64)])
def test_decode_without_a_workspace(Hq, Hkv, D):
    c = I.Case([1500, 3, 700, 33], Hq, Hkv, D, seed=Hq)
    out = torch.full(c.q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    for _ in range(2):
        pkv.paged_attention_decode_noalloc(c.pool, c.q.cuda(), c.kc, c.vc, c.bt, c.sl, c.scale, out)
        assert c.pool.get_device_error() == (pkv.OK, 0)
        B.check(out, *B.bound(c, 16))
