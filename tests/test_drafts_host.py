"""Drafted tokens and windows without a GPU: refusals, and the definition that the GPU tests check against."""
import itertools

import numpy as np
import pytest
import torch

import paged_kv_cache_159_gb300 as pkv
from tests import _drafts as T


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int4"])
def test_a_pool_without_a_device_is_refused(kind):
    L = pkv.lib()
    p = pkv.Pool(8, 2, 64, T.KINDS[kind], 1.0, 1.0)
    # (addresses that nothing follows: an unattached pool is refused first)
    a = 4096
    assert L.pkv_extend_tables(p.handle, a, a, 1, 4, 1, a, a, 1, a, a, a, a, None) == pkv.ERR_INVALID
    assert L.pkv_accept_rows(p.handle, a, a, a, a, a, a, a, 1, 4, 1, a, None) == pkv.ERR_INVALID
    assert L.pkv_paged_attention_tree(p.handle, a, a, a, a, a, a, a, 1, 8, 4, 1, 1, 0.1, 0, 0, a, a, 1 << 20, None) == pkv.ERR_INVALID
    assert L.pkv_paged_attention_tree(p.handle, a, a, a, a, a, None, a, 1, 8, 4, 1, 1, 0.1, 0, 0, a, a, 1 << 20, None) == pkv.ERR_INVALID
    assert L.pkv_paged_attention_window(p.handle, a, a, a, a, a, 1, 8, 4, 0.1, 4, 1, a, a, 1 << 20, None) == pkv.ERR_INVALID
    for args in ((None, a, a, 1, 4, 1, a, a, 1, a, a, a, a, None),):
        assert L.pkv_extend_tables(*args) == pkv.ERR_INVALID
    assert L.pkv_tree_workspace_bytes(None, 1, 8, 1) == 0


def test_host_tensors_are_refused():
    p = pkv.Pool(8, 2, 64)
    i = lambda *s: torch.zeros(s, dtype=torch.int32)                     # noqa: E731
    q = torch.zeros(3, 8, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        pkv.paged_attention_tree(p, q, q, q, i(1, 4), i(1), i(2), None, 3, 0.1, q, i(64))
    with pytest.raises(ValueError):
        pkv.paged_attention_window(p, q, q, q, i(3, 4), i(3), 0.1, 4, 1, q, i(64))
    with pytest.raises(ValueError):
        pkv.paged_attention_window(p, q.view(3, 4, 128), q, q, i(3, 4), i(3), 0.1, 4, 1, q, i(64))
    with pytest.raises(ValueError):
        pkv.extend_tables(p, i(1), i(2), i(1, 4), i(4), i(2), i(1), torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError):
        pkv.accept_rows(p, q, q, i(1, 4), i(1), i(2), i(1, 3), i(1), i(1))


class OnDevice:
    """What the binding asks of a CUDA tensor, of a host one: the refusals below come before any address is used."""
    is_cuda = True

    def __init__(self, t):
        self.t, self.dtype, self.shape, self.nbytes = t, t.dtype, t.shape, t.nbytes

    def __getattr__(self, name):
        return getattr(self.t, name)


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def halves(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


CALLS = {
    "paged_attention_tree": (dict(q=halves(3, 8, 64), key_cache=halves(8, 2, 16, 64), value_cache=halves(8, 2, 16, 64), block_tables=i32(1, 4),
                                  seq_lens=i32(1), cu_q=i32(2), tree_mask=torch.zeros(3, 1, dtype=torch.int64), max_q=3, scale=0.1,
                                  out=halves(3, 8, 64), workspace=i32(64)), ["q", "block_tables", "seq_lens", "cu_q", "tree_mask", "out"]),
    "paged_attention_window": (dict(q=halves(3, 8, 64), key_cache=halves(8, 2, 16, 64), value_cache=halves(8, 2, 16, 64), block_tables=i32(3, 4),
                                    seq_lens=i32(3), scale=0.1, window=4, sinks=1, out=halves(3, 8, 64), workspace=i32(64)),
                               ["q", "block_tables", "seq_lens", "out"]),
    "extend_tables": (dict(seq_lens=i32(1), cu_q=i32(2), block_tables=i32(1, 4), reserve=i32(4), state=i32(2), new_lens=i32(1),
                           slots=torch.zeros(3, dtype=torch.int64), positions=i32(3)),
                      ["seq_lens", "cu_q", "block_tables", "reserve", "state", "new_lens", "slots", "positions"]),
    "accept_rows": (dict(key_cache=halves(8, 2, 16, 64), value_cache=halves(8, 2, 16, 64), block_tables=i32(1, 4), seq_lens=i32(1), cu_q=i32(2),
                         path=i32(1, 3), num_accepted=i32(1), lens_out=i32(1)),
                    ["block_tables", "seq_lens", "cu_q", "path", "num_accepted", "lens_out"]),
}


@pytest.mark.parametrize("call,name", [(c, n) for c, (_, names) in CALLS.items() for n in names])
def test_a_tensor_of_another_type_is_refused(call, name):
    """A float16 q has the size of a bfloat16 one and would be read as it: types are those documented."""
    args = dict(CALLS[call][0])
    other = {2: torch.float16, 4: torch.float32, 8: torch.float64}[args[name].element_size()]
    args[name] = args[name].to(other)
    args = {k: OnDevice(x) if torch.is_tensor(x) else x for k, x in args.items()}
    with pytest.raises(ValueError, match="%s must be of type" % name):
        getattr(pkv, call)(pkv.Pool(8, 2, 64), **args)


def test_windowed_plan_refusals():
    p = pkv.Pool(8, 2, 64)
    for kw in (dict(window=-1), dict(window=8, sinks=-1)):
        with pytest.raises(pkv.PkvError) as e:
            pkv.prefill_plan(p, [0, 3], [40], 8, 4, **kw)
        assert e.value.status == pkv.ERR_INVALID


def test_ancestors_are_those_on_the_way_up():
    """Every tree of up to 4 tokens, against a walk from the token to the root."""
    for n in range(1, 5):
        for par in itertools.product(*[range(-1, i) for i in range(n)]):
            see = T.ancestors(list(par))
            for i in range(n):
                up, x = set(), i
                while x >= 0:
                    up.add(x)
                    x = par[x]
                assert set(np.flatnonzero(see[i])) == up


@pytest.mark.parametrize("C,window,sinks", [(0, 0, 0), (5, 0, 0), (9, 4, 0), (9, 4, 2), (9, 1, 0), (9, 1, 9), (9, 100, 1)])
def test_a_chain_of_drafts_is_the_chain(C, window, sinks):
    """A tree without branches sees what a chain does: each row's window ends at its own place.  (Windows that
    reach all drafts; a tree's drafts do not leave it.)"""
    n = 4
    chain = T.visible(C, n, window, sinks)
    tree = T.visible(C, n, window, sinks, T.ancestors([-1, 0, 1, 2]))
    assert np.array_equal(chain[:, :C], tree[:, :C])
    if window == 0 or window >= n:
        assert np.array_equal(chain, tree)
    for i in range(n):
        p = C + i
        want = [j <= p and (window == 0 or p - j < window or j < sinks) for j in range(C + n)]
        assert chain[i].tolist() == want


def test_siblings_do_not_see_each_other():
    see = T.visible(6, 3, 0, 0, T.ancestors([-1, 0, 0]))
    assert see[:, :6].all()
    assert see[:, 6:].tolist() == [[True, False, False], [True, True, False], [True, False, True]]
    near = T.visible(6, 3, 3, 1, T.ancestors([-1, 0, 0]))               # both children stand at place 7
    assert near[1].tolist() == [True] + [False] * 4 + [True, True, True, False]
    assert near[2].tolist() == [True] + [False] * 4 + [True, True, False, True]
