"""Host-side refusals of the calls over trees of drafted tokens, pages and the
layer norm: every case is rejected before anything is launched."""
import ctypes

import pytest

from linear_attention_chunk_gb300 import binding
from linear_attention_chunk_gb300.build import build

FAKE, ODD = 0x10000, 0x10008   # never dereferenced
OK, BAD, NOT, WS = binding.GLA_OK, binding.GLA_ERR_INVALID_ARG, binding.GLA_ERR_UNSUPPORTED, binding.GLA_ERR_WORKSPACE


@pytest.fixture(scope="module")
def L():
    build()
    return binding.lib()


def fwd(L, q=FAKE, lq=192, k=FAKE, lk=192, v=FAKE, lv=384, log=FAKE, cu=FAKE, par=FAKE, slots=FAKE, pool=FAKE, ns=4,
        nseq=2, T=8, H=2, dk=96, dv=192, dt=0, o=2 * FAKE, name="gla_tree_fwd"):
    return getattr(L, name)(q, lq, k, lk, v, lv, log, 0.1, cu, par, slots, pool, ns, nseq, T, H, dk, dv, dt, o, None)


@pytest.mark.parametrize("name", ["gla_tree_fwd", "gla_tree_fwd_gated"])
def test_tree_forward(L, name):
    def st(**kw):
        return fwd(L, name=name, **kw)

    for null in ("q", "k", "v", "log", "cu", "par", "pool", "o"):
        assert st(**{null: None}) == BAD, null
    for odd in ("q", "k", "v", "pool", "o"):
        assert st(**{odd: ODD}) == BAD, odd
    assert st(slots=None, ns=1) == BAD and st(ns=-1) == BAD and st(nseq=-1) == BAD and st(T=-1) == BAD and st(H=-1) == BAD
    assert st(lq=191) == BAD and st(lk=196) == BAD and st(lv=100) == BAD and st(cu=FAKE + 2) == BAD and st(par=FAKE + 1) == BAD
    assert st(dk=64, lq=128, lk=128) == NOT and st(dt=1, dk=129) == NOT and st(dt=1, dv=257) == NOT and st(dt=3) == BAD
    assert st(ns=1 << 24, H=2) == NOT                              # rows of pages past an int
    assert st(dk=0) == BAD and st(o=FAKE) == BAD and st(nseq=1 << 20, ns=1 << 20, H=1 << 12) == BAD
    assert st(nseq=0, q=None, cu=None, o=None) == OK and st(H=0, q=None) == OK and st(T=0, q=None, o=None, par=None) == OK


def commit(L, k=FAKE, lk=192, v=FAKE, lv=384, log=FAKE, cu=FAKE, par=FAKE, last=FAKE, slots=FAKE, pool=FAKE, x=FAKE,
           lx=64, win=FAKE, ns=4, nseq=2, T=8, H=2, dk=96, dv=192, D=64, dt=0, name="gla_tree_commit"):
    return getattr(L, name)(k, lk, v, lv, log, cu, par, last, slots, pool, x, lx, win, ns, nseq, T, H, dk, dv, D, dt, None)


@pytest.mark.parametrize("name", ["gla_tree_commit", "gla_tree_commit_gated"])
def test_tree_commit(L, name):
    def st(**kw):
        return commit(L, name=name, **kw)

    for null in ("k", "v", "log", "cu", "par", "last", "pool", "x", "win"):
        assert st(**{null: None}) == BAD, null
    for odd in ("k", "v", "pool", "x", "win"):
        assert st(**{odd: ODD}) == BAD, odd
    assert st(D=12) == NOT and st(D=0) == NOT and st(lx=60) == BAD and st(last=FAKE + 2) == BAD and st(dk=90) == NOT
    assert st(slots=None, ns=1) == BAD and st(T=-1) == BAD
    assert st(nseq=0, k=None) == OK and st(T=0, k=None, par=None) == OK and st(H=0, x=None, win=None) == OK


def test_conv1d_tree(L):
    def st(x=FAKE, lx=64, w=FAKE, b=FAKE, cu=FAKE, par=FAKE, slots=FAKE, win=FAKE, ns=4, nseq=2, T=8, D=64, dt=0, y=2 * FAKE):
        return L.gla_conv1d_tree(x, lx, w, b, cu, par, slots, win, ns, nseq, T, D, dt, y, None)

    for null in ("x", "w", "cu", "par", "win", "y"):
        assert st(**{null: None}) == BAD, null
    for odd in ("x", "w", "b", "win", "y"):
        assert st(**{odd: ODD}) == BAD, odd
    assert st(D=20) == NOT and st(lx=63) == BAD and st(lx=68) == BAD and st(y=FAKE) == BAD and st(slots=None, ns=1) == BAD
    assert st(nseq=0, x=None) == OK and st(T=0, x=None, par=None) == OK


def test_pages(L):
    def arrays(ptrs, sizes):
        return (ctypes.c_void_p * len(ptrs))(*ptrs), (ctypes.c_int64 * len(sizes))(*sizes)

    def copy(ptrs=(FAKE, FAKE), sizes=(64, 8), n_pools=2, ns=4, src=FAKE, dst=FAKE, n=3):
        return L.gla_pages_copy(*arrays(ptrs, sizes), n_pools, ns, src, dst, n, None)

    assert copy(src=None) == BAD and copy(dst=None) == BAD and copy(src=FAKE + 2) == BAD and copy(n=-1) == BAD
    assert copy(ns=-1) == BAD and copy(n_pools=-1) == BAD and copy(ptrs=(FAKE, None)) == BAD and copy(ptrs=(ODD, FAKE)) == BAD
    assert copy(sizes=(64, 6)) == NOT and copy(sizes=(64, 0)) == NOT and copy(sizes=(64, 1 << 40)) == BAD
    assert copy((FAKE,) * 129, (4,) * 129, 129) == NOT
    assert copy(n=0, src=None) == OK and copy(n_pools=0, ptrs=(), sizes=()) == OK
    assert L.gla_pages_copy(None, None, 2, 4, FAKE, FAKE, 1, None) == BAD
    assert L.gla_pages_clear(*arrays((FAKE,), (64,)), 1, 4, None, 2, None) == BAD

    def compact(ns=4, live=FAKE, to=FAKE, count=FAKE, ws=FAKE, size=1 << 20):
        return L.gla_pages_compact(*arrays((FAKE,), (64,)), 1, ns, live, to, count, ws, size, None)

    assert compact(live=None) == BAD and compact(to=None) == BAD and compact(count=None) == BAD and compact(ns=-1) == BAD
    assert compact(to=FAKE + 1) == BAD and compact(ns=5000, ws=None) == BAD and compact(ns=5000, size=8) == WS
    assert [L.gla_pages_compact_workspace_size(n) for n in (-1, 0, 4096)] == [0, 0, 0]
    assert L.gla_pages_compact_workspace_size(5000) >= 4 * 5001
    assert L.gla_pages_compact_workspace_size(2 ** 31 - 1) >= 4 * (2 ** 31 - 1)


def test_layernorm(L):
    def st(x=FAKE, res=FAKE, w=FAKE, b=FAKE, eps=1e-6, rows=4, D=64, dt=0, s=FAKE, y=2 * FAKE):
        return L.gla_layernorm_fwd(x, res, w, b, eps, rows, D, dt, s, y, None)

    assert st(x=None) == BAD and st(y=None) == BAD and st(eps=-1.0) == BAD and st(eps=float("nan")) == BAD
    for odd in ("x", "res", "w", "b", "s", "y"):
        assert st(**{odd: ODD}) == BAD, odd
    assert st(D=60) == NOT and st(D=8200) == NOT and st(D=0) == NOT and st(rows=-1) == BAD and st(dt=2) == BAD
    assert st(y=FAKE) == BAD and st(rows=0, x=None, y=None) == OK

    def bwd(s=FAKE, w=FAKE, dy=FAKE, ds=FAKE, eps=1e-6, rows=4, D=64, dt=0, dx=2 * FAKE, dw=FAKE, db=FAKE, ws=FAKE, size=1 << 30):
        return L.gla_layernorm_bwd(s, w, dy, ds, eps, rows, D, dt, dx, dw, db, ws, size, None)

    for null in ("s", "dy", "dx", "ws"):
        assert bwd(**{null: None}) == BAD, null
    for odd in ("s", "w", "dy", "ds", "dx", "dw", "db", "ws"):
        assert bwd(**{odd: ODD}) == BAD, odd
    assert bwd(dx=FAKE) == BAD and bwd(size=4) == WS and bwd(dw=None, size=4) == WS and bwd(D=60) == NOT
    assert L.gla_layernorm_bwd_workspace_size(0, 64, 0) == 0 and L.gla_layernorm_bwd_workspace_size(4, 60, 0) == 0
    assert L.gla_layernorm_bwd_workspace_size(4, 64, 0) == 4 * 2 * 64 * 4


def test_tensors_on_the_host_are_refused():
    import torch

    q, v, ints = torch.zeros(3, 2, 96, dtype=torch.bfloat16), torch.zeros(3, 2, 192, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    pool = torch.zeros(2, 2, 96, 192)
    for f in (lambda: binding.gla_tree_fwd(q, q, v, torch.zeros(2), ints, ints, pool),
              lambda: binding.gla_tree_commit(q, v, torch.zeros(2), ints, ints, ints, pool),
              lambda: binding.gla_conv1d_tree(q[:, 0], torch.zeros(96, 4), None, ints, ints, torch.zeros(2, 4, 96)),
              lambda: binding.gla_pages_copy(pool, ints, ints), lambda: binding.gla_pages_clear([pool], ints),
              lambda: binding.gla_pages_compact(pool, torch.ones(2, dtype=torch.bool)),
              lambda: binding.gla_layernorm(q), lambda: binding.gla_layernorm_bwd(q, None, q)):
        with pytest.raises(binding.GlaError):
            f()
