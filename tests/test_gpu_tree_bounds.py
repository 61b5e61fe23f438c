"""The commit's and the fp32 readout's own error bounds (tree_plain.py's also
cover the readout at bf16, with its halves of 16 bits).

In units of 2^-24, with CUDA's expf at 2 steps (4 units) and a decay's last
rounding 1: a decay is off by 5 of itself, however many nodes it runs over. An
entry of a committed page is a decay times the page's entry (6 units of it)
plus, for every node of a path of L, fma(decay k, v): 6 units of the term, and
one of the sum so far for each of L additions. Together at most L + 6 of the
sum of the terms' magnitudes.
A readout's terms: sums of dk products, one unit of their magnitudes an fma;
the decay's product 6; L additions, the scale 1: dk + L + 8."""
import pytest
import torch

import tree_plain as plain
from test_gpu_tree import BF, FP, INF, Case, gla, ints

pytestmark = pytest.mark.gpu
UNIT = 2.0 ** -24


def within(got, ref, tol, name):
    off = (got.double().cpu() - ref).abs()
    assert (off <= tol + 1e-36).all(), (name, float((off / (tol + 1e-36)).max()))


def committed(c):
    """Pages after the commit and their bounds, float64 on the host."""
    _, k, v = c.host()
    pool, logs = c.pool.double().cpu(), c.logs()
    tol = torch.zeros_like(pool)
    for n, first, par in plain.each(c.cu, c.parents):
        if c.last[n] < 0:
            continue
        S = pool[c.slots[n]]
        A, path = S.abs(), plain.way(par, c.last[n])
        for t in (first + j for j in path):
            w, kv = torch.exp(logs[t])[:, None, None], k[t][:, :, None] * v[t][:, None, :]
            S, A = torch.where(w == 0, 0 * kv, w * S) + kv, torch.where(w == 0, 0 * kv, w * A) + kv.abs()
        pool[c.slots[n]], tol[c.slots[n]] = S, (len(path) + 6) * UNIT * A
    return pool, tol


PAGES = [(BF, 96, 192), (FP, 96, 192), (FP, 33, 130), (FP, 40, 76), (FP, 5, 7)]


@pytest.mark.parametrize("dtype,dk,dv", PAGES)
@pytest.mark.parametrize("shape", ["chain", "mixed", "star"])
@pytest.mark.parametrize("gates", [0.0, 0.2, 3.0])
def test_committed_pages(gla, dtype, dk, dv, shape, gates):
    c = Case(dtype, [64, 40, 3, 1, 17], 3, dk, dv, shape=shape, gated=gates > 0, seed=1, gates=gates)
    c.last = [63, 39, 2, 0, 9]
    ref, tol = committed(c)
    c.commit(gla)
    gla.gla_check()
    within(c.pool, ref, tol, "pool")


@pytest.mark.parametrize("dtype,dk,dv", PAGES)
@pytest.mark.parametrize("gated", [False, True])
def test_decays_of_long_paths(gla, dtype, dk, dv, gated):
    """With k = 0 a page is its old value times the path's decay: 6 units, of 64 nodes as of one."""
    for last in ([63, 40], [0, 31], [32, 1]):
        c = Case(dtype, [64, 50], 6, dk, dv, shape="chain", gated=gated, seed=2, gates=0.45)
        if not gated:
            c.log = torch.tensor([-0.3, -0.1234, -1.0 / 3, -0.7, 0.0, -1e-4], device="cuda")
        c.last = last
        c.k.zero_()
        before, logs = c.pool.double().cpu(), c.logs()
        c.commit(gla)
        gla.gla_check()
        for n, s in enumerate(c.slots):
            decay = torch.exp(logs[c.cu[n]: c.cu[n] + last[n] + 1].sum(0))[:, None, None]
            within(c.pool[s], decay * before[s], 6 * UNIT * (decay * before[s]).abs(), (n, last[n]))


@pytest.mark.parametrize("dk,dv", [(96, 192), (128, 256), (33, 130), (5, 7), (1, 1)])
@pytest.mark.parametrize("shape", ["chain", "mixed", "star"])
@pytest.mark.parametrize("gates", [0.0, 0.2, 3.0])
def test_readout_at_fp32(gla, dk, dv, shape, gates):
    c = Case(FP, [64, 21, 1, 34], 2, dk, dv, shape=shape, gated=gates > 0, seed=3, gates=gates)
    q, k, v = c.host()
    pool, logs, o = c.pool.double().cpu(), c.logs(), c.fwd(gla)
    gla.gla_check()
    for n, first, par in plain.each(c.cu, c.parents):
        for i, (S, A, _) in enumerate(plain.states(k, v, logs, pool[c.slots[n]], par, first)):
            t, bound = first + i, (dk + len(plain.way(par, i)) + 8) * UNIT * c.scale
            within(o[t], c.scale * torch.einsum("hd,hdv->hv", q[t], S), bound * torch.einsum("hd,hdv->hv", q[t].abs(), A), t)


@pytest.mark.parametrize("dtype", [BF, FP])
def test_a_decay_of_zero_among_long_paths(gla, dtype):
    c = Case(dtype, [64, 64], 2, 96, 192, shape="chain", gated=True, seed=4, gates=0.5)
    c.log[30] = c.log[64 + 50, 1] = -INF
    c.last = [63, 63]
    ref, tol = committed(c)
    c.pool[c.slots[0]] = float("nan")            # cleared: what lies before counts nothing
    c.commit(gla)
    gla.gla_check()
    within(c.pool, ref, tol, "pool")


@pytest.mark.parametrize("dtype,dk,dv", PAGES)
def test_fixed_decays_of_zero_and_one(gla, dtype, dk, dv):
    """log_lambda -inf keeps a path's last node alone, whatever the page holds; 0 keeps everything; -60 and -104 run out on the way."""
    c = Case(dtype, [64, 9], 4, dk, dv, shape="chain", seed=6)
    c.log = torch.tensor([-INF, 0.0, -60.0, -104.0], device="cuda")
    c.last = [63, 8]
    ref, tol = committed(c)
    c.pool[:, 0] = float("nan")
    used = c.slots[:2]
    o = c.fwd(gla)[: c.T]
    c.commit(gla)
    gla.gla_check()
    within(c.pool[used], ref[used], tol[used], "pool")
    assert torch.isfinite(o.float()).all()
