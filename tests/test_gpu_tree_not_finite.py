"""Entries of q, k, v and the page that are not finite, in the readout of
drafted trees: a result is an infinity of the same sign, or NaN, where the sum
of its terms is one,
    o_i = scale (F_i sum_r q_ir S_r + sum_j W_ij (sum_r q_ir k_jr) v_j),
and all others are what they are without such entries."""
import pytest
import torch

import tree_plain as plain
from test_gpu_tree import BF, FP, INF, NAN, Case, gla, ints

pytestmark = pytest.mark.gpu


def terms(c):
    """The sum of terms in float64 (no term of these inputs passes fp32's range unless it is infinite)."""
    (q, k, v), logs, pool = c.host(), c.logs(), c.pool.double().cpu()
    o = torch.zeros(c.T, c.H, c.dv, dtype=torch.float64)
    for n, first, par in plain.each(c.cu, c.parents):
        for i in range(len(par)):
            total, t = torch.zeros(c.H, dtype=torch.float64), first + i
            for j in plain.way(par, i)[::-1]:
                score = torch.exp(total) * (q[t] * k[first + j]).sum(-1)
                o[t] += score[:, None] * v[first + j]
                total = total + logs[first + j]
            o[t] += torch.exp(total)[:, None] * torch.einsum("hd,hdv->hv", q[t], pool[c.slots[n]])
    return c.scale * o


def kinds(o):
    o = o.double().cpu()
    return torch.where(o.isnan(), 2.0, torch.where(o.isinf(), o.sign(), 0.0))


PLACES = {
    "q": lambda c: c.q[5, 1, 3:4], "q twice": lambda c: c.q[5, 1, 3:90:60], "k": lambda c: c.k[5, 1, 3:4], "v": lambda c: c.v[5, 1, 20:90:23],
    "q and v": lambda c: (c.q[9, 1, 3:4], c.v[5, 1, 20:21]), "k and v": lambda c: (c.k[5, 1, 3:4], c.v[5, 1, 20:90:23]),
    "q and page": lambda c: (c.q[9, 1, 3:4], c.pool[c.slots[0], 1, 3, 20:21], c.pool[c.slots[0], 1, 8, 50:51]),
    "v and page": lambda c: (c.v[2, 1, 70:71], c.pool[c.slots[0], 1, 3, 70:71]),
    "all rows of q": lambda c: c.q[:, :, 3],
}


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("shape", ["binary", "chain", "star"])
@pytest.mark.parametrize("where", list(PLACES))
@pytest.mark.parametrize("value", [INF, -INF, NAN])
@pytest.mark.parametrize("one_sign", [True, False])
def test_sums_of_terms(gla, dtype, shape, where, value, one_sign):
    """With operands of one sign every infinity keeps its own, in each of one to four tiles of nodes."""
    for sizes in ([40, 16], [12], [64], [30, 1]):
        c = Case(dtype, sizes, 2, 96, 192, shape=shape, seed=8, gated=True)
        for name in "qkv":
            t = getattr(c, name)
            t = torch.where(t == 0, torch.ones_like(t), t)
            setattr(c, name, t.abs() if one_sign else t)
        c.pool = c.pool.abs() if one_sign else c.pool
        clean = c.fwd(gla)[: c.T].clone()
        at = PLACES[where](c)
        for t in at if isinstance(at, tuple) else (at,):
            t.fill_(value)
        want, got = kinds(terms(c)), c.fwd(gla)[: c.T]
        gla.gla_check()
        assert torch.equal(kinds(got), want)
        assert not one_sign or value != value or (want.abs() == 1).any() and not (want == 2).any() or "and" in where
        untouched = (want == 0).cuda()
        assert torch.equal(got[untouched], clean[untouched])


@pytest.mark.parametrize("value", [INF, -INF])
def test_an_infinite_q_as_the_steps(gla, value):
    """Operands of one sign: as gla_decode_step along the path, in every channel."""
    c = Case(BF, [20], 2, 96, 192, shape="chain", seed=9)
    c.q, c.k, c.v, c.pool = (torch.where(t == 0, torch.ones_like(t), t).abs() for t in (c.q, c.k, c.v, c.pool))
    c.q[:, :, 7] = value
    o, S = c.fwd(gla), c.pool[c.slots[0]][None].clone()
    for i in range(20):
        step = gla.gla_decode_step(c.q[i][None], c.k[i][None], c.v[i][None], c.log, S, c.scale)
        assert (o[i] == value).all() and (step == value).all()
    gla.gla_check()


@pytest.mark.parametrize("dtype", [BF, FP])
def test_scores_past_the_largest_number(gla, dtype):
    """q.k overflows where q and k are finite: an infinite score, with the sign of v."""
    c = Case(dtype, [33, 5], 2, 96, 192, shape="binary", seed=10)
    c.v = torch.where(c.v == 0, torch.ones_like(c.v), c.v)
    c.q[6, 0], c.k[6, 0] = 1e20, 1e20
    c.pool.abs_()
    o = c.fwd(gla)[: c.T]
    gla.gla_check()
    assert torch.equal(o[6, 0], c.v[6, 0].sign() * INF) and torch.isfinite(o[:6].float()).all() and torch.isfinite(o[7:13].float()).all()


@pytest.mark.parametrize("dtype", [BF, FP])
def test_a_decay_of_zero_hides_them(gla, dtype):
    """What lies before a clearing node, however far from finite: results as without it."""
    c = Case(dtype, [40, 16], 2, 96, 192, shape="chain", gated=True, seed=11)
    c.log[12, 1] = c.log[25, 1] = -INF
    clean = c.fwd(gla)[: c.T].clone()
    c.v[7, 1, 20], c.k[8, 1, 4], c.pool[c.slots[0], 1, 3, 70] = INF, -INF, NAN
    o = c.fwd(gla)[: c.T]
    gla.gla_check()
    assert torch.equal(o[12:], clean[12:]) and torch.equal(o[:, 0], clean[:, 0]) and not torch.isfinite(o[8:12, 1].float()).any()


def test_the_next_tree_s_rows_do_not_matter(gla):
    """A tile of 16 rows may hold rows of the next tree: not finite there, nothing here changes."""
    c = Case(BF, [5, 11, 3], 2, 96, 192, seed=12)
    clean = c.fwd(gla)[: c.T].clone()
    for t in (c.q, c.k, c.v):
        t[5:16] = NAN
    c.q[16:] = torch.where(torch.arange(c.q.shape[0] - 16, device="cuda")[:, None, None] < 3, c.q[16:], INF)
    o = c.fwd(gla)[: c.T]
    gla.gla_check()
    assert torch.equal(o[:5], clean[:5]) and torch.equal(o[16:], clean[16:]) and o[5:16].isnan().all()


@pytest.mark.parametrize("gated", [False, True])
def test_repeated_runs_are_equal(gla, gated):
    c = Case(BF, [(13 * n) % 33 for n in range(200)], 16, 96, 192, gated=gated, seed=13)
    first = c.fwd(gla)[: c.T].clone()
    for _ in range(20):
        assert torch.equal(c.fwd(gla)[: c.T], first)
    gla.gla_check()
