"""The serving steps of speculative decoding run together, as a layer of a
serving loop runs them: the layer norm, the convolution along the drafted
trees, the mixer over them, its epilogue, the accepted paths kept, and the
pools' pages copied, moved and cleared between the steps -- against the same
tokens taken one by one through the steps that serve without drafts."""
import random

import pytest
import torch

from ssm_plain import half_step
from tree_plain import forest, way

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
H, DK, DV, D = 4, 96, 192, 256


@pytest.fixture(scope="module")
def gla():
    import linear_attention_chunk_gb300 as m
    from linear_attention_chunk_gb300.build import build
    build()
    return m


def ints(v):
    return torch.tensor(v, dtype=torch.int32).cuda()


class Layer:
    """A layer's parameters, and the projections that the library leaves to others."""

    def __init__(self, gated):
        g = torch.Generator().manual_seed(3)

        def rn(*s, std=1.0):
            return (torch.randn(*s, generator=g) * std).cuda()

        self.gated = gated
        self.w, self.b = 1 + rn(D, std=0.1), rn(D, std=0.1)
        self.cw, self.cb = rn(D, 4, std=0.5), rn(D, std=0.1)
        self.proj = rn(D, H * (2 * DK + 2 * DV), std=D ** -0.5).to(BF)
        self.gate = rn(D, H, std=D ** -0.5)
        self.lam = torch.log1p(-torch.exp2(-3.0 - torch.arange(H))).cuda()
        self.aug, self.nw = rn(H, DK, std=0.3), 1 + rn(H, DV, std=0.1)

    def split(self, y):
        """q, k, v (column ranges of one product), the output gate, and the log decays."""
        p = y @ self.proj
        q, k, v, z = (t.unflatten(1, (H, -1)) for t in p.split([H * DK, H * DK, H * DV, H * DV], 1))
        return q, k, v, z.contiguous(), -torch.nn.functional.softplus(y.float() @ self.gate)

    def tree(self, gla, x, res, cu, par, pool, win, slots):
        """A drafted step over every node: the layer's output, and what its commit needs."""
        h, s = gla.gla_layernorm(x, self.w, self.b, res)
        y = gla.gla_conv1d_tree(h, self.cw, self.cb, cu, par, win, slots)
        q, k, v, z, g = self.split(y)
        if self.gated:
            o = gla.gla_tree_fwd_gated(q, k, v, g, cu, par, pool, slots)
        else:
            o = gla.gla_tree_fwd(q, k, v, self.lam, cu, par, pool, slots)
        out = gla.gla_mixer_epilogue(o, q.contiguous(), k.contiguous(), v.contiguous(), z, self.aug, self.nw)
        return out, (h, k, v, g)

    def commit(self, gla, held, cu, par, last, pool, win, slots):
        h, k, v, g = held
        if self.gated:
            gla.gla_tree_commit_gated(k, v, g, cu, par, last, pool, slots, x=h, win_pool=win)
        else:
            gla.gla_tree_commit(k, v, self.lam, cu, par, last, pool, slots, x=h, win_pool=win)

    def step(self, gla, x, res, S, win):
        """One token a sequence, S and win in place."""
        h, s = gla.gla_layernorm(x, self.w, self.b, res)
        y = gla.gla_conv1d_step(h, self.cw, self.cb, win)
        q, k, v, z, g = self.split(y)
        q, k, v = (t.contiguous() for t in (q, k, v))
        o = gla.gla_decode_step_gated(q, k, v, g, S) if self.gated else gla.gla_decode_step(q, k, v, self.lam, S)
        return gla.gla_mixer_epilogue(o, q, k, v, z, self.aug, self.nw)


@pytest.mark.parametrize("gated", [False, True])
def test_a_serving_loop(gla, gated):
    """Three rounds: five sequences draft trees, keep a path each, one ends (its
    page is cleared), one is continued twice (its page is copied), the pools are
    compacted. The pages are then those of the tokens taken one by one.

    Tolerance. Both ways round h, y, o and z to bf16 from fp32. The step's SiLU
    (approximate tanh, 2^-11) differs from the tree's, so that y may round the
    other way, one step, 2^-7 relative; k, v and z carry that on by way of a
    product (bf16 again), and the states and outputs sum such terms: 2 % of the
    largest entry, the library's own bar for bf16, holds for all of them."""
    layer, rng = Layer(gated), random.Random(5)
    g = torch.Generator().manual_seed(9)
    n_slots, live = 12, [0, 3, 4, 8, 11]
    pool, win = torch.zeros(n_slots, H, DK, DV, device="cuda"), torch.zeros(n_slots, 4, D, device="cuda")
    pool[live] = (torch.randn(5, H, DK, DV, generator=g) * 0.1).cuda()
    win[live] = torch.randn(5, 4, D, generator=g).to(BF).float().cuda()
    alone = {s: (pool[s][None].clone(), win[s][None].clone()) for s in live}       # by page: a state and a window

    def close(a, b, name):
        assert torch.isfinite(a.float()).all() and float((a.double() - b.double()).abs().max() / b.double().abs().max()) < 2e-2, name

    for _ in range(3):
        sizes = [rng.choice([1, 5, 16, 33]) for _ in live]
        cu, par = forest(sizes, "mixed", rng.randrange(1000))
        T = cu[-1]
        x, res = ((torch.randn(T, D, generator=g)).to(BF).cuda() for _ in range(2))
        last = [rng.randrange(-1, n) for n in sizes]
        args = ints(cu), ints(par)
        out, held = layer.tree(gla, x, res, *args, pool, win, ints(live))
        layer.commit(gla, held, *args, ints(last), pool, win, ints(live))
        for n, slot in enumerate(live):
            tree = par[cu[n]:cu[n + 1]]
            for i in (last[n], len(tree) - 1):                     # the accepted path, and one that is not kept
                S, w = (t.clone() for t in alone[slot])
                for j in way(tree, i):
                    t = cu[n] + j
                    z = layer.step(gla, x[t][None], res[t][None], S, w)
                    close(out[t], z[0], "o")
                if i == last[n]:
                    kept = S, w
            alone[slot] = kept
            close(pool[slot], kept[0][0], "state")
            assert torch.equal(win[slot], kept[1][0])
        # one sequence ends, one is continued twice, the holes close up
        ended, copied, free = live.pop(1), live[0], next(s for s in range(n_slots) if s not in live)
        gla.gla_pages_clear([pool, win], ints([ended]))
        gla.gla_pages_copy([pool, win], ints([copied]), ints([free]))
        del alone[ended]
        alone[free] = tuple(t.clone() for t in alone[copied])
        live.append(free)
        used = torch.zeros(n_slots, dtype=torch.bool, device="cuda")
        used[live] = True
        moved, count = gla.gla_pages_compact([pool, win], used)
        moved = moved.tolist()
        assert count.item() == len(live) and sorted(moved[s] for s in live) == list(range(len(live)))
        alone = {moved[s]: alone[s] for s in live}
        live = [moved[s] for s in live]
        for s in live:
            close(pool[s], alone[s][0][0], "state")
            assert torch.equal(win[s], alone[s][1][0])
    gla.gla_check()


def test_a_training_pass_of_the_layer_norm(gla):
    """Two norms in a row with the residual between them, forward and backward,
    against autograd in float64 through the formula at the same rounded sums."""
    g = torch.Generator().manual_seed(1)

    def rn(*s, std=1.0):
        return torch.randn(*s, generator=g) * std

    x, r = rn(70, 264).to(BF).cuda(), rn(70, 264).to(BF).cuda()
    w, b = (1 + rn(2, 264, std=0.1)).cuda(), rn(2, 264, std=0.1).cuda()
    up = rn(70, 264).to(BF).cuda()
    y1, s1 = gla.gla_layernorm(x, w[0].contiguous(), b[0].contiguous(), r)
    y2, s2 = gla.gla_layernorm(y1, w[1].contiguous(), b[1].contiguous(), s1)
    d2, dw2, db2 = gla.gla_layernorm_bwd(s2, w[1].contiguous(), up)                 # of y1 and of s1 alike
    d1, dw1, db1 = gla.gla_layernorm_bwd(s1, w[0].contiguous(), d2, d2)
    gla.gla_check()

    def norm(s, w, b):
        c = s - s.mean(-1, keepdim=True)
        return c / (c.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w + b

    W, B = w.double().cpu().requires_grad_(), b.double().cpu().requires_grad_()
    a1 = s1.double().cpu().requires_grad_()
    a2 = s2.double().cpu().requires_grad_()
    (norm(a2, W[1], B[1]) * up.double().cpu()).sum().backward()
    e = d2.double().cpu()
    near(d2, a2.grad, 4e-5)
    near(dw2, W.grad[1], 4e-5)
    near(db2, B.grad[1], 4e-5)
    (norm(a1, W[0], B[0]) * e).sum().backward()
    near(d1, a1.grad + e, 4e-5)
    near(dw1, W.grad[0], 4e-5)
    near(db1, B.grad[0], 4e-5)


def near(got, ref, fp32):
    """Off by the output's rounding, and fp32 sums of 264 or 70 terms: (264 / 32 + 10) 2^-24 of magnitudes a few times
    the largest entry, 4e-5 of it with room for a sum of twenty such terms."""
    off = (got.double().cpu() - ref).abs()
    assert (off <= half_step(got.dtype) * ref.abs() + fp32 * ref.abs().max()).all(), float(off.max())
