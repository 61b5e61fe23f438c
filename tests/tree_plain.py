"""Trees of drafted tokens for the tests, and what the calls over them compute,
from the definition in float64 on the host: every node's state formed, one
update after the other, beside it what bounds an fp32 result's error.

A state entry is a sum of terms, each a product with a decay. Products, sums
and the decay's exponential are fp32: off by at most SUM = 5e-5 of the sum of
the terms' magnitudes (S.q over dk <= 128 products and as many additions,
128 2^-23 = 1.6e-5; q.k likewise; a term split in two bf16 halves for the
tensor cores, 2^-17 = 8e-6 each for S and P; 64 terms of the path, 64 2^-24).
The logarithms of a path's decays, up to 64, are added in fp32: the decay is off
by 64 2^-24 = 4e-6 of their sum, relative to itself."""
import random

import torch

SUM, LOG = 5e-5, 4e-6


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def tree(n, shape, seed):
    """Parents of a tree of n nodes: 'chain', 'star' (all roots), 'binary', or 'mixed'."""
    rng = random.Random(seed * 97 + n)
    pick = dict(chain=lambda i: i - 1, star=lambda i: -1, binary=lambda i: (i + 1) // 2 - 1,
                mixed=lambda i: i - 1 if rng.random() < 0.4 else rng.randint(-1, i - 1))[shape]
    return [pick(i) for i in range(n)]


def forest(sizes, shape, seed=0):
    """(offsets, parents) of trees packed one behind another, as lists."""
    cu, parents = [0], []
    for n, size in enumerate(sizes):
        parents += tree(size, shape, seed + n)
        cu.append(cu[-1] + size)
    return cu, parents


def way(par, i):
    """The nodes from the root's child down to i."""
    out = []
    while i >= 0:
        out.append(i)
        i = par[i]
    return out[::-1]


def each(cu, parents):
    for n in range(len(cu) - 1):
        yield n, cu[n], parents[cu[n]:cu[n + 1]]


def states(k, v, log, root, par, first):
    """For every node of a tree its state, the sum of the terms' magnitudes and
    the decays' error, from the page `root` [H, dk, dv]; log [T, H]."""
    out, start = [], (root, root.abs(), torch.zeros_like(root))
    for i, p in enumerate(par):
        S, A, E = start if p < 0 else out[p]
        t = first + i
        w = torch.exp(log[t])[:, None, None]
        kv = k[t][:, :, None] * v[t][:, None, :]
        grown = w * (E + LOG * log[t].abs().clamp(max=1e30)[:, None, None] * A)
        out.append((torch.where(w == 0, 0 * kv, w * S) + kv, torch.where(w == 0, 0 * kv, w * A) + kv.abs(),
                    torch.where(w == 0, 0 * kv, grown)))
    return out


def tree_fwd(q, k, v, log, scale, cu, parents, slots, pool):
    """o of every node and its tolerance without the output's rounding, float64 host tensors."""
    o, tol = torch.zeros_like(v), torch.zeros_like(v)
    for n, first, par in each(cu, parents):
        for i, (S, A, E) in enumerate(states(k, v, log, pool[slots[n]], par, first)):
            t = first + i
            o[t] = scale * torch.einsum("hd,hdv->hv", q[t], S)
            tol[t] = abs(scale) * torch.einsum("hd,hdv->hv", q[t].abs(), SUM * A + E)
    return o, tol


def commit(k, v, log, cu, parents, last, slots, pool):
    pool, tol = pool.clone(), torch.zeros_like(pool)
    for n, first, par in each(cu, parents):
        if last[n] >= 0:
            S, A, E = states(k, v, log, pool[slots[n]], par, first)[last[n]]
            pool[slots[n]], tol[slots[n]] = S, SUM * A + E
    return pool, tol


def windows(x, cu, parents, last, slots, win):
    win = win.clone()
    for n, first, par in each(cu, parents):
        rows = torch.cat([win[slots[n]]] + [x[first + i][None] for i in way(par, last[n])])
        win[slots[n]] = rows[-4:]
    return win


def conv_tree(x, w, b, cu, parents, slots, win):
    """y and its tolerance: four products and sums in fp32, 1e-6 of their
    magnitudes, SiLU's slope at most 1.1, its exponential and reciprocal 1e-6."""
    y, tol = torch.zeros_like(x), torch.zeros_like(x)
    for n, first, par in each(cu, parents):
        for i in range(len(par)):
            rows = torch.cat([win[slots[n], 1:], x[[first + j for j in way(par, i)[-4:]]]])[-4:]
            acc = b + (rows * w.t()).sum(0)
            y[first + i] = acc * torch.sigmoid(acc)
            tol[first + i] = 2e-6 * ((rows * w.t()).abs().sum(0) + b.abs()) + 4e-6 * y[first + i].abs()
    return y, tol
