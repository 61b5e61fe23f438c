"""Batches of drafted trees far larger than what the GPU works on at a time."""
import pytest
import torch

import tree_plain as plain
from test_gpu_tree import BF, FP, Case, gla, ints, near

pytestmark = pytest.mark.gpu


def test_convolution_of_2560_full_trees(gla):
    """1.3 GB of packed rows: the same as its two halves, and a few trees as the definition."""
    N, D, some = 2560, 4096, [0, 1, 1279, 1280, 2559]
    c = Case(BF, [64] * N, 1, 96, 192, seed=3, behind=0)
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(c.T, D, generator=g, device="cuda", dtype=BF)
    win = torch.randn(N + 2, 4, D, generator=g, device="cuda")
    w, b = torch.randn(D, 4, generator=g, device="cuda") * 0.5, torch.randn(D, generator=g, device="cuda")
    slots, parents = ints(c.slots), ints(c.parents)
    y = gla.gla_conv1d_tree(x, w, b, ints(c.cu), parents, win, slots)
    gla.gla_check()
    half = N // 2
    for n in (0, half):
        rows = slice(c.cu[n], c.cu[n + half])
        part = gla.gla_conv1d_tree(x[rows], w, b, ints([64 * i for i in range(half + 1)]), parents[rows], win, slots[n:n + half])
        assert torch.equal(part, y[rows])
    gla.gla_check()
    rows = [t for n in some for t in range(64 * n, 64 * n + 64)]
    ref, tol = plain.conv_tree(x[rows].double().cpu(), w.double().cpu(), b.double().cpu(), [64 * i for i in range(len(some) + 1)],
                               [c.parents[t] for t in rows], [c.slots[n] for n in some], win.double().cpu())
    near(y[rows], ref, tol, "y")


def kept_page(c, n, pool, k, v, logs):
    """Sequence n's page after its path, and the sum of its terms' magnitudes, float64 on the GPU."""
    first = c.cu[n]
    S = pool[c.slots[n]].double()
    A = S.abs()
    path = plain.way(c.parents[first: c.cu[n + 1]], c.last[n])
    for t in (first + j for j in path):
        w, kv = torch.exp(logs[t])[:, None, None], k[t][:, :, None] * v[t][:, None, :]
        S, A = w * S + kv, w * A + kv.abs()
    return S, (len(path) + 6) * 2.0 ** -24 * A      # test_gpu_tree_bounds.py derives the bound


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("N,shape", [(200, "mixed"), (190, "chain"), (40, "chain")])
def test_commit_of_many_units_a_cta(gla, dtype, gated, N, shape):
    """Up to 21 pages a CTA one behind another, paths of 1 to 64 nodes: with some that stay and two bad entries between
    those that change, and several pieces of the windows a warp."""
    H, D = 16, 1032
    c = Case(dtype, [(7 * n) % 65 for n in range(N)], H, 96, 192, shape=shape, gated=gated, seed=N, D=D)
    c.last = [-1 if n % 9 == 4 else last if n % 3 else c.cu[n + 1] - c.cu[n] - 1 for n, last in enumerate(c.last)]
    bad = [17, 29]                                  # a parent behind its node, an accepted node that is not there
    assert all(c.cu[n + 1] - c.cu[n] > 3 for n in bad)
    pool, win = c.pool.clone(), c.win.clone()
    _, k, v = (t.double() for t in (c.q, c.k, c.v))
    logs = (c.log if gated else c.log.expand(c.q.shape[0], -1)).double()
    kept = [n for n in range(N) if c.last[n] >= 0 and n not in bad]
    windows = plain.windows(c.x.double().cpu(), c.cu, c.parents, [last if n in kept else -1 for n, last in enumerate(c.last)], c.slots,
                            win.double().cpu())
    want = {n: kept_page(c, n, pool, k, v, logs) for n in kept}
    c.parents[c.cu[bad[0]] + 2] = 2
    c.last[bad[1]] = c.cu[bad[1] + 1] - c.cu[bad[1]]
    results = []
    for _ in range(2):
        c.pool, c.win = pool.clone(), win.clone()
        c.commit(gla)
        with pytest.raises(gla.GlaError):
            gla.gla_check()
        results.append((c.pool, c.win))
    assert all(torch.equal(a, b) for a, b in zip(*results))
    for n, (S, tol) in want.items():
        off = (c.pool[c.slots[n]].double() - S).abs()
        assert (off <= tol + 1e-36).all(), (n, float((off / (tol + 1e-36)).max()))
    still = [s for s in range(N + 2) if s not in [c.slots[n] for n in kept]]
    assert len(still) > N // 9 and torch.equal(c.pool[still], pool[still]) and torch.equal(c.win.double().cpu(), windows)


@pytest.mark.parametrize("dtype,D", [(BF, 8), (BF, 4096), (FP, 516)])
def test_windows_without_heads(gla, dtype, D):
    """A layer's windows alone (H = 0), a bad parent among them."""
    N = 70
    c = Case(dtype, [(5 * n) % 65 for n in range(N)], 1, 96, 192, seed=5, D=D)
    empty, log = c.k[:, :0], torch.empty(0, device="cuda")
    c.parents[c.cu[9] + 2] = 5
    kept = [last if n != 9 else -1 for n, last in enumerate(c.last)]
    want = plain.windows(c.x.double().cpu(), c.cu, c.parents, kept, c.slots, c.win.double().cpu())
    gla.gla_tree_commit(empty, empty.new_empty(empty.shape[0], 0, 192), log, *c.tree_args(), ints(c.last),
                        torch.empty(N + 2, 0, 96, 192, device="cuda"), ints(c.slots), x=c.x, win_pool=c.win)
    with pytest.raises(gla.GlaError):
        gla.gla_check()
    assert torch.equal(c.win.double().cpu(), want)
