"""Batches of drafted trees far larger than what the GPU works on at a time."""
import pytest
import torch

import tree_plain as plain
from test_gpu_tree import BF, Case, gla, ints, near

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
