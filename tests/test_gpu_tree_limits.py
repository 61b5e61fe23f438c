"""Calls over drafted trees and pages next to the largest numbers they take:
channels and pages just below 2^31."""
import pytest
import torch

import tree_plain as plain
from test_gpu_tree import BF, FP, gla, ints, near

pytestmark = pytest.mark.gpu
MOST = 2 ** 31 - 1


@pytest.fixture(autouse=True)
def give_back():
    """Up to 120 GB a test."""
    yield
    torch.cuda.empty_cache()


def rn(*shape, seed, dtype=FP):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda", dtype=dtype)


@pytest.mark.parametrize("dtype,D", [(BF, MOST // 8 * 8), (FP, MOST // 4 * 4)])
def test_convolution_of_the_most_channels(gla, dtype, D):
    parents = [-1, 0]
    x, win, w = rn(2, D, seed=1, dtype=dtype), rn(1, 4, D, seed=2), rn(D, 4, seed=3)
    y = gla.gla_conv1d_tree(x, w, None, ints([0, 2]), ints(parents), win)
    gla.gla_check()
    for a in (0, D // 2 // 256 * 256 - 8, D - 520):
        cut = slice(a, a + 520)
        ref, tol = plain.conv_tree(x[:, cut].double().cpu(), w[cut].double().cpu(), torch.zeros(520).double(), [0, 2], parents, [0],
                                   win[..., cut].double().cpu())
        near(y[:, cut], ref, tol, "y")


def test_windows_of_the_most_channels(gla):
    D = MOST // 8 * 8
    k, v, pool = rn(2, 1, 96, seed=1, dtype=BF), rn(2, 1, 192, seed=2, dtype=BF), rn(1, 1, 96, 192, seed=3)
    x, win = rn(2, D, seed=4, dtype=BF), rn(1, 4, D, seed=5)
    want = [win[0, 2].clone(), win[0, 3].clone(), x[0], x[1]]
    gla.gla_tree_commit(k, v, torch.zeros(1, device="cuda"), ints([0, 2]), ints([-1, 0]), ints([1]), pool, x=x, win_pool=win)
    gla.gla_check()
    for r in range(4):
        assert torch.equal(win[0, r], want[r].float()), r


def test_compaction_of_the_most_pages(gla):
    """Pages of 4 bytes: three not in use, two of those past the front move."""
    n = MOST
    pool, live = torch.arange(n, dtype=torch.int32, device="cuda"), torch.ones(n, dtype=torch.bool, device="cuda")
    live[[5, 1000, n - 3]] = False
    where, count = gla.gla_pages_compact(pool, live)
    gla.gla_check()
    same = torch.arange(n, dtype=torch.int32, device="cuda")
    assert int(count) == n - 3 and pool[[5, 1000]].tolist() == [n - 2, n - 1]
    assert where[[5, 1000, n - 3, n - 2, n - 1]].tolist() == [-1, -1, -1, 5, 1000]
    for t, odd in ((pool, [5, 1000]), (where, [5, 1000, n - 3, n - 2, n - 1])):
        t[odd] = same[odd]
        assert torch.equal(t, same)


def test_page_numbers_of_a_pool_without_pages(gla):
    """Every number is outside: the call moves nothing and the next check says so."""
    pools = [torch.empty(0, 4, device="cuda"), torch.empty(0, 3, 5, device="cuda")]
    for call in (lambda: gla.gla_pages_copy(pools, ints([0]), ints([1])), lambda: gla.gla_pages_clear(pools, ints([0]))):
        call()
        with pytest.raises(gla.GlaError) as e:
            gla.gla_check()
        assert e.value.status == gla.GLA_ERR_INVALID_ARG
    where, count = gla.gla_pages_compact(pools, torch.empty(0, dtype=torch.bool, device="cuda"))
    gla.gla_pages_copy(pools, ints([]), ints([]))
    gla.gla_check()
    assert where.numel() == 0 and int(count) == 0
