"""Rates at the edge of fp32 in the selective scan: A of the type's lowest
value, and -inf, clear the state at every step above 0 and keep it at a step of
0, in sequences that end inside a tile too (the tokens behind their end have a
step of 0). Against the definition in float64, where the lowest value's decay
is exactly 0; -inf gives the same bits as the lowest value."""
import pytest
import torch

import test_gpu_ssm as fw
import test_gpu_ssm_bwd as bw
from ssm_plain import close
from test_gpu_ssm import BF, FP, gla  # noqa: F401

pytestmark = pytest.mark.gpu
LOWEST = torch.finfo(FP).min


def cleared(s, value):
    """The same inputs with `value` as the rate of some states and of one whole channel."""
    A = s["A"].clone()
    A[:, 1] = value
    A[3] = value
    return dict(s, A=A)


@pytest.mark.parametrize("dtype,B,T,D,N", [(FP, 2, 16, 24, 16), (BF, 1, 21, 24, 16), (FP, 1, 1, 8, 8), (FP, 1, 45, 40, 32),
                                           (FP, 1, 2501, 64, 16), (BF, 43, 19, 520, 16)])
def test_forward(gla, dtype, B, T, D, N):  # noqa: F811
    s = fw.inputs((B, T), D, N, dtype, 500 + T)
    h0 = torch.randn(B, D, N, generator=torch.Generator().manual_seed(T)).cuda()
    low = cleared(s, LOWEST)
    y, hT = fw.call_fwd(gla, low, h0)
    ry, my, rh, mh = fw.ref_fwd(low, h0)
    close(y, ry, my, T, "y")
    close(hT, rh, mh, T, "hT")
    y1, h1 = fw.call_fwd(gla, cleared(s, float("-inf")), h0)
    gla.gla_check()
    assert torch.equal(y1, y) and torch.equal(h1, hT)


@pytest.mark.parametrize("lens", [[5, 0, 33, 1], [1300, 17]])
def test_packed_prompts(gla, lens):  # noqa: F811
    D, N, n = 40, 16, len(lens)
    cu = [sum(lens[:i]) for i in range(n + 1)]
    s = fw.inputs((cu[-1],), D, N, FP, 3)
    pool, win, w, b = fw.pools(n, D, N, 8)
    got = []
    for value in (LOWEST, float("-inf")):
        p1, w1 = pool.clone(), win.clone()
        got.append((fw.call_varlen(gla, cleared(s, value), fw.i32(cu), p1, None, w, b, w1), p1))
    gla.gla_check()
    for i, (ry, my, rh, mh, _) in enumerate(fw.ref_packed(cleared(s, LOWEST), cu, list(range(n)), pool, win, w, b)):
        close(got[0][0][cu[i]:cu[i + 1]], ry, my, lens[i], f"y of {i}")
        close(got[0][1][i], rh, mh, max(lens[i], 1), f"state of {i}")
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


def test_single_tokens_and_a_step_of_zero(gla):  # noqa: F811
    D, N, n = 24, 16, 5
    s = fw.inputs((n,), D, N, FP, 4, bias=False)
    s["dt"][2:4] = -300.0                                   # softplus underflows to 0
    pool = torch.randn(n, D, N, generator=torch.Generator().manual_seed(2)).cuda()
    got = []
    for value in (LOWEST, float("-inf")):
        p1 = pool.clone()
        got.append((fw.call_step(gla, cleared(s, value), p1), p1))
    gla.gla_check()
    for i, (ry, my, rh, mh, _) in enumerate(fw.ref_packed(cleared(s, LOWEST), list(range(n + 1)), list(range(n)), pool,
                                                          None, None, None)):
        close(got[0][0][i:i + 1], ry, my, 1, f"y of {i}")
        close(got[0][1][i], rh, mh, 1, f"state of {i}")
    assert torch.equal(got[0][1][2:4], pool[2:4])
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


@pytest.mark.parametrize("dtype,B,T,D,N", [(FP, 2, 16, 24, 16), (BF, 1, 21, 24, 16), (FP, 1, 5, 8, 8), (FP, 1, 45, 40, 32),
                                           (FP, 1, 1001, 16, 16), (FP, 620, 17, 12, 8)])
def test_gradients(gla, dtype, B, T, D, N):  # noqa: F811
    s = fw.inputs((B, T), D, N, dtype, 700 + T)
    dy, h0, dhT = bw.extras(s, True, T)
    low = cleared(s, LOWEST)
    got = bw.call(gla, low, dy, h0, dhT)
    bw.check(got, *bw.reference(low, dy, h0, dhT), T)
    again = bw.call(gla, cleared(s, float("-inf")), dy, h0, dhT)
    gla.gla_check()
    assert all(torch.equal(v, again[k]) for k, v in got.items())


def test_a_rate_that_is_not_a_number_stays_one(gla):  # noqa: F811
    s = fw.inputs((1, 21), 16, 16, FP, 6)
    s["A"][5, 2] = float("nan")
    y, hT = fw.call_fwd(gla, s)
    gla.gla_check()
    assert torch.isnan(y[0, :, 5]).all() and torch.isnan(y).sum() == 21
    assert torch.isnan(hT[0, 5, 2]) and torch.isnan(hT).sum() == 1
