"""gla_conv1d_bwd on the GPU against its formula in float64, against the
library's own forward by differences, and on its edges.

Tolerances. a_t is a sum of five terms and SiLU'(a) has a slope below 0.5 and
its own exponential and reciprocal (2^-22 each), so dp_t is off by at most
A = 2e-6 |dy| (1 + |w| . |x|); dx adds four such products; dw and db are sums
over tiles of tokens and CTAs, a further (tokens in a tile + 40) 2^-24 < 1e-5
relative to the sum of magnitudes."""
import pytest
import torch

from ssm_plain import F64, d, half_step

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def gla():
    import linear_attention_chunk_gb300 as m
    from linear_attention_chunk_gb300.build import build
    build()
    return m


def make(B, T, D, dtype, seed, window=True, bias=True):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s, std=1.0, dt=FP: (torch.randn(*s, generator=g) * std).to(dt).cuda()  # noqa: E731
    return (rn(B, T, D, dt=dtype), rn(D, 4, std=0.5), rn(D, std=0.1) if bias else None, rn(B, T, D, dt=dtype),
            rn(B, 4, D) if window else None)


def formula(x, w, b, dy, win):
    """(dx, dw, db) by autograd in float64, and the magnitudes of their terms."""
    B, T, D = x.shape
    xd, wd = d(x).requires_grad_(), d(w).requires_grad_()
    bd = (torch.zeros(D, dtype=F64) if b is None else d(b)).requires_grad_()
    past = torch.zeros(B, 3, D, dtype=F64) if win is None else d(win)[:, 1:]
    rows = torch.cat([past, xd], 1)
    acc = bd + sum(rows[:, j:j + T] * wd[:, j] for j in range(4))
    (acc * torch.sigmoid(acc) * d(dy)).sum().backward()
    r = rows.detach().abs()
    amag = bd.detach().abs() + sum(r[:, j:j + T] * wd.detach()[:, j].abs() for j in range(4))
    dp = d(dy).abs() * (1 + amag)
    ahead = torch.cat([dp, torch.zeros(B, 3, D, dtype=F64)], 1)
    mx = sum(wd.detach()[:, j].abs() * ahead[:, 3 - j:3 - j + T] for j in range(4))
    mw = torch.stack([(dp * r[:, j:j + T]).sum((0, 1)) for j in range(4)], 1)
    return (xd.grad, wd.grad, bd.grad), (mx, mw, dp.sum((0, 1)))


def check(got, ref, mag):
    for name, g, r, m, k in zip(("dx", "dw", "db"), got, ref, mag, (4e-6, 1.2e-5, 1.2e-5)):
        tol = half_step(g.dtype) * r.abs() + k * m + 1e-30
        assert d(g).shape == r.shape and ((d(g) - r).abs() <= tol).all(), (name, float(((d(g) - r).abs() / tol).max()))


@pytest.mark.parametrize("dtype,B,T,D,window,bias", [
    (BF, 1, 1, 8, True, True), (FP, 2, 2, 4, True, True), (FP, 1, 3, 516, False, True), (BF, 3, 53, 1032, True, True),
    (BF, 2, 130, 72, True, False), (FP, 2, 257, 68, True, True), (BF, 1, 1000, 520, False, False),
    (FP, 5, 16, 1028, True, True), (BF, 1, 4, 64, True, True)])
def test_gradients_are_the_formula_s(gla, dtype, B, T, D, window, bias):
    a = make(B, T, D, dtype, 10 + T, window, bias)
    got = gla.gla_conv1d_bwd(*a)
    gla.gla_check()
    check(got, *formula(*a))
    again = gla.gla_conv1d_bwd(*a)
    assert all(torch.equal(u, v) for u, v in zip(got, again))
    dx, dw, db = gla.gla_conv1d_bwd(*a, want_db=False)
    gla.gla_check()
    assert db is None and torch.equal(dw, got[1]) and torch.equal(dx, got[0])


def test_against_differences_of_the_forward(gla):
    """fp32: (L(x + h v) - L(x - h v)) / 2h, off by the forward's rounding (2^-21 of sum |y dy|) / h and h^2."""
    x, w, b, dy, win = make(2, 20, 16, FP, 3)
    dx, dw, db = gla.gla_conv1d_bwd(x, w, b, dy, win)
    g = torch.Generator().manual_seed(5)
    h = 1e-2
    for of, grad in ((0, dx), (1, dw), (2, db)):
        v = torch.randn([x, w, b][of].shape, generator=g).cuda()
        vals = []
        for k in (h, -h):
            args = [x, w, b]
            args[of] = (args[of] + k * v).contiguous()
            vals.append((gla.gla_conv1d_fwd(*args, win, want_window=False)[0].double() * dy.double()).sum().item())
        want, got = (vals[0] - vals[1]) / (2 * h), (grad.double() * v.double()).sum().item()
        mag = (grad.double() * v.double()).abs().sum().item()
        assert abs(want - got) <= 640 * 2.0 ** -21 / h + 5 * h * h * (mag + 640)


def test_not_a_number_reaches_four_tokens_and_its_channel(gla):
    x, w, b, dy, win = make(1, 40, 16, FP, 7)
    clean = gla.gla_conv1d_bwd(x, w, b, dy, win)
    dy[0, 20, 3] = float("nan")
    dx, dw, db = gla.gla_conv1d_bwd(x, w, b, dy, win)
    gla.gla_check()
    bad = torch.zeros(1, 40, 16, dtype=torch.bool, device="cuda")
    bad[0, 17:21, 3] = True
    assert torch.equal(torch.isnan(dx), bad) and torch.equal(dx[~bad], clean[0][~bad])
    assert torch.isnan(dw[3]).all() and torch.isnan(dw).sum() == 4 and torch.isnan(db).sum() == 1


def test_large_inputs_stay_finite(gla):
    x, w, b, dy, win = make(1, 30, 16, FP, 8)
    x = x * 1e4
    got = gla.gla_conv1d_bwd(x, w, b, dy, win)
    gla.gla_check()
    assert all(torch.isfinite(v).all() for v in got)


def test_no_tokens_and_capture(gla):
    x, w, b, dy, win = make(2, 40, 64, BF, 9)
    dx, dw, db = gla.gla_conv1d_bwd(x[:, :0].contiguous(), w, b, dy[:, :0].contiguous(), win)
    gla.gla_check()
    assert dx.shape == (2, 0, 64) and not dw.any() and not db.any()
    want = gla.gla_conv1d_bwd(x, w, b, dy, win)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = gla.gla_conv1d_bwd(x, w, b, dy, win)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(got, want))
