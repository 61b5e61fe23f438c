"""Residual addition, RMSNorm, its 8-bit output, and its gradients on the GPU
against their formulas in float64.

Tolerances. The row's sum of D squares and the mean of g xn are fp32 sums over
threads, warps and a tree: off by at most (D / threads + 10) 2^-24 relative to
the sum of magnitudes, under SUM = 1e-5 for D <= 8192; the other operations add
a few 2^-24. Outputs add half a step of their type."""
import pytest
import torch

from ssm_plain import F64, d, half_step

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float32
SUM = 1e-5


@pytest.fixture(scope="module")
def gla():
    import linear_attention_chunk_gb300 as m
    from linear_attention_chunk_gb300.build import build
    build()
    return m


def rn(*shape, seed, dtype=FP, std=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * std).to(dtype).cuda()


def near(got, ref, mag, name):
    g = d(got)
    tol = half_step(got.dtype) * ref.abs() + SUM * mag + 1e-30
    assert g.shape == ref.shape and ((g - ref).abs() <= tol).all(), (name, float(((g - ref).abs() / tol).max()))


def formula(x, res, w, eps):
    s = d(x) + (0 if res is None else d(res))
    y = s / (s.square().mean(-1, keepdim=True) + eps).sqrt()
    return s, y if w is None else y * d(w)


SHAPES = [(BF, 1, 8), (BF, 3, 72), (FP, 2, 4), (FP, 5, 516), (BF, 700, 1032), (BF, 2, 4096), (FP, 33, 2048),
          (BF, 9, 8192), (FP, 3, 8192), (BF, 1100, 264), (BF, 700, 2048)]


@pytest.mark.parametrize("dtype,rows,D", SHAPES)
@pytest.mark.parametrize("with_res,with_w", [(True, True), (False, False)])
def test_forward(gla, dtype, rows, D, with_res, with_w):
    x, res = rn(rows, D, seed=1, dtype=dtype), rn(rows, D, seed=2, dtype=dtype, std=3.0) if with_res else None
    w = 1 + rn(D, seed=3, std=0.2) if with_w else None
    y, s = gla.gla_rmsnorm(x, w, res, 1e-6)
    gla.gla_check()
    rs, ry = formula(x, res, w, 1e-6)
    near(y, ry, ry.abs(), "y")
    assert (s is None) == (res is None)
    if with_res:
        near(s, rs, 0 * rs, "s")
        inplace = res.clone()
        y1, s1 = gla.gla_rmsnorm(x, w, inplace, 1e-6, s=inplace)
        gla.gla_check()
        assert s1 is inplace and torch.equal(s1, s) and torch.equal(y1, y)


@pytest.mark.parametrize("dtype,rows,D", SHAPES)
@pytest.mark.parametrize("group", [0, 32, 64, 128])
def test_eight_bit_output(gla, dtype, rows, D, group):
    """The scale is the block's maximum over 448, and every stored value is the
    e4m3 number nearest to y / scale (half a step of e4m3 is 2^-4 relative,
    2^-10 below the least normal 2^-6; y and the quotient themselves are off
    by SUM and 2^-23, which can move a value at a border to its neighbour)."""
    x, res, w = rn(rows, D, seed=4, dtype=dtype), rn(rows, D, seed=5, dtype=dtype), 1 + rn(D, seed=6, std=0.2)
    y8, scale, s = gla.gla_rmsnorm_q8(x, w, res, 1e-6, group)
    gla.gla_check()
    _, ry = formula(x, res, w, 1e-6)
    g = group or D
    assert y8.dtype == torch.float8_e4m3fn and scale.shape == (rows, -(-D // g))
    parts = ry.split(g, 1)
    top = torch.stack([p.abs().amax(1) for p in parts], 1)
    assert ((d(scale) - top / 448).abs() <= 2 * SUM * top / 448).all()
    q = torch.cat([p / d(scale)[:, i:i + 1] for i, p in enumerate(parts)], 1)
    got = y8.float().cpu().to(F64)
    assert torch.isfinite(got).all() and got.abs().max() <= 448
    assert ((got - q).abs() <= (2.0 ** -4 + 4 * SUM) * q.abs() + 2.0 ** -10).all()
    assert torch.equal(s, gla.gla_rmsnorm(x, w, res, 1e-6)[1])


def test_zero_rows_blocks_and_not_a_number(gla):
    x = rn(4, 256, seed=7)
    x[1] = 0
    x[2, 128:] = 0
    y8, scale, s = gla.gla_rmsnorm_q8(x, group=128)
    gla.gla_check()
    assert s is None and (scale[1] == 1).all() and scale[2, 1] == 1 and scale[2, 0] != 1
    assert not y8[1].float().any() and not y8[2, 128:].float().any()
    y, _ = gla.gla_rmsnorm(x)
    assert not y[1].any()
    x[0, 5] = float("nan")
    x[3, 7] = float("inf")
    y1, _ = gla.gla_rmsnorm(x)
    y8, scale, _ = gla.gla_rmsnorm_q8(x, group=0)
    gla.gla_check()
    assert torch.isnan(y1[0]).all() and torch.isnan(scale[0]).all() and torch.isnan(y8[0].float()).all()
    assert torch.equal(y1[1:3], y[1:3]) and torch.isnan(y1[3, 7])       # inf / inf
    tiny = torch.full((1, 128), 1e-44, device="cuda")
    y8, scale, _ = gla.gla_rmsnorm_q8(tiny, group=128, eps=1.0)
    gla.gla_check()
    assert torch.isfinite(y8.float()).all() and scale.item() == 2.0 ** -126


@pytest.mark.parametrize("dtype,rows,D", SHAPES + [(FP, 5000, 64)])
@pytest.mark.parametrize("with_ds,with_w", [(True, True), (False, False)])
def test_backward_is_the_formula_s(gla, dtype, rows, D, with_ds, with_w):
    s, dy = rn(rows, D, seed=8, dtype=dtype), rn(rows, D, seed=9, dtype=dtype)
    ds = rn(rows, D, seed=10, dtype=dtype) if with_ds else None
    w = 1 + rn(D, seed=11, std=0.2) if with_w else None
    dx, dw = gla.gla_rmsnorm_bwd(s, w, dy, ds, 1e-6)
    gla.gla_check()
    x = d(s).requires_grad_()
    wt = (torch.ones(D, dtype=F64) if w is None else d(w)).requires_grad_()
    y = x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt() * wt
    ((y * d(dy)).sum() + (0 if ds is None else (x * d(ds)).sum())).backward()
    r = 1 / (d(s).square().mean(-1, keepdim=True) + 1e-6).sqrt()
    g = (d(dy) * (1 if w is None else d(w))).abs()
    mag = r * (g + (d(s) * r).abs() * (g * (d(s) * r).abs()).mean(-1, keepdim=True)) + (0 if ds is None else d(ds).abs())
    near(dx, x.grad, mag, "dx")
    near(dw, wt.grad, (d(dy) * d(s) * r).abs().sum(0), "dw")
    again = dy.clone()
    dx1, dw1 = gla.gla_rmsnorm_bwd(s, w, again, ds, 1e-6, dx=again)     # in place, and the same bits again
    gla.gla_check()
    assert torch.equal(dx1, dx) and torch.equal(dw1, dw)
    assert gla.gla_rmsnorm_bwd(s, w, dy, ds, 1e-6, want_dw=False)[1] is None


def test_backward_against_differences(gla):
    """fp32, step h along a direction: the forward's own rounding (2^-24 of
    sum |y dy|) over 2h and the third derivative's h^2 bound the difference."""
    s, dy, w, v = (rn(6, 64, seed=k) for k in (12, 13, 14, 15))
    w = w[0].contiguous()
    h = 1e-2
    up, down = ((gla.gla_rmsnorm((s + k * v).contiguous(), w)[0].double() * dy.double()).sum() for k in (h, -h))
    dx, _ = gla.gla_rmsnorm_bwd(s, w, dy)
    want, got = ((up - down) / (2 * h)).item(), (dx.double() * v.double()).sum().item()
    assert abs(want - got) <= 6 * 64 * 3 * 2 ** -24 / h + 30 * h * h * 6


def test_empty_and_leading_dimensions(gla):
    x = rn(2, 3, 64, seed=1, dtype=BF)
    y, _ = gla.gla_rmsnorm(x)
    y1, _ = gla.gla_rmsnorm(x.view(6, 64))
    assert y.shape == x.shape and torch.equal(y.view(6, 64), y1)
    y8, scale, _ = gla.gla_rmsnorm_q8(x, group=32)
    assert scale.shape == (2, 3, 2)
    e = x[:, :0]
    assert gla.gla_rmsnorm(e)[0].shape == (2, 0, 64)
    dx, dw = gla.gla_rmsnorm_bwd(e, None, e)
    gla.gla_check()
    assert dx.shape == (2, 0, 64) and not dw.any()


def test_capture_and_another_stream(gla):
    s, dy = rn(50, 256, seed=2, dtype=BF), rn(50, 256, seed=3, dtype=BF)
    w = 1 + rn(256, seed=4, std=0.1)
    want = gla.gla_rmsnorm_bwd(s, w, dy)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = gla.gla_rmsnorm_bwd(s, w, dy, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = gla.gla_rmsnorm_bwd(s, w, dy)
        q = gla.gla_rmsnorm_q8(s, w)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(q[0].float(), gla.gla_rmsnorm_q8(s, w)[0].float())
