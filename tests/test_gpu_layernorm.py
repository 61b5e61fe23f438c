"""Residual addition and layer norm, and its gradients, on the GPU against
their formulas in float64 and against differences.

Tolerances. A row's sums of D values are fp32 sums over threads, warps and a
tree: off by at most (D / threads + 10) 2^-24 relative to the sum of
magnitudes, under SUM = 1e-5 for D <= 8192; the other operations add a few
2^-24. The mean's own error, SUM mean|s|, moves every centred value: relative
to the row's deviation it is what a mean far from 0 costs any fp32 norm of a
rounded row, and enters the tolerances as SHIFT. Outputs add half a step."""
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


def rn(*shape, seed, dtype=FP, std=1.0, mean=0.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * std + mean).to(dtype).cuda()


def near(got, ref, mag, name):
    g = d(got)
    tol = half_step(got.dtype) * ref.abs() + SUM * mag + 1e-30
    assert g.shape == ref.shape and ((g - ref).abs() <= tol).all(), (name, float(((g - ref).abs() / tol).max()))


def formula(x, res, w, b, eps):
    """s, y, and the sum of magnitudes that bounds y's error (over SUM)."""
    s = d(x) + (0 if res is None else d(res))
    c = s - s.mean(-1, keepdim=True)
    sd = (c.square().mean(-1, keepdim=True) + eps).sqrt()
    w = torch.ones(s.shape[-1], dtype=F64) if w is None else d(w)
    y = c / sd * w + (0 if b is None else d(b))
    shift = s.abs().mean(-1, keepdim=True) / sd          # the mean's error in deviations
    mag = (1 + shift) * (w.abs() * (1 + c.abs() / sd)) + (0 if b is None else d(b).abs())
    return s, y, mag


SHAPES = [(BF, 1, 8), (BF, 3, 72), (FP, 2, 4), (FP, 5, 516), (BF, 700, 1032), (BF, 2, 4096), (FP, 33, 2048),
          (BF, 9, 8192), (FP, 3, 8192), (BF, 1100, 264), (BF, 700, 2048), (FP, 3, 8188), (BF, 400, 4104)]


@pytest.mark.parametrize("dtype,rows,D", SHAPES)
@pytest.mark.parametrize("with_res,with_wb", [(True, True), (False, False)])
def test_forward(gla, dtype, rows, D, with_res, with_wb):
    x, res = rn(rows, D, seed=1, dtype=dtype, mean=0.5), rn(rows, D, seed=2, dtype=dtype, std=3.0) if with_res else None
    w, b = (1 + rn(D, seed=3, std=0.2), rn(D, seed=4, std=0.3)) if with_wb else (None, None)
    y, s = gla.gla_layernorm(x, w, b, res, 1e-6)
    gla.gla_check()
    rs, ry, mag = formula(x, res, w, b, 1e-6)
    near(y, ry, mag, "y")
    assert (s is None) == (res is None)
    if with_res:
        near(s, rs, 0 * rs, "s")
        inplace = res.clone()
        y1, s1 = gla.gla_layernorm(x, w, b, inplace, 1e-6, s=inplace)
        gla.gla_check()
        assert s1 is inplace and torch.equal(s1, s) and torch.equal(y1, y)


def grads(s, w, dy, ds, eps):
    """dx, dw, db, and the sums of magnitudes that bound their errors."""
    s, dy = d(s), d(dy)
    D = s.shape[-1]
    w = torch.ones(D, dtype=F64) if w is None else d(w)
    c = s - s.mean(-1, keepdim=True)
    r = 1 / (c.square().mean(-1, keepdim=True) + eps).sqrt()
    n, g = c * r, dy * w
    dx = r * (g - g.mean(-1, keepdim=True) - n * (g * n).mean(-1, keepdim=True)) + (0 if ds is None else d(ds))
    shift = 1 + s.abs().mean(-1, keepdim=True) * r
    mag = r * shift * (2 * g.abs() + g.abs().mean(-1, keepdim=True) + 4 * (1 + n.abs()) * (g * n).abs().mean(-1, keepdim=True)
                       + 4 * n.abs() * g.abs().mean(-1, keepdim=True))
    if ds is not None:
        mag = mag + d(ds).abs()
    return dx, (dy * n).sum(0), dy.sum(0), mag, (dy.abs() * (n.abs() + 1) * shift).sum(0), dy.abs().sum(0)


@pytest.mark.parametrize("dtype,rows,D", SHAPES)
@pytest.mark.parametrize("with_ds,with_w", [(True, True), (False, False)])
def test_gradients(gla, dtype, rows, D, with_ds, with_w):
    s, dy = rn(rows, D, seed=5, dtype=dtype, std=2.0, mean=-0.7), rn(rows, D, seed=6, dtype=dtype)
    ds = rn(rows, D, seed=7, dtype=dtype) if with_ds else None
    w = 1 + rn(D, seed=8, std=0.2) if with_w else None
    dx, dw, db = gla.gla_layernorm_bwd(s, w, dy, ds, 1e-6)
    gla.gla_check()
    rx, rw, rb, mx, mw, mb = grads(s, w, dy, ds, 1e-6)
    near(dx, rx, mx, "dx")
    near(dw, rw, mw, "dw")      # rows / CTAs, then up to 1,216 partial sums: (rows / 1216 + 80) 2^-24 stays under SUM
    near(db, rb, mb, "db")
    again = gla.gla_layernorm_bwd(s, w, dy, ds, 1e-6)
    assert all(torch.equal(a, b) for a, b in zip((dx, dw, db), again))
    inplace = dy.clone()
    only, none, _ = gla.gla_layernorm_bwd(s, w, inplace, ds, 1e-6, dx=inplace, want_dw=False, want_db=False)
    assert none is None and torch.equal(only, dx)
    assert torch.equal(gla.gla_layernorm_bwd(s, w, dy, ds, 1e-6, want_dw=False)[2], db)
    assert torch.equal(gla.gla_layernorm_bwd(s, w, dy, ds, 1e-6, want_db=False)[1], dw)
    gla.gla_check()


def test_gradients_against_differences(gla):
    """Central differences of <dy, y> + <ds, s> over the formula in float64."""
    rows, D, eps = 3, 20, 1e-3
    s, dy, ds, w = (rn(rows, D, seed=i) for i in (1, 2, 3, 4))
    w = w[0].contiguous()
    dx, dw, db = gla.gla_layernorm_bwd(s, w, dy, ds, eps)

    def loss(s, w, b):
        c = s - s.mean(-1, keepdim=True)
        y = c / (c.square().mean(-1, keepdim=True) + eps).sqrt() * w + b
        return float((d(dy) * y).sum() + (d(ds) * s).sum())

    at, h = [d(s), d(w), torch.zeros(D, dtype=F64)], 1e-5
    for got, which in ((dx, 0), (dw, 1), (db, 2)):
        flat = d(got).reshape(-1)
        for i in range(flat.numel()):
            up, down = ([t.clone() for t in at] for _ in range(2))
            up[which].view(-1)[i] += h
            down[which].view(-1)[i] -= h
            # the difference is off by h^2 times a third derivative: well under 1e-6; the kernel by SUM of O(10) magnitudes
            assert abs((loss(*up) - loss(*down)) / (2 * h) - float(flat[i])) < 3e-4


def test_a_mean_far_from_zero(gla):
    """Rows of 1000 +- 1 in fp32: the variance is that of the centred values."""
    x = rn(64, 2048, seed=11, mean=1000.0)
    y, _ = gla.gla_layernorm(x)
    s, ry, mag = formula(x, None, None, None, 1e-6)
    near(y, ry, mag, "y")                                  # mag holds the shift of 1000 deviations: 1e-2
    assert abs(float(d(y).square().mean()) - 1) < 1e-4     # squared deviations alone: no cancellation
    gla.gla_check()


@pytest.mark.parametrize("dtype", [BF, FP])
def test_rows_are_independent(gla, dtype):
    x, dy, ds = (rn(900, 264, seed=i, dtype=dtype) for i in (1, 2, 3))
    y, _ = gla.gla_layernorm(x)
    dx, _, _ = gla.gla_layernorm_bwd(x, None, dy, ds)
    x2 = x.clone()
    x2[::7] = float("nan")
    x2[3] = float("inf")
    keep = torch.ones(900, dtype=torch.bool)
    keep[::7] = False
    keep[3] = False
    y2, _ = gla.gla_layernorm(x2)
    dx2, _, _ = gla.gla_layernorm_bwd(x2, None, dy, ds)
    assert torch.equal(y2[keep], y[keep]) and torch.equal(dx2[keep], dx[keep])
    assert y2[~keep].isnan().all()
    gla.gla_check()


def test_constant_rows(gla):
    """No deviation: y is b, and eps = 0 is as the formula, 0 / 0."""
    x, b = torch.full((4, 264), 3.0, device="cuda"), rn(264, seed=1)
    y, _ = gla.gla_layernorm(x, None, b, eps=1e-6)
    assert torch.equal(y, b.expand(4, -1))
    assert gla.gla_layernorm(x, eps=0.0)[0].isnan().all()
    gla.gla_check()


@pytest.mark.parametrize("rows,D,dtype", [(5000, 2048, BF), (3000, 516, FP), (40000, 72, BF), (1000, 8192, FP)])
def test_many_rows_a_cta(gla, rows, D, dtype):
    s, dy, ds, w = rn(rows, D, seed=1, dtype=dtype), rn(rows, D, seed=2, dtype=dtype), rn(rows, D, seed=3, dtype=dtype), 1 + rn(D, seed=4, std=0.1)
    y, out = gla.gla_layernorm(s, w, w, ds, 1e-6)
    rs, ry, mag = formula(s, ds, w, w, 1e-6)
    near(y, ry, mag, "y")
    near(out, rs, 0 * rs, "s")
    dx, dw, db = gla.gla_layernorm_bwd(s, w, dy, ds, 1e-6)
    rx, rw, rb, mx, mw, mb = grads(s, w, dy, ds, 1e-6)
    near(dx, rx, mx, "dx")
    near(dw, rw, mw, "dw")
    near(db, rb, mb, "db")
    gla.gla_check()


def test_more_elements_than_32_bits(gla):
    rows = (1 << 31) // 4096 + 3
    x = torch.zeros(rows, 4096, dtype=BF, device="cuda")
    x[-2:] = rn(2, 4096, seed=1, dtype=BF)
    y, _ = gla.gla_layernorm(x)
    _, ry, mag = formula(x[-2:], None, None, None, 1e-6)
    near(y[-2:], ry, mag, "y")
    del y
    dy = torch.zeros_like(x)
    dy[-2:] = rn(2, 4096, seed=2, dtype=BF)
    dx, dw, db = gla.gla_layernorm_bwd(x, None, dy)
    rx, rw, rb, mx, mw, mb = grads(x[-2:], None, dy[-2:], None, 1e-6)
    near(dx[-2:], rx, mx, "dx")
    near(dw, rw, mw, "dw")
    near(db, rb, mb, "db")
    gla.gla_check()


def test_captured_beside_eager_calls_and_on_a_stream(gla):
    """A captured training pass and an eager one on the same leaves, each with its own workspace."""
    s, dy, w = rn(300, 1032, seed=1, dtype=BF), rn(300, 1032, seed=2, dtype=BF), 1 + rn(1032, seed=3, std=0.1)
    want = gla.gla_layernorm_bwd(s, w, dy)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, _ = gla.gla_layernorm(s, w)
        got = gla.gla_layernorm_bwd(s, w, dy)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        for t in got:
            t.fill_(7.0)
        side.wait_stream(torch.cuda.current_stream())
        graph.replay()
        other = gla.gla_layernorm_bwd(s, w, dy, stream=side)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(want, got, other))
    gla.gla_check()


def test_no_rows_and_refusals(gla):
    x = torch.zeros(0, 64, dtype=BF, device="cuda")
    assert gla.gla_layernorm(x)[0].shape == (0, 64)
    dw, db = (torch.full((64,), 7.0, device="cuda") for _ in range(2))
    gla.gla_layernorm_bwd(x, None, x, dw=dw, db=db)
    assert not dw.any() and not db.any()
    s = rn(4, 64, seed=1, dtype=BF)
    for f in (lambda: gla.gla_layernorm(s[:, :60].contiguous()), lambda: gla.gla_layernorm(s, y=s),
              lambda: gla.gla_layernorm(s, w=s[0]), lambda: gla.gla_layernorm(s, res=s[:3]),
              lambda: gla.gla_layernorm(s.t()), lambda: gla.gla_layernorm(s, eps=-1.0),
              lambda: gla.gla_layernorm(s.cpu()), lambda: gla.gla_layernorm(s.half()),
              lambda: gla.gla_layernorm(torch.zeros(2, 8200, dtype=BF, device="cuda")),
              lambda: gla.gla_layernorm_bwd(s, None, s, dx=s), lambda: gla.gla_layernorm_bwd(s, None, s.float()),
              lambda: gla.gla_layernorm_bwd(s, None, s, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(gla.GlaError):
            f()
    gla.gla_check()
