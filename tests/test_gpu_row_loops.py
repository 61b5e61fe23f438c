"""Calls whose CTAs take several turns: the norm and its gradients with more
rows than CTAs (the next rows on their way, the sums' two buffers, in place
too), the Conv1d's gradients with tiles of many tokens."""
import pytest
import torch

import test_gpu_conv_bwd as conv
import test_gpu_norm as norm
from ssm_plain import d, half_step
from test_gpu_norm import BF, FP, gla  # noqa: F401

pytestmark = pytest.mark.gpu


# -------------------------------------------------------------------- norm
MANY = [(BF, 3001, 2048), (FP, 500, 8192), (FP, 4001, 1028), (BF, 5003, 264), (BF, 603, 8192)]


@pytest.mark.parametrize("dtype,rows,D", MANY)
@pytest.mark.parametrize("with_res,with_w", [(True, True), (False, False)])
def test_norm_of_many_rows(gla, dtype, rows, D, with_res, with_w):  # noqa: F811
    norm.test_forward(gla, dtype, rows, D, with_res, with_w)          # in place too


@pytest.mark.parametrize("dtype,rows,D", MANY)
@pytest.mark.parametrize("group", [0, 128])
def test_eight_bit_norm_of_many_rows(gla, dtype, rows, D, group):  # noqa: F811
    norm.test_eight_bit_output(gla, dtype, rows, D, group)
    x, res, w = norm.rn(rows, D, seed=4, dtype=dtype), norm.rn(rows, D, seed=5, dtype=dtype), 1 + norm.rn(D, seed=6, std=0.2)
    y8, scale, s = gla.gla_rmsnorm_q8(x, w, res, 1e-6, group)
    inplace = res.clone()
    y1, scale1, s1 = gla.gla_rmsnorm_q8(x, w, inplace, 1e-6, group, s=inplace)
    gla.gla_check()
    assert s1 is inplace and torch.equal(s1, s) and torch.equal(scale1, scale)
    assert torch.equal(y1.view(torch.uint8), y8.view(torch.uint8))


@pytest.mark.parametrize("dtype,rows,D", MANY)
def test_norm_gradients_of_many_rows(gla, dtype, rows, D):  # noqa: F811
    norm.test_backward_is_the_formula_s(gla, dtype, rows, D, True, True)


# --------------------------------------------------------- Conv1d gradients
@pytest.mark.parametrize("B,T,D", [(600, 301, 16), (10000, 40, 8), (200, 333, 72), (1200, 700, 8), (1000, 270, 16)])
@pytest.mark.parametrize("dtype,window,bias", [(BF, True, True), (FP, False, True), (FP, True, False)])
def test_conv_gradients_over_long_tiles(gla, B, T, D, dtype, window, bias):  # noqa: F811
    """The sums of dw and db run over a tile's tokens in one accumulator (one of
    two in a pair), then over the tiles (the second stage: a lane adds every
    64th tile in eight accumulators, then a tree and the CTA's 16 warps): at
    most (tile + B tiles / 512 + 40) 2^-24 relative to the sum of magnitudes,
    and 2e-6 of each term's own (see test_gpu_conv_bwd)."""
    a = conv.make(B, T, D, dtype, 20 + T, window, bias)
    got = gla.gla_conv1d_bwd(*a)
    gla.gla_check()
    code = gla.GLA_BF16 if dtype == BF else gla.GLA_FP32
    tiles = gla.gla_conv1d_bwd_workspace_size(B, T, D, code) // (B * 5 * D * 4)
    assert tiles < -(-T // 16) or T <= 40                   # longer than the least tile
    many = min(-(-T // tiles) + 4, T) + B * tiles / 512 + 40   # (a tile is a multiple of four tokens)
    ref, mag = conv.formula(*a)
    for name, v, r, m, k in zip(("dx", "dw", "db"), got, ref, mag, (4e-6,) + (many * 2.0 ** -24 + 2e-6,) * 2):
        tol = half_step(v.dtype) * r.abs() + k * m + 1e-30
        assert d(v).shape == r.shape and ((d(v) - r).abs() <= tol).all(), (name, float(((d(v) - r).abs() / tol).max()))
    again = gla.gla_conv1d_bwd(*a)
    assert all(torch.equal(u, v) for u, v in zip(got, again))
