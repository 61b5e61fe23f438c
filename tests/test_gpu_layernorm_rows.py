"""Residual addition, layer norm and its gradients in every configuration of
threads, vectors and rows in flight, with many rows a CTA. The bounds are
test_gpu_layernorm.py's. A channel's dw and db add up rows / CTAs values in a
CTA, then the partial sums of up to 16 CTAs an SM (2,432 at 152 SMs) in eight
chains of 16 groups and 24 additions behind them, a few units a product: at
most 17 + 2432 / 128 + 30 units of 2^-24 for the rows here, 4e-6, under SUM."""
import pytest
import torch

from test_gpu_layernorm import BF, FP, formula, gla, grads, near, rn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,D,dtype", [
    (40000, 72, FP), (9000, 252, FP), (9000, 256, BF), (9000, 256, FP), (20000, 4, FP), (20000, 8, BF),     # a vector a thread, rows of a warp
    (1000, 5000, FP), (1000, 6144, BF), (1000, 6144, FP), (1000, 4104, BF), (700, 5000, BF),                # at most 384 threads
    (300, 4096, BF), (300, 4096, FP), (304, 2056, BF), (200, 4096, FP), (305, 4096, BF),                    # few and wide rows, one vector a thread
    (2000, 2568, BF), (2000, 2572, FP), (900, 2052, FP), (1500, 260, FP), (3000, 1028, FP), (620, 8188, FP)])
@pytest.mark.parametrize("joined", [True, False])
def test_rows_in_flight(gla, rows, D, dtype, joined):
    s, dy, w = rn(rows, D, seed=1, dtype=dtype, std=2.0, mean=0.3), rn(rows, D, seed=2, dtype=dtype), 1 + rn(D, seed=4, std=0.1)
    ds = rn(rows, D, seed=3, dtype=dtype) if joined else None
    y, out = gla.gla_layernorm(s, w, w, ds, 1e-6)
    gla.gla_check()
    rs, ry, mag = formula(s, ds, w, w, 1e-6)
    near(y, ry, mag, "y")
    if joined:
        near(out, rs, 0 * rs, "s")
    dx, dw, db = gla.gla_layernorm_bwd(s, w, dy, ds, 1e-6)
    gla.gla_check()
    rx, rw, rb, mx, mw, mb = grads(s, w, dy, ds, 1e-6)
    near(dx, rx, mx, "dx")
    near(dw, rw, mw, "dw")
    near(db, rb, mb, "db")
