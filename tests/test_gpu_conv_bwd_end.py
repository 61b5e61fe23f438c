"""The Conv1d's gradients at a sequence's end where a filter sum that no token
has would overflow: a large last input times a large early tap belongs to a
token behind the end, and nothing of that token reaches a gradient."""
import pytest
import torch

from test_gpu_conv_bwd import BF, FP, check, formula, gla  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("T", [3, 5, 18, 64])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_a_sum_behind_the_end_that_overflows_leaves_the_gradients_finite(gla, dtype, T, sign):  # noqa: F811
    g = torch.Generator().manual_seed(T)
    D = 16
    x = torch.randn(1, T, D, generator=g).to(dtype).cuda()
    x[0, T - 3] = sign * 2e38                               # times tap 0: past the largest float, at token T
    w = torch.tensor([2.0, 1e-3, 1e-3, 1e-3]).repeat(D, 1).cuda()
    dy = (torch.randn(1, T, D, generator=g) * 1e-3).to(dtype).cuda()
    got = gla.gla_conv1d_bwd(x, w, None, dy)
    gla.gla_check()
    ref, mag = formula(x, w, None, dy, None)
    assert all(torch.isfinite(v).all() for v in ref)
    assert all(torch.isfinite(v).all() for v in got), [int((~torch.isfinite(v)).sum()) for v in got]
    check(got, ref, mag)
