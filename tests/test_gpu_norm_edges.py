"""The layer norm on the GPU at the ends of rows and of the number range."""
import pytest
import torch

from test_gpu_norm import HALF, U, _adds, _x

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("c", [5, 100, 104, 129, 200, 300, 301, 1000, 1003, 8200, 17000, 33001])
def test_backward_of_far_constant_rows(hip, c, dtype):
    """mean times rstd is beyond fp32, every x - mean is 0: the lanes behind a row's last
    column, which hold x = 0, must not bring the product in."""
    rows = 20
    x, dy = torch.full((rows, c), 2.0 ** 119, dtype=dtype), _x(rows, c, 5, dtype, 0.0)
    mean, rstd = torch.full((rows,), 2.0 ** 119), torch.full((rows,), 1000.0)
    x[::2], mean[::2] = -x[::2], -mean[::2]
    dx, dw, db = hip.layer_norm_backward(dy.cuda(), x.cuda(), mean.cuda(), rstd.cuda())
    # xhat = 0 exactly: dx = rstd (dy - mean(dy)), the mean off by its additions and a
    # division, then three roundings, one of them dx's own type
    d = dy.double()
    want = 1000 * (d - d.mean(1, keepdim=True))
    size = d.abs().mean(1, keepdim=True)
    tol = 1000 * ((_adds(c) + 2) * U * size + 3 * U * (d.abs() + size))
    half = HALF[dtype]
    err = (dx.double().cpu() - want).abs()
    assert bool((err <= tol * (1 + half) + half * want.abs()).all())
    assert bool((dw == 0).all())
    assert bool(((db.double().cpu() - d.sum(0)).abs() <= rows * U * d.abs().sum(0)).all())


@pytest.mark.parametrize("eps", [1e-46, 1e-60, 1e-45])
@pytest.mark.parametrize("c", [7, 300, 5120])
def test_forward_of_constant_rows_under_a_tiny_eps(hip, c, eps):
    """A positive eps below float's least is not 0: equal values give the bias, not NaN."""
    x, b = torch.full((3, c), 0.5, device="cuda"), torch.randn(c, device="cuda")
    y, mean, rstd = hip.layer_norm(x, torch.ones(c, device="cuda"), b, eps=eps)
    assert torch.equal(y, b.expand(3, c)) and bool((mean == 0.5).all())
    # the least float, 2^-149: its root is 2^-74.5
    assert bool(((rstd.double() - 2.0 ** 74.5).abs() <= 4 * U * 2.0 ** 74.5).all())
