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


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,c", [(9, 192), (9, 1024), (2100, 5120), (5, 16448)])
def test_quantizing_forms_of_rows_that_are_not_finite(hip, rows, c, dtype):
    """NaN and infinities stay in their rows; the codes are those of the two calls."""
    x, w, b = _x(rows, c, 1, dtype).cuda(), torch.ones(c, device="cuda"), torch.zeros(c, device="cuda")
    want = hip.layer_norm(x, w, b)[0]
    x[1, 3], x[3, c - 1], x[rows - 1, 0] = float("nan"), float("inf"), -float("inf")
    y = hip.layer_norm(x, w, b)[0]
    good = torch.ones(rows, dtype=torch.bool, device="cuda")
    good[[1, 3, rows - 1]] = False
    assert torch.equal(y[good], want[good]) and bool(torch.isnan(y[~good]).all())
    # (HiF4 codes of values that are not finite are unspecified)
    for got, two, at in ((hip.layer_norm_quantize(x, w, b)[:2], hip.quantize(y.to(torch.bfloat16))[:2], good),
                         (hip.layer_norm_quantize_fp8(x, w, b), hip.quantize_fp8(y), torch.ones_like(good))):
        for g, r in zip(got, two):
            assert torch.equal(g.contiguous().view(torch.uint8)[at], r.contiguous().view(torch.uint8)[at])
    # the backward: dx of those rows is NaN, of the others as before
    x[~good] = 0.5
    dy = _x(rows, c, 2, dtype, 0.0).cuda()
    _, mean, rstd = hip.layer_norm(x)
    dx = hip.layer_norm_backward(dy, x, mean, rstd, weight=w)[0]
    dy[1, 5] = float("nan")
    again = hip.layer_norm_backward(dy, x, mean, rstd, weight=w)[0]
    keep = torch.arange(rows, device="cuda") != 1
    assert torch.equal(again[keep], dx[keep]) and bool(torch.isnan(again[1]).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,c", [(513, 1003), (2051, 5120), (70001, 128), (1027, 250), (515, 16400)])
def test_in_place_over_many_rows(hip, rows, c, dtype):
    """Rows that a workgroup reads again at the end are not taken from what it has written."""
    x, w = _x(rows, c, 3, dtype).cuda(), torch.full((c,), 1.5, device="cuda")
    y, mean, rstd = hip.layer_norm(x, w)
    z = x.clone()
    _, m2, r2 = hip.layer_norm(z, w, y=z)
    assert torch.equal(z, y) and torch.equal(m2, mean) and torch.equal(r2, rstd)


@pytest.mark.parametrize("rows,c", [(270001, 8192), (16800001, 128)])
def test_offsets_beyond_32_bits(hip, rows, c):
    """The last rows of more than 2^31 elements, both ways and into the quantizers."""
    x = torch.zeros((rows, c), dtype=torch.bfloat16, device="cuda")
    last = _x(40, c, 4).cuda()
    x[-40:] = last
    w = torch.full((c,), 1.25, device="cuda")
    y, mean, rstd = hip.layer_norm(x, w)
    y2, m2, r2 = hip.layer_norm(last, w)
    assert torch.equal(y[-40:], y2) and torch.equal(mean[-40:], m2) and torch.equal(rstd[-40:], r2)
    assert not bool(y[:-40].view(torch.int32).any())
    del y
    codes, scales = hip.layer_norm_quantize_fp8(x, w)
    c2, s2 = hip.layer_norm_quantize_fp8(last, w)
    assert torch.equal(codes[-40:].view(torch.uint8), c2.view(torch.uint8))
    assert torch.equal(scales[-40:].view(torch.uint8), s2.view(torch.uint8))
    del codes, scales
    dx, dw, db = hip.layer_norm_backward(x, x, mean, rstd, weight=w)
    d2, w2, b2 = hip.layer_norm_backward(last, last, m2, r2, weight=w)
    assert torch.equal(dx[-40:], d2) and not bool(dx[:-40].view(torch.int32).any())
    # the same terms added in another order: at most 40 additions that round each
    xhat = (last.double() - m2.double()[:, None]) * r2.double()[:, None]
    assert bool(((dw - w2).double().abs() <= 80 * U * (last.double() * xhat).abs().sum(0)).all())
    assert bool(((db - b2).double().abs() <= 80 * U * last.double().abs().sum(0)).all())
