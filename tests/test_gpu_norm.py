"""The layer norm on the GPU against 64-bit references, its quantizing forms
against the two calls in turn, and the operators run together."""
import pytest
import torch

import ref64

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
EPS = 1e-6


def _x(rows, c, seed=0, dtype=torch.bfloat16, offset=0.1):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, c), generator=g) * torch.exp(0.7 * torch.randn((1, c), generator=g)) + offset
    return x.to(dtype)


def _affine(c, dtype, seed=1):
    if dtype is None:
        return None, None
    g = torch.Generator().manual_seed(seed)
    return ((1 + 0.3 * torch.randn((c,), generator=g)).to(dtype), (0.3 * torch.randn((c,), generator=g)).to(dtype))


def _cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


def _adds(c):
    """Rounded additions on the way to one sum over a row: at most 64 elements in
    a lane (two at a time are added first), 6 steps of a wave, 16 waves."""
    return min(c, 64 + 16) + 6 + 16


def _check_forward(x, w, b, y, mean, rstd, half):
    """Sums of A rounded additions: |d mean| <= (A + 2) U max|x|; var is off by
    (A + 4) U of itself and by (d mean)^2; rstd by half of that and 4 roundings;
    each of y's factors rounds once more."""
    want, m, r = ref64.layer_norm(x, w, b, EPS)
    c = x.shape[1]
    xd = x.double()
    dm = (_adds(c) + 2) * U * xd.abs().amax(1)
    rel = (_adds(c) / 2 + 8) * U + (dm * r) ** 2
    if mean is not None:
        assert bool(((mean.double().cpu() - m).abs() <= dm).all())
        # each deviation is off by dm and a rounding of itself
        assert bool(((rstd.double().cpu() - r).abs() <= r * (rel + 2 * U + dm * r * U)).all())
    xhat = (xd - m[:, None]).abs() * r[:, None]
    wa = torch.ones(c) if w is None else w.abs().double()
    ba = torch.zeros(c) if b is None else b.abs().double()
    tol = wa * (r[:, None] * dm[:, None] + xhat * (rel[:, None] + 4 * U)) + U * (wa * xhat + ba)
    tol = tol * (1 + half) + half * want.abs()
    err = (y.double().cpu() - want).abs()
    assert bool((err <= tol).all()), (x.shape, float((err - tol).max()))


CS = [1, 2, 7, 8, 63, 64, 200, 1003, 1024, 1025, 2048, 3000, 5120, 8192, 8200, 13824, 16400]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("c", CS)
def test_forward(hip, c, dtype):
    for rows, wd, seed in ((1, torch.float32, 1), (5, None, 2), (67, torch.bfloat16, 3)):
        x = _x(rows, c, seed, dtype)
        w, b = _affine(c, wd)
        y, mean, rstd = hip.layer_norm(*_cuda(x, w, b), eps=EPS)
        assert y.dtype == dtype
        _check_forward(x, w, b, y, mean, rstd, HALF[dtype])


@pytest.mark.parametrize("offset", [0.0, 100.0, -3000.0])
def test_forward_far_mean(hip, offset):
    """A mean far above the spread: the variance comes from the deviations."""
    x = _x(9, 1000, 4, torch.float32, offset=offset)
    y, mean, rstd = hip.layer_norm(x.cuda(), eps=EPS)
    _check_forward(x, None, None, y, mean, rstd, HALF[torch.float32])


def test_forward_constant_and_special_rows(hip):
    x = _x(8, 300, 5, torch.float32)
    x[1] = 0.0
    x[2] = 0.5
    x[3, 7] = float("nan")
    x[4, 7] = float("inf")
    y, mean, rstd = hip.layer_norm(x.cuda(), eps=EPS)
    y = y.cpu()
    assert bool((y[1] == 0).all()) and bool((y[2].abs() <= 1e-3).all())
    assert abs(float(rstd[1]) - EPS ** -0.5) <= 4 * U * EPS ** -0.5 + 1e-7 * EPS ** -0.5
    assert bool(torch.isnan(y[3]).all()) and bool(torch.isnan(y[4]).all())
    good = [0, 5, 6, 7]
    _check_forward(x[good], None, None, y[good], None, None, HALF[torch.float32])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("ld,offset", [(1032, 0), (1003, 0), (1031, 3), (1032, 8)])
def test_forward_strides_and_surroundings(hip, ld, offset, dtype):
    rows, c = 13, 1003
    x = _x(rows, c, 6, dtype)
    w, b = _affine(c, torch.float32)
    full = torch.full((rows * ld + offset + 8,), 5.0, dtype=dtype, device="cuda")
    xv = full[offset:offset + rows * ld].view(rows, ld)[:, :c]
    xv.copy_(x)
    out = torch.full((rows + 2, ld), 7.0, dtype=dtype, device="cuda")
    y, mean, rstd = hip.layer_norm(xv, *_cuda(w, b), eps=EPS, y=out[1:-1, :c])
    _check_forward(x, w, b, y, mean, rstd, HALF[dtype])
    assert bool((out[[0, -1]] == 7).all()) and bool((out[:, c:] == 7).all())
    hip.layer_norm(xv, *_cuda(w, b), eps=EPS, y=xv)  # in place
    assert torch.equal(xv, y)
    # weights at odd addresses
    wb = torch.zeros(c + 1, device="cuda")
    wb[1:] = w.cuda()
    y2, _, _ = hip.layer_norm(x.cuda(), wb[1:], b.cuda(), eps=EPS)
    assert torch.equal(y2, y)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("c", [30001, 65535, 65536])
def test_widest_rows(hip, c, dtype):
    x, (w, b) = _x(3, c, c, dtype), _affine(c, torch.float32)
    xd, wd, bd = _cuda(x, w, b)
    y, mean, rstd = hip.layer_norm(xd, wd, bd, eps=EPS)
    _check_forward(x, w, b, y, mean, rstd, HALF[dtype])
    got, want = hip.layer_norm_quantize_fp8(xd, wd, bd, eps=EPS), hip.quantize_fp8(y)
    if c % 64 == 0:
        got = (*got, *hip.layer_norm_quantize(xd, wd, bd, eps=EPS)[:2])
        want = (*want, *hip.quantize(y.to(torch.bfloat16))[:2])
    for g, r in zip(got, want):
        assert torch.equal(g.contiguous().view(torch.uint8), r.contiguous().view(torch.uint8))
    dy = _x(3, c, c + 1, dtype, offset=0.0)
    dx, dw, db = hip.layer_norm_backward(dy.cuda(), xd, mean, rstd, weight=wd)
    _check_backward(dy, x, mean.cpu(), rstd.cpu(), w, dx, dw, db)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows", [511, 512, 513, 2051])
@pytest.mark.parametrize("c", [5, 9, 127, 128, 130, 256, 500, 512, 1003, 1024, 4104, 5119])
def test_forward_rows_at_once(hip, c, rows, dtype):
    """Workgroups that take two rows, the last of them one."""
    x, (w, b) = _x(rows, c, rows, dtype), _affine(c, torch.bfloat16)
    y, mean, rstd = hip.layer_norm(*_cuda(x, w, b), eps=EPS)
    _check_forward(x, w, b, y, mean, rstd, HALF[dtype])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("c", [64, 192, 1024, 1088, 2048, 5120, 8192, 13824, 16448])
def test_quantizing_forms_are_the_two_calls(hip, c, dtype):
    for rows, wd in ((1, None), (70, torch.float32)):
        x, w, b = _cuda(_x(rows, c, c, dtype), *_affine(c, wd))
        y, _, _ = hip.layer_norm(x, w, b, eps=EPS)
        yb = y if dtype == torch.bfloat16 else None
        codes, meta, _ = hip.layer_norm_quantize(x, w, b, eps=EPS)
        if yb is None:  # rounded to bf16 from the same fp32 value that y holds
            yb = y.to(torch.bfloat16)
        want = hip.quantize(yb)
        assert torch.equal(codes, want[0]) and torch.equal(meta, want[1])
        for n_mask in (0, 1, c // 3, c):
            mask = torch.zeros(c, dtype=torch.uint8, device="cuda")
            mask[torch.randperm(c, generator=torch.Generator().manual_seed(c))[:n_mask].cuda()] = 1
            got = hip.layer_norm_quantize(x, w, b, eps=EPS, mask=mask)
            want = hip.quantize(yb, mask=mask)
            for g, r in zip(got, want):
                assert torch.equal(g, r)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("c", [1, 100, 128, 1000, 1024, 1030, 5120, 8190, 13824, 16400])
def test_fp8_form_is_the_two_calls(hip, c, dtype):
    for rows, wd in ((1, None), (70, torch.bfloat16)):
        x, w, b = _cuda(_x(rows, c, c, dtype), *_affine(c, wd))
        y, _, _ = hip.layer_norm(x, w, b, eps=EPS)
        want, ws = hip.quantize_fp8(y)
        got, gs = hip.layer_norm_quantize_fp8(x, w, b, eps=EPS)
        assert torch.equal(got.view(torch.uint8), want.view(torch.uint8))
        assert torch.equal(gs.contiguous().view(torch.uint8), ws.contiguous().view(torch.uint8))


@pytest.mark.parametrize("c", [64, 128, 192, 256, 448, 512, 576, 1024, 1088, 2048, 3136, 4096, 4160, 5120, 5184, 6144, 6208, 8192, 13824])
def test_quantizing_forms_are_the_two_calls_over_many_rows(hip, c):
    rows = 2100 if c > 4096 else 8200
    x, w, b = _cuda(_x(rows, c, c), *_affine(c, torch.float32))
    y, _, _ = hip.layer_norm(x, w, b, eps=EPS)
    mask = torch.zeros(c, dtype=torch.uint8, device="cuda")
    mask[torch.randperm(c, generator=torch.Generator().manual_seed(c))[:c // 50].cuda()] = 1
    for got, want in ((hip.layer_norm_quantize(x, w, b, eps=EPS, mask=mask), hip.quantize(y, mask=mask)),
                      (hip.layer_norm_quantize(x, w, b, eps=EPS)[:2], hip.quantize(y)[:2]),
                      (hip.layer_norm_quantize_fp8(x, w, b, eps=EPS), hip.quantize_fp8(y))):
        for g, r in zip(got, want):
            assert torch.equal(g.contiguous().view(torch.uint8), r.contiguous().view(torch.uint8))
    pick = torch.tensor([0, 1, 7, 1000, rows - 2, rows - 1])
    _check_forward(x.cpu()[pick], w.cpu(), b.cpu(), y[pick.cuda()], None, None, HALF[torch.bfloat16])


def _check_backward(dy, x, mean, rstd, w, dx, dw, db):
    """mean and rstd are inputs. A row's two means are off by (A + 4) U of the mean
    of absolute terms (xhat and g round, too); dx adds four roundings of its terms.
    dw and db add at most rows products, xhat off by 2 U."""
    wx, ww, wb = ref64.layer_norm_backward(dy, x, mean, rstd, w)
    rows, c = x.shape
    xhat = ((x.double() - mean.double()[:, None]) * rstd.double()[:, None]).abs()
    # x - mean rounds by U of the larger of the two before the difference
    dev = U * (x.double().abs() + mean.double().abs()[:, None]) * rstd.double()[:, None] + 2 * U * xhat
    g = dy.double().abs() * (1 if w is None else w.double().abs())
    a = _adds(c) + 4
    r = rstd.double()[:, None]
    m1, m2 = g.mean(1, keepdim=True), (g * xhat).mean(1, keepdim=True)
    tol = r * (a * U * (m1 + xhat * m2) + dev * m2 + xhat * (g * dev).mean(1, keepdim=True)
               + 5 * U * (g + m1 + xhat * m2))
    half = HALF[x.dtype]
    err = (dx.double().cpu() - wx).abs()
    assert bool((err <= tol * (1 + half) + half * wx.abs()).all()), (x.shape, float((err - tol).max()))
    if dw is not None:
        hw = HALF[dw.dtype]
        d = dy.double().abs()
        tw = (rows + 2) * U * (d * xhat).sum(0) + (d * dev).sum(0)
        tb = rows * U * d.sum(0)
        assert bool(((dw.double().cpu() - ww).abs() <= tw * (1 + hw) + hw * ww.abs()).all())
        assert bool(((db.double().cpu() - wb).abs() <= tb * (1 + hw) + hw * wb.abs()).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("c", CS + [20000])
def test_backward(hip, c, dtype):
    for rows, wd, seed in ((1, torch.float32, 1), (5, None, 2), (67, torch.bfloat16, 3), (1100, torch.float32, 4)):
        if rows * c > 6_000_000:
            rows = 523
        x, dy = _x(rows, c, seed, dtype), _x(rows, c, seed + 50, dtype, offset=0.0)
        w, _ = _affine(c, wd)
        xc, dyc, wc = _cuda(x, dy, w)
        _, mean, rstd = hip.layer_norm(xc, wc, None, eps=EPS)
        dx, dw, db = hip.layer_norm_backward(dyc, xc, mean, rstd, weight=wc)
        assert dw.dtype == (wd or torch.float32)
        _check_backward(dy, x, mean.cpu(), rstd.cpu(), w, dx, dw, db)
        again = hip.layer_norm_backward(dyc, xc, mean, rstd, weight=wc)
        assert all(torch.equal(p, q) for p, q in zip((dx, dw, db), again))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("c", [3, 8, 100, 128, 129, 250, 256, 257])
@pytest.mark.parametrize("rows", [15, 17, 1025, 9001])
def test_backward_narrow_rows(hip, rows, c, dtype):
    x, dy = _x(rows, c, c, dtype), _x(rows, c, c + 50, dtype, offset=0.0)
    w, _ = _affine(c, torch.float32)
    xc, dyc, wc = _cuda(x, dy, w)
    _, mean, rstd = hip.layer_norm(xc, wc, None, eps=EPS)
    dx, dw, db = hip.layer_norm_backward(dyc, xc, mean, rstd, weight=wc)
    _check_backward(dy, x, mean.cpu(), rstd.cpu(), w, dx, dw, db)


def test_backward_strides(hip):
    rows, c = 41, 1003
    x, dy = _x(rows, c, 1, torch.float32), _x(rows, c, 2, torch.float32, 0.0)
    fx = torch.zeros((rows, 1032), device="cuda")
    fd = torch.zeros((rows, 1005), device="cuda")
    fx[:, :c], fd[:, 1:c + 1] = x.cuda(), dy.cuda()
    _, mean, rstd = hip.layer_norm(x.cuda())
    out = hip.layer_norm_backward(fd[:, 1:c + 1], fx[:, :c], mean, rstd)
    _check_backward(dy, x, mean.cpu(), rstd.cpu(), None, *out)


def test_backward_no_rows(hip):
    e = torch.empty((0, 300), device="cuda")
    z = torch.empty((0,), device="cuda")
    dx, dw, db = hip.layer_norm_backward(e, e, z, z, weight=torch.ones(300, device="cuda"))
    assert dx.shape == (0, 300) and bool((dw == 0).all()) and bool((db == 0).all())


def test_backward_against_differences(hip):
    """Central differences of the 64-bit forward (truncation O(h^2))."""
    rows, c = 7, 96
    g = torch.Generator().manual_seed(3)
    x, dy = _x(rows, c, 8, torch.float32), torch.randn((rows, c), generator=g)
    w, b = _affine(c, torch.float32)
    xc, dyc, wc, bc = _cuda(x, dy, w, b)
    _, mean, rstd = hip.layer_norm(xc, wc, bc, eps=EPS)
    dx, dw, db = (t.double().cpu() for t in hip.layer_norm_backward(dyc, xc, mean, rstd, weight=wc))

    def loss(a, ww, bb):
        return float((ref64.layer_norm(a, ww, bb, EPS)[0] * dy.double()).sum())

    h = 1e-4
    x, w, b = x.double(), w.double(), b.double()
    for _ in range(4):
        v = torch.randn(x.shape, generator=g).double()
        q, s = torch.randn(c, generator=g).double(), torch.randn(c, generator=g).double()
        want = (loss(x + h * v, w + h * q, b + h * s) - loss(x - h * v, w - h * q, b - h * s)) / (2 * h)
        got = float((dx * v).sum() + (dw * q).sum() + (db * s).sum())
        # fp32 gradients: 100 U of the absolute terms; truncation h^2 times a third
        # derivative of order (rows c)
        size = float((dx * v).abs().sum() + (dw * q).abs().sum() + (db * s).abs().sum())
        assert abs(got - want) <= 100 * U * size + h * h * rows * c


# ---------------------------------------------------------------- together


def test_norm_into_w4a4_linear(hip):
    """The norm's HiF4 codes and kept channels feed linear_w4a4 as they are."""
    m, k, n = 100, 640, 130
    x, w, b = _cuda(_x(m, k, 1), *_affine(k, torch.float32))
    wt = (0.02 * _x(n, k, 2)).cuda()
    mask = torch.zeros(k, dtype=torch.uint8, device="cuda")
    mask[::29] = 1
    wc, wm, wk = hip.quantize(wt, mask)
    codes, meta, kept = hip.layer_norm_quantize(x, w, b, mask=mask)
    y = hip.linear_w4a4(wc, wm, x_codes=codes, x_meta=meta, x_kept=kept, w_kept=wk)
    h, _, _ = hip.layer_norm(x, w, b)
    assert torch.equal(y, hip.linear_w4a4(wc, wm, x=h, mask=mask, w_kept=wk))


def _step(hip, x, w, b, wq, wtq, dy):
    """Forward and backward of norm -> 8-bit linear."""
    codes, scales = hip.layer_norm_quantize_fp8(x, w, b)
    y = hip.linear_fp8(codes, scales, *wq, y_dtype=torch.bfloat16)
    h, mean, rstd = hip.layer_norm(x, w, b)
    ht = hip.quantize_fp8(h, transposed=True)
    dh, dwt = hip.linear_fp8_backward(dy, *ht, *wtq)
    return (y, dwt, *hip.layer_norm_backward(dh, x, mean, rstd, weight=w))


def _step_inputs(hip, m, k, n):
    x, w, b = _cuda(_x(m, k, 1), *_affine(k, torch.float32))
    wt = (0.02 * _x(n, k, 2)).cuda()
    wc, ws, wtc, wts = hip.quantize_fp8_both(wt, block_rows=128)
    return x, w, b, (wc, ws), (wtc, wts), (1e-3 * _x(m, n, 3)).cuda()


@pytest.mark.parametrize("m", [20, 333])
def test_training_step_together(hip, m):
    k, n = 640, 384
    x, w, b, wq, wtq, dy = _step_inputs(hip, m, k, n)
    y, dwt, dx, dw, db = (t.double().cpu() for t in _step(hip, x, w, b, wq, wtq, dy))
    h = ref64.layer_norm(x.cpu(), w.cpu(), b.cpu(), EPS)[0].to(torch.bfloat16)
    by = (lambda t: t.contiguous().view(torch.uint8).cpu())
    wv = ref64.fp8_values(by(wq[0]), by(wq[1]), 128)
    # a value of the norm next to a bf16 border may round the other way (1 step in
    # 2^8), and its code with it (one step in 2^3 of a few codes): compare norms
    near = (lambda a, r, t: float((a - r).norm() / r.norm()) <= t)
    hq = ref64.fp8_values(*ref64.fp8_quantize(h))
    assert near(y, hq @ wv.T, 2.0 ** -8 + 2.0 ** -7)
    dyc = dy.cpu()
    htq = ref64.fp8_values(*ref64.fp8_quantize(h.T))
    assert near(dwt, ref64.fp8_values(*ref64.fp8_quantize(dyc.T)) @ htq.T, 2.0 ** -7)
    dh = (ref64.fp8_values(*ref64.fp8_quantize(dyc)) @ wv).to(torch.bfloat16)
    _, mean, rstd = ref64.layer_norm(x.cpu(), None, None, EPS)
    rx, rw, rb = ref64.layer_norm_backward(dh, x.cpu(), mean, rstd, w.cpu())
    assert near(dx, rx, 2.0 ** -7) and near(dw, rw, 2.0 ** -7) and near(db, rb, 2.0 ** -7)


@pytest.mark.parametrize("m", [20, 333])
def test_training_step_in_a_graph(hip, m):
    """Captured once, replayed with new inputs between eager calls."""
    x, w, b, wq, wtq, dy = _step_inputs(hip, m, 640, 384)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        _step(hip, x, w, b, wq, wtq, dy)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = _step(hip, x, w, b, wq, wtq, dy)
    for i in range(4):
        x.copy_(_x(m, 640, 20 + i))
        dy.copy_(1e-3 * _x(m, 384, 40 + i))
        want = [t.clone() for t in _step(hip, x, w, b, wq, wtq, dy)]
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for p, q in zip(out, want):
            assert torch.equal(p, q), i
