"""The 4-bit microscaled format on the GPU against 64-bit references: codes and scales bit
for bit, products within the bound that counts their fp32 additions, and exactly where
every sum is representable."""
import pytest
import torch

import mx4_ref

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float32]


def _x(rows, k, seed=0, dtype=torch.bfloat16, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((rows, k), generator=g) * torch.exp(spread * torch.randn((1, k), generator=g))).to(dtype)


def _bytes(t):
    return t.contiguous().view(torch.uint8).cpu()


def _strided(x, ld, offset=0):
    rows, k = x.shape
    full = torch.full((rows * ld + offset + 16,), 7.0, dtype=x.dtype, device="cuda")
    v = full[offset:offset + rows * ld].view(rows, ld)[:, :k]
    v.copy_(x)
    return v


def _same(got, x):
    """got: (codes, scales) of the library for x."""
    rc, rs = mx4_ref.quantize(x)
    gs = _bytes(got[1])
    assert torch.equal(gs, rs), (tuple(x.shape), (gs != rs).nonzero()[:4])
    gc = _bytes(got[0])
    assert torch.equal(gc, rc), (tuple(x.shape), (gc != rc).nonzero()[:4])


SHAPES = [(1, 1), (130, 132), (7, 1300), (1, 128), (3, 31), (3, 33), (5, 129), (127, 16), (128, 128), (129, 257),
          (64, 1000), (300, 640), (1, 5120)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,k", SHAPES)
def test_quantize_every_form(hip, rows, k, dtype):
    x = _x(rows, k, seed=rows * 7 + k, dtype=dtype)
    d = x.cuda()
    both = hip.quantize_mxfp4_both(d)
    for t, src, b in ((False, x, both[:2]), (True, x.T, both[2:])):
        one = hip.quantize_mxfp4(d, transposed=t)
        _same(one, src)
        assert torch.equal(_bytes(b[0]), _bytes(one[0])) and torch.equal(_bytes(b[1]), _bytes(one[1]))


@pytest.mark.parametrize("ld,offset", [(264, 0), (259, 0), (264, 1), (264, 8)])
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("dtype", DTYPES)
def test_quantize_strides(hip, ld, offset, transposed, dtype):
    x = _x(131, 259 if ld == 259 else 250, seed=ld + offset, dtype=dtype)
    _same(hip.quantize_mxfp4(_strided(x, ld, offset), transposed=transposed), x.T if transposed else x)


def test_quantize_rule_at_its_edges(hip):
    """Zeros, subnormal and largest values, the border at 6, ties, blocks that are not finite."""
    x = torch.zeros((13, 256), dtype=torch.float32)
    x[1, 5] = -0.0
    x[2, :128] = torch.linspace(-6, 6, 128)
    x[2, 128:] = torch.linspace(-6.0001, 6.0001, 128)  # just above 6: the next scale
    x[3, :] = 2.0 ** -149
    x[4, :] = torch.finfo(torch.float32).max
    x[4, 1::2] *= -1
    x[5, ::32] = 6.0                                    # scale 1: every tie
    x[5, 1:8] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    x[5, 33:40] = -torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    x[5, 65:72] = torch.tensor([0.2500001, 0.7499999, 1.2500001, 1.7499999, 2.5000002, 3.4999998, 4.9999995])
    x[6, 3] = float("inf")
    x[6, 40] = 1.0
    x[7, 130] = float("nan")
    x[7, 0] = 3.0
    x[8, :] = 2.0 ** -130
    x[8, 7] = 2.0 ** -125
    x[9, :] = 2.0 ** -127 * 6                           # the smallest scale holds
    x[10, :] = 1.0 / 3.0
    x[11, ::40] = -float("inf")
    x[12, :] = 6 * 2.0 ** -126
    for dtype in DTYPES:
        xd = x.to(dtype)
        _same(hip.quantize_mxfp4(xd.cuda()), xd)
        _same(hip.quantize_mxfp4(xd.cuda(), transposed=True), xd.T)


def test_every_bf16_value_alone(hip):
    """Each finite bf16 value first in a block of its own, others of it beside."""
    v = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    v = v[torch.isfinite(v)]
    x = torch.zeros((v.numel(), 32), dtype=torch.bfloat16)
    x[:, 0] = v
    x[:, 1] = v * 0.3125
    x[:, 2] = v * -0.0117
    x[:, 3] = v * 0.4167
    _same(hip.quantize_mxfp4(x.cuda()), x)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("experts,n,k", [(1, 5, 40), (3, 130, 257), (5, 128, 128)])
def test_quantize_experts(hip, experts, n, k, dtype):
    x = torch.stack([_x(n, k, seed=e, dtype=dtype) for e in range(experts)])
    codes, scales = hip.quantize_mxfp4(x.cuda())
    tc, ts = hip.quantize_mxfp4(x.cuda(), transposed=True)
    both = hip.quantize_mxfp4_both(x.cuda())
    for e in range(experts):
        _same((codes[e], scales[e]), x[e])
        _same((tc[e], ts[e]), x[e].T)
    for a, b in zip(both, (codes, scales, tc, ts)):
        assert torch.equal(_bytes(a), _bytes(b))


# rows, offsets: empty groups anywhere, one row, all in one group, rows before and behind, more than 64 groups
GROUPS = [(10, [0, 10]), (300, [0, 0, 128, 128, 129, 300, 300]), (257, [3, 3, 131, 250]), (64, [0] * 70 + [64]),
          (1, [0, 0, 1]), (500, list(range(0, 131)) + [499]), (5, [2, 2, 2]), (130, [0, 1, 129, 130])]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,offsets", GROUPS)
def test_quantize_groups(hip, rows, offsets, dtype):
    for k in (1, 130, 264):
        x = _x(rows, k, seed=rows + k, dtype=dtype)
        off = torch.tensor(offsets, device="cuda")
        assert hip.mxfp4_columns(rows, len(offsets) - 1) == mx4_ref.columns(rows, len(offsets) - 1)
        want = mx4_ref.spaced(x, offsets).T
        _same(hip.quantize_mxfp4(x.cuda(), transposed=True, offsets=off), want)
        codes, scales, tc, ts = hip.quantize_mxfp4_both(x.cuda(), offsets=off)
        _same((tc, ts), want)
        _same((codes[offsets[0]:offsets[-1]], scales.view(torch.uint8)[offsets[0]:offsets[-1]]),
              x[offsets[0]:offsets[-1]])


def test_groups_without_rows(hip):
    off = torch.zeros(201, dtype=torch.int64, device="cuda")
    codes, scales = hip.quantize_mxfp4(torch.empty((0, 50), device="cuda"), transposed=True, offsets=off)
    assert codes.shape == (50, 198 * 64) and not codes.any() and not scales.view(torch.uint8).any()


@pytest.mark.parametrize("out", DTYPES)
@pytest.mark.parametrize("rows,k", [(1, 1), (130, 257), (256, 1024), (3, 7)])
def test_dequantize(hip, rows, k, out):
    g = torch.Generator().manual_seed(rows)
    kp = mx4_ref.up128(k)
    codes = torch.randint(0, 256, (rows, kp // 2), generator=g, dtype=torch.uint8)
    scales = torch.randint(0, 252, (rows, kp // 32), generator=g).to(torch.uint8)
    scales[0, 0] = 255
    want = mx4_ref.values(codes, scales)[:, :k]
    s = scales.cuda().view(torch.float8_e8m0fnu)
    for place in (0, 1):  # whole pieces, and at the elements' own alignment
        o = torch.full((rows * k + 3,), 5.0, dtype=out, device="cuda")
        got = hip.dequantize_mxfp4(codes.cuda(), s, k=k, out_dtype=out, out=o[place:place + rows * k].view(rows, k))
        assert torch.equal(torch.nan_to_num(got.double().cpu(), nan=77.0), torch.nan_to_num(want, nan=77.0))
        assert bool((o[place + rows * k:] == 5).all())


def _random(rows, k, seed, lo=119, hi=135):
    """Code and scale bytes, scales in lo .. hi."""
    g = torch.Generator().manual_seed(seed)
    return (torch.randint(0, 256, (rows, k // 2), generator=g, dtype=torch.uint8),
            torch.randint(lo, hi + 1, (rows, k // 32), generator=g).to(torch.uint8))


def _cuda(c):
    return c[0].cuda(), c[1].cuda().view(torch.float8_e8m0fnu)


def _near(y, xv, wv, parts=64):
    ref, s = xv @ wv.T, xv.abs() @ wv.abs().T
    err = (y.double().cpu() - ref).abs()
    tol = mx4_ref.bound(xv.shape[1], s, y.dtype, parts)
    assert bool((err <= tol).all()), (tuple(y.shape), y.dtype, float((err / tol).max()))


# up to 16 and 32 rows, tiles of 64 x 64 whole and with K split, of 128 x 128; depths of one run, an
# odd and an even count of them (sizes for every kernel, tiles of 256 x 256 among them: mx4_cases.py)
LINEAR = [(1, 1, 128), (1, 13, 384), (3, 96, 5120), (16, 41, 2176), (17, 41, 128), (70, 96, 512), (300, 96, 5120),
          (301, 97, 4224), (129, 257, 13824), (1408, 1536, 256), (1409, 1535, 384), (2176, 2304, 256), (2049, 2305, 640),
          (2048, 9000, 256), (4097, 4099, 384), (5120, 8192, 128)]


@pytest.mark.parametrize("y_dtype", DTYPES)
@pytest.mark.parametrize("m,n,k", LINEAR)
def test_linear(hip, m, n, k, y_dtype):
    x, w = _random(m, k, seed=m + k), _random(n, k, seed=n + k + 1)
    y = hip.linear_mxfp4(*_cuda(x), *_cuda(w), y_dtype=y_dtype)
    _near(y, mx4_ref.values(*x), mx4_ref.values(*w))


@pytest.mark.parametrize("m,n,k", LINEAR)
def test_linear_exact_sums(hip, m, n, k):
    """Scales within 2^4 of each other: products are multiples of 2^-2 of the smallest; up to
    some 2^12 of them keep every partial sum below 2^24 such steps on random signs."""
    k = min(k, 4096)
    x, w = _random(m, k, seed=m + k + 5, lo=126, hi=128), _random(n, k, seed=n + k + 6, lo=126, hi=128)
    xv, wv = mx4_ref.values(*x), mx4_ref.values(*w)
    ref = xv @ wv.T
    assert float((xv.abs() @ wv.abs().T).max()) < 2.0 ** 20  # steps of 2^-4: exact in fp32 in any order
    y = hip.linear_mxfp4(*_cuda(x), *_cuda(w))
    assert torch.equal(y.double().cpu(), ref)
    yb = hip.linear_mxfp4(*_cuda(x), *_cuda(w), y_dtype=torch.bfloat16)
    assert torch.equal(yb.cpu(), ref.float().to(torch.bfloat16))


@pytest.mark.parametrize("m,n", [(3, 40), (70, 96), (1408, 1536), (2304, 2304), (4352, 4352)])
def test_linear_keeps_small_products_beside_large_ones_that_cancel(hip, m, n):
    """In every run of 8 along k 36 2^12 and -36 2^12 beside six products of 0.25: each sum, of a part of
    a run too, is a whole number of 2^-2 below 2^24 of them, so fp32 additions are exact."""
    k = 256
    x, w = _random(m, k, 1, 127, 127), _random(n, k, 2, 127, 127)
    for c, large in ((x, 0x77), (w, 0xF7)):
        c[0][:] = (c[0] & 0x88) | 0x11
        c[0][:, ::4] = large
    big = torch.zeros(k // 32, dtype=torch.bool)
    big[::2] = True  # blocks of 2^12 that cancel, blocks of 1
    x[1][:, big] = 133
    w[1][:, big] = 133
    xv, wv = mx4_ref.values(*x), mx4_ref.values(*w)
    want = xv @ wv.T
    assert float(want.abs().max()) < 2.0 ** 22 and bool(want.any())
    assert torch.equal(hip.linear_mxfp4(*_cuda(x), *_cuda(w)).double().cpu(), want)


@pytest.mark.parametrize("m,n,k", [(2, 33, 512), (80, 96, 512), (1500, 1500, 512), (4352, 4352, 256)])
def test_linear_every_scale_byte(hip, m, n, k):
    """Scales 0 to 254 whose products stay in range; NaN where one is 255, and nowhere else."""
    x, w = _random(m, k, 1, 127, 127), _random(n, k, 2, 127, 127)
    b = torch.arange(k // 32) * 254 // (k // 32 - 1)
    x[1][:] = b.to(torch.uint8)
    w[1][:] = (254 - b).to(torch.uint8)
    xv, wv = mx4_ref.values(*x), mx4_ref.values(*w)
    assert torch.equal(hip.linear_mxfp4(*_cuda(x), *_cuda(w)).double().cpu(), xv @ wv.T)
    x[1][1, 3] = 255
    w[1][n - 1, 5] = 255
    y = hip.linear_mxfp4(*_cuda(x), *_cuda(w), y_dtype=torch.bfloat16).float().cpu()
    bad = torch.isnan(y)
    want = torch.zeros_like(bad)
    want[1, :] = True
    want[:, n - 1] = True
    assert torch.equal(bad, want)


def test_linear_empty(hip):
    x, w = _cuda(_random(5, 128, 0)), _cuda(_random(7, 128, 1))
    none = (torch.empty((5, 0), dtype=torch.uint8, device="cuda"),
            torch.empty((5, 0), dtype=torch.float8_e8m0fnu, device="cuda"))
    none7 = (torch.empty((7, 0), dtype=torch.uint8, device="cuda"),
             torch.empty((7, 0), dtype=torch.float8_e8m0fnu, device="cuda"))
    assert torch.equal(hip.linear_mxfp4(*none, *none7), torch.zeros((5, 7), device="cuda"))
    assert hip.linear_mxfp4(x[0][:0], x[1][:0], *w).shape == (0, 7)
    assert hip.linear_mxfp4(*x, w[0][:0], w[1][:0]).shape == (5, 0)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (7, 130, 33), (130, 7, 257), (300, 700, 129), (1001, 1300, 640),
                                   (2100, 2200, 2111), (129, 4000, 2000)])
def test_linear_backward(hip, m, n, k, dtype):
    dy, x, w = _x(m, n, 1, dtype), _x(m, k, 2, dtype), _x(n, k, 3, dtype, 0.2)
    xt, wt = hip.quantize_mxfp4(x.cuda(), transposed=True), hip.quantize_mxfp4(w.cuda(), transposed=True)
    dyd = _strided(dy, n + 3, 1)
    dx, dw = hip.linear_mxfp4_backward(dyd, *xt, *wt)
    assert dx.dtype == dtype and dw.dtype == torch.float32
    q = lambda t: mx4_ref.values(*mx4_ref.quantize(t))  # noqa: E731
    _near(dx, q(dy), q(w.T.contiguous()))
    _near(dw, q(dy.T), q(x.T.contiguous()))
    other = torch.bfloat16 if dtype == torch.float32 else torch.float32
    dx2, dw2 = hip.linear_mxfp4_backward(dyd, *xt, *wt, dx_dtype=other, dw_dtype=torch.bfloat16)
    _near(dx2, q(dy), q(w.T.contiguous()))
    assert torch.equal(dw2, dw.to(torch.bfloat16))


def _experts(count, n, k, seed, lo=119, hi=135):
    c = [_random(n, k, seed + 10 * e, lo, hi) for e in range(count)]
    return torch.stack([a for a, _ in c]), torch.stack([b for _, b in c])


MANY = [(1000, [0, 17, 17, 800, 1000]), (2600, [0, 1, 1300, 2599, 2600]), (5000, [100, 2400, 2400, 4901]),
        (700, [0, 300, 300, 700])]


@pytest.mark.parametrize("y_dtype", DTYPES)
@pytest.mark.parametrize("n,k", [(1, 128), (70, 384), (300, 640)])
@pytest.mark.parametrize("rows,offsets", GROUPS + MANY)
def test_linear_grouped(hip, rows, offsets, n, k, y_dtype):
    groups = len(offsets) - 1
    x, w = _random(rows, k, rows), _experts(groups, n, k, 7)
    y = torch.full((rows, n), 3.0, dtype=y_dtype, device="cuda")
    got = hip.linear_mxfp4_grouped(*_cuda(x), *_cuda(w), torch.tensor(offsets, device="cuda"), y_dtype=y_dtype, y=y)
    xv = mx4_ref.values(*x)
    for e, (b, t) in enumerate(zip(offsets[:-1], offsets[1:])):
        if t > b:
            _near(got[b:t], xv[b:t], mx4_ref.values(w[0][e], w[1][e]))
    assert bool((y[:offsets[0]] == 3).all()) and bool((y[offsets[-1]:] == 3).all())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,k", [(1, 5), (130, 70), (300, 640)])
@pytest.mark.parametrize("rows,offsets", GROUPS + MANY)
def test_linear_grouped_backward(hip, rows, offsets, n, k, dtype):
    groups = len(offsets) - 1
    off = torch.tensor(offsets, device="cuda")
    dy, x = _x(rows, n, 1, dtype), _x(rows, k, 2, dtype)
    w = torch.stack([_x(n, k, 3 + e, dtype, 0.2) for e in range(groups)])
    xt = hip.quantize_mxfp4(x.cuda(), transposed=True, offsets=off)
    wt = hip.quantize_mxfp4(w.cuda(), transposed=True)
    dx, dw = hip.linear_mxfp4_grouped_backward(dy.cuda(), *xt, *wt, off)
    assert dx.dtype == dtype and dw.dtype == torch.float32 and dw.shape == (groups, n, k)
    q = lambda t: mx4_ref.values(*mx4_ref.quantize(t))  # noqa: E731
    for e, (b, t) in enumerate(zip(offsets[:-1], offsets[1:])):
        if t > b:
            _near(dx[b:t], q(dy[b:t]), q(w[e].T.contiguous()))
            _near(dw[e], q(dy[b:t].T), q(x[b:t].T.contiguous()))
        else:
            assert not dw[e].any()


def test_grouped_empty(hip):
    w = _cuda(_experts(3, 7, 128, 0))
    off = torch.zeros(4, dtype=torch.int64, device="cuda")
    x = _cuda(_random(4, 128, 1))
    assert hip.linear_mxfp4_grouped(x[0][:0], x[1][:0], *w, off).shape == (0, 7)
    y = torch.full((4, 7), 9.0, device="cuda")  # no row is in a group
    hip.linear_mxfp4_grouped(*x, *w, off, y=y)
    assert bool((y == 9).all())
    none = (torch.empty((4, 0), dtype=torch.uint8, device="cuda"), torch.empty((4, 0), dtype=torch.float8_e8m0fnu, device="cuda"))
    now = (torch.empty((3, 7, 0), dtype=torch.uint8, device="cuda"), torch.empty((3, 7, 0), dtype=torch.float8_e8m0fnu, device="cuda"))
    off = torch.tensor([0, 1, 1, 3], device="cuda")
    hip.linear_mxfp4_grouped(*none, *now, off, y=y)  # an empty contraction
    assert not y[:3].any() and bool((y[3] == 9).all())
    # no rows at all: the weights' gradients are zero
    xt = hip.quantize_mxfp4(torch.empty((0, 40), device="cuda"), transposed=True, offsets=off * 0)
    wt = hip.quantize_mxfp4(torch.ones((3, 7, 40), device="cuda"), transposed=True)
    dx, dw = hip.linear_mxfp4_grouped_backward(torch.empty((0, 7), device="cuda"), *xt, *wt, off * 0)
    assert dx.shape == (0, 40) and dw.shape == (3, 7, 40) and not dw.any()


def test_gradients_are_those_of_the_layer(hip):
    """Differences of the layer's own output: with dY a single 1, dX is a row of W and dW a row of X."""
    m, n, k = 40, 50, 64
    x, w = _x(m, k, 1, torch.float32), _x(n, k, 2, torch.float32)
    off = torch.tensor([0, 15, 15, 40], device="cuda")
    we = torch.stack([w, w * 2, w * 3]).cuda()
    xt = hip.quantize_mxfp4(x.cuda(), transposed=True, offsets=off)
    wt = hip.quantize_mxfp4(we, transposed=True)
    dy = torch.zeros((m, n), device="cuda")
    dy[20, 33] = 1.0
    dx, dw = hip.linear_mxfp4_grouped_backward(dy, *xt, *wt, off)
    wv = hip.dequantize_mxfp4(*wt, k=n)  # [3][k][n]
    xv = hip.dequantize_mxfp4(*xt)       # group 2 begins at column 128
    assert torch.equal(dx[20], wv[2][:, 33]) and not dx[:20].any() and not dx[21:].any()
    assert torch.equal(dw[2][33], xv[:, 128 + 5]) and not dw[:2].any() and not dw[2][:33].any()


def _layer(hip, x, g, b, w, off, dy):
    """An experts' layer behind a norm, forward and backward."""
    h, mean, rstd = hip.layer_norm(x, g, b)
    hc, hs, ht, hts = hip.quantize_mxfp4_both(h, offsets=off)
    wc, ws, wt, wts = hip.quantize_mxfp4_both(w)
    y = hip.linear_mxfp4_grouped(hc, hs, wc, ws, off, y_dtype=torch.bfloat16)
    dh, dw = hip.linear_mxfp4_grouped_backward(dy, ht, hts, wt, wts, off)
    return y, dw, *hip.layer_norm_backward(dh, x, mean, rstd, weight=g)


def test_a_run_of_them_captured_and_replayed(hip):
    """A layer of experts captured once and replayed with other inputs and other offsets, eager
    work in between; the same on another stream."""
    def inputs(seed, offsets):
        x = _x(600, 256, seed).cuda()
        g, b = _x(1, 256, seed + 1, torch.float32)[0].cuda(), _x(1, 256, seed + 2, torch.float32)[0].cuda()
        w = torch.stack([_x(300, 256, seed + 3 + e) for e in range(4)]).cuda()
        return [x, g, b, w, torch.tensor(offsets, device="cuda"), _x(600, 300, seed + 9).cuda()]
    sets = [inputs(1, [0, 100, 100, 350, 600]), inputs(20, [0, 0, 599, 600, 600]), inputs(40, [0, 128, 256, 384, 600])]
    eager = [[t.clone() for t in _layer(hip, *s)] for s in sets]
    held = [t.clone() for t in sets[0]]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        warm = _layer(hip, *held)
        for a, b in zip(warm, eager[0]):
            assert torch.equal(a, b)
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _layer(hip, *held)
    for i in (1, 0, 2, 1, 1):
        for h, t in zip(held, sets[i]):
            h.copy_(t)
        graph.replay()
        again = _layer(hip, *sets[i])  # eager work beside the graph's
        torch.cuda.synchronize()
        for a, b, c in zip(out, eager[i], again):
            assert torch.equal(a, b) and torch.equal(c, b)


def test_calls_on_a_stream_of_their_own(hip):
    x, w = _x(300, 512, 1).cuda(), _x(200, 512, 2).cuda()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    xq, wq = hip.quantize_mxfp4(x, stream=side), hip.quantize_mxfp4(w, stream=side)
    y = hip.linear_mxfp4(*xq, *wq, stream=side)
    side.synchronize()
    assert torch.equal(y, hip.linear_mxfp4(*hip.quantize_mxfp4(x), *hip.quantize_mxfp4(w)))


def test_results_do_not_change_from_run_to_run(hip):
    for m, n, k in ((9, 500, 5120), (300, 96, 13824), (2304, 2304, 512)):
        x, w = _cuda(_random(m, k, 1)), _cuda(_random(n, k, 2))
        first = hip.linear_mxfp4(*x, *w)
        for _ in range(3):
            assert torch.equal(hip.linear_mxfp4(*x, *w), first)


@pytest.mark.parametrize("affine", [torch.float32, torch.bfloat16, None])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,c", [(1, 1), (5, 7), (77, 1003), (3, 128), (700, 96), (900, 200), (600, 400), (530, 640),
                                    (2100, 5120), (2050, 6000), (9, 16385), (2, 20000)])
def test_norm_into_mxfp4_is_the_two_calls_in_turn(hip, rows, c, dtype, affine):
    x = _x(rows, c, rows + c, dtype).cuda()
    w = b = None
    if affine is not None:
        w, b = 1 + 0.2 * _x(1, c, 5, torch.float32)[0], 0.2 * _x(1, c, 6, torch.float32)[0]
        w, b = w.to(affine).cuda(), b.to(affine).cuda()
    codes, scales = hip.layer_norm_quantize_mxfp4(x, w, b)
    y, _, _ = hip.layer_norm(x, w, b)
    want = hip.quantize_mxfp4(y)
    assert torch.equal(codes, want[0]) and torch.equal(_bytes(scales), _bytes(want[1]))
    _same((codes, scales), y.cpu())


def test_norm_into_mxfp4_strides_and_values(hip):
    x = _x(520, 1002, 3)
    for ld, offset in ((1002, 0), (1008, 0), (1011, 1)):
        xs = _strided(x, ld, offset)
        codes, scales = hip.layer_norm_quantize_mxfp4(xs, eps=1e-5)
        _same((codes, scales), hip.layer_norm(xs, eps=1e-5)[0].cpu())
    x[7, 3] = float("nan")  # that row alone
    codes, scales = hip.layer_norm_quantize_mxfp4(x.cuda())
    v = hip.dequantize_mxfp4(codes, scales, k=1002)
    assert bool(torch.isnan(v[7]).all()) and not torch.isnan(v[:7]).any() and not torch.isnan(v[8:]).any()


@pytest.mark.parametrize("offsets", [[0, 300, 100, 260], [-50, 10, 5000, 200], [400, 400, 0, 300], [300, 200, 100, 0],
                                     [1 << 40, -(1 << 40), 1 << 62, 7]])
def test_offsets_that_do_not_ascend_stay_within_the_arguments(hip, offsets):
    """What the results are is not said; what lies before and behind them is left alone."""
    rows, n, k = 300, 72, 256
    off = torch.tensor(offsets, device="cuda")
    x, w = _random(rows, k, 1), _experts(3, n, k, 2)
    held = torch.full((rows * n + 4096,), 5.0, device="cuda")
    hip.linear_mxfp4_grouped(*_cuda(x), *_cuda(w), off, y=held[2048:-2048].view(rows, n))
    codes = torch.full((k * (mx4_ref.columns(rows, 3) // 2) + 4096,), 77, dtype=torch.uint8, device="cuda")
    v = _x(rows, k, 3).cuda()
    out = codes[2048:-2048].view(k, -1)
    _, scales = hip.quantize_mxfp4(v, transposed=True, offsets=off, codes=out)
    dx, dw = hip.linear_mxfp4_grouped_backward(_x(rows, n, 4).cuda(), out, scales,
                                               *hip.quantize_mxfp4(torch.ones((3, n, k), device="cuda"), transposed=True),
                                               off)
    torch.cuda.synchronize()
    assert bool((held[:2048] == 5).all()) and bool((held[-2048:] == 5).all())
    assert bool((codes[:2048] == 77).all()) and bool((codes[-2048:] == 77).all())
    assert dx.shape == (rows, k) and dw.shape == (3, n, k)


def test_many_groups(hip):
    """More groups than one pass over their offsets takes at once, most of them empty."""
    g = torch.Generator().manual_seed(5)
    counts = (torch.rand(1500, generator=g) < 0.1).long() * torch.randint(1, 60, (1500,), generator=g)
    off = torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)])
    rows, n, k = int(off[-1]), 20, 128
    x, w = _random(rows, k, 1), _random(1500 * n, k, 2)
    wq = tuple(t.view(1500, n, -1) for t in _cuda(w))
    y = hip.linear_mxfp4_grouped(*_cuda(x), *wq, off.cuda())
    wv, xv = mx4_ref.values(*w).view(1500, n, k), mx4_ref.values(*x)
    expert = torch.repeat_interleave(torch.arange(1500), counts)
    want = torch.bmm(wv[expert], xv[:, :, None])[:, :, 0]
    s = torch.bmm(wv[expert].abs(), xv.abs()[:, :, None])[:, :, 0]
    assert bool(((y.double().cpu() - want).abs() <= mx4_ref.bound(k, s, torch.float32)).all())
    v = _x(rows, 40, 3)
    _same(hip.quantize_mxfp4(v.cuda(), transposed=True, offsets=off.cuda()), mx4_ref.spaced(v, off.tolist()).T)
