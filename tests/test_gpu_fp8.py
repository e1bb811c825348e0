"""The 8-bit block format on the GPU against 64-bit references: codes and scales
bit for bit, products within the bound that counts their fp32 additions."""
import pytest
import torch

import ref64

pytestmark = pytest.mark.gpu

U = 2.0 ** -24           # half a step of fp32
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}  # half a step of the output type


def _x(rows, k, seed=0, dtype=torch.bfloat16, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, k), generator=g) * torch.exp(spread * torch.randn((1, k), generator=g))
    return x.to(dtype)


def _bytes(t):
    return t.contiguous().view(torch.uint8).cpu()


def _strided(x, ld, offset=0):
    """x on the GPU as a view with leading dimension ld, starting offset elements in."""
    rows, k = x.shape
    full = torch.full((rows * ld + offset + 16,), 7.0, dtype=x.dtype, device="cuda")
    v = full[offset:offset + rows * ld].view(rows, ld)[:, :k]
    v.copy_(x)
    return v


def _check_quantized(x, codes, scales, block_rows):
    rc, rs = ref64.fp8_quantize(x, block_rows)
    assert torch.equal(_bytes(scales), rs), (x.shape, block_rows)
    got = _bytes(codes)
    assert torch.equal(got, rc), (x.shape, block_rows, (got != rc).nonzero()[:4])


SHAPES = [(1, 1), (130, 132), (7, 1300), (1, 128), (3, 127), (5, 129), (127, 16), (128, 128), (129, 257), (64, 1000),
          (300, 640), (1, 5120)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("rows,k", SHAPES)
def test_quantize_every_form(hip, rows, k, block_rows, dtype):
    x = _x(rows, k, seed=rows * 7 + k, dtype=dtype)
    d = x.cuda()
    both = hip.quantize_fp8_both(d, block_rows=block_rows)
    for t, src, (bc, bs) in ((False, x, both[:2]), (True, x.T, both[2:])):
        codes, scales = hip.quantize_fp8(d, block_rows=block_rows, transposed=t)
        _check_quantized(src, codes, scales, block_rows)
        assert torch.equal(_bytes(bc), _bytes(codes)) and torch.equal(_bytes(bs), _bytes(scales))


@pytest.mark.parametrize("ld,offset", [(264, 0), (259, 0), (264, 1), (264, 8)])
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantize_strides(hip, ld, offset, transposed, dtype):
    x = _x(131, 259 if ld == 259 else 250, seed=ld + offset, dtype=dtype)
    codes, scales = hip.quantize_fp8(_strided(x, ld, offset), transposed=transposed)
    _check_quantized(x.T if transposed else x, codes, scales, 1)


def test_quantize_rule_at_its_edges(hip):
    """Zero, subnormal and largest values, the 448 border, rounding ties, non-finite blocks."""
    x = torch.zeros((12, 256), dtype=torch.float32)
    x[1, 5] = -0.0
    x[2, :128] = torch.linspace(-448, 448, 128)
    x[2, 128:] = torch.linspace(-448.0001, 448.0001, 128)   # just above 448: the next scale
    x[3, :] = 2.0 ** -149
    x[4, :] = torch.finfo(torch.float32).max
    x[4, 1::2] *= -1
    x[5, 0] = 256.0                                          # scale 1: ties of every binade follow
    x[5, 1:113] = torch.arange(1, 113) * 2.0 ** -10 + 2.0 ** -11
    x[5, 128:] = 256 + 8 * torch.arange(128) / 128
    x[6, 3] = float("inf")
    x[6, 200] = 1.0
    x[7, 130] = float("nan")
    x[7, 0] = 3.0
    x[8, :] = 2.0 ** -130
    x[8, 7] = 2.0 ** -118
    x[9, :] = 2.0 ** -119 * 1.75                             # 448 * 2^-127: the smallest scale holds
    x[10, :] = 1.0 / 3.0
    x[11, ::3] = -float("inf")
    for dtype in (torch.float32, torch.bfloat16):
        xd = x.to(dtype)
        for t in (False, True):
            codes, scales = hip.quantize_fp8(xd.cuda(), transposed=t)
            _check_quantized(xd.T if t else xd, codes, scales, 1)
        codes, scales = hip.quantize_fp8(xd.cuda(), block_rows=128)
        _check_quantized(xd, codes, scales, 128)


def test_every_bf16_value_alone(hip):
    """Each finite bf16 value in a block of its own beside each of a few maxima."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16)
    v = bits.view(torch.bfloat16)
    v = v[torch.isfinite(v)]
    x = torch.zeros((v.numel(), 128), dtype=torch.bfloat16)
    x[:, 0] = v
    x[:, 1] = v * 0.3125
    x[:, 2] = v * -0.0117
    codes, scales = hip.quantize_fp8(x.cuda())
    _check_quantized(x, codes, scales, 1)


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,k", [(1, 1), (130, 257), (256, 1024)])
def test_dequantize(hip, rows, k, out):
    x = _x(rows, k, seed=5).cuda()
    for block_rows in (1, 128):
        codes, scales = hip.quantize_fp8(x, block_rows=block_rows)
        want = ref64.fp8_values(_bytes(codes), _bytes(scales), block_rows)[:, :k]
        got = hip.dequantize_fp8(codes, scales, k=k, out_dtype=out)
        assert torch.equal(got.double().cpu(), want)  # E4M3 times a power of two: exact in both
    s32 = torch.rand(scales.shape, device="cuda") + 0.5
    want = ref64.fp8_values(_bytes(codes), s32.cpu(), 128)[:, :k]
    got = hip.dequantize_fp8(codes, s32, k=k, out_dtype=out).double().cpu()
    # the product is rounded to fp32, then to the output type
    assert bool(((got - want).abs() <= (U + HALF[out] * (1 + U)) * want.abs()).all())


def _linear_case(hip, m, n, k, kind, seed=0):
    """Quantized operands on the GPU and their 64-bit values."""
    xc, xs = hip.quantize_fp8(_x(m, k, seed + 1).cuda())
    w = _x(n, k, seed + 2, spread=0.2).cuda()
    wc, ws = hip.quantize_fp8(w, block_rows=1 if kind == "rows" else 128)
    xv = ref64.fp8_values(_bytes(xc), _bytes(xs))
    if kind == "f32":
        g = torch.Generator().manual_seed(seed)
        ws = (0.01 + torch.rand(ws.shape, generator=g)).cuda()
        wv = ref64.fp8_values(_bytes(wc), ws.cpu(), 128)
    else:
        wv = ref64.fp8_values(_bytes(wc), _bytes(ws), 1 if kind == "rows" else 128)
    return (xc, xs, wc, ws), xv, wv


def _check_product(y, xv, wv):
    """Every product is exact (4 + 4 significant bits). A float32 result: at most k
    additions round (each by U of a partial sum, itself at most S = sum |x||w|), a
    float32 scale rounds once per block (k / 128 more), and the result once. A
    bf16 result may come from the fp8 matrix instructions, which cut each of 8
    products that are added at once to 2^-13 of the largest one's power of two: at
    most 7 * 2^-13 of that product, so of S, more; then it rounds to bf16."""
    want, s = xv @ wv.T, xv.abs() @ wv.abs().T
    k = xv.shape[1]
    tol = (k + k // 128 + 1) * U * s
    if y.dtype == torch.bfloat16:
        tol = (tol + 7 * 2.0 ** -13 * s) * (1 + HALF[y.dtype]) + HALF[y.dtype] * want.abs()
    err = (y.double().cpu() - want).abs()
    assert bool((err <= tol).all()), (float((err / s.clamp(min=1e-300)).max()), k)


MS = [1, 2, 15, 16, 17, 33, 64, 65, 100, 127, 128, 129, 200, 257, 300]
NS = [1, 3, 15, 16, 17, 130, 255, 256, 300]


@pytest.mark.parametrize("kind", ["tiles", "rows", "f32"])
@pytest.mark.parametrize("m", MS)
def test_linear_shapes(hip, m, kind):
    for i, n in enumerate(NS):
        k = (128, 256, 384, 640, 1152)[(i + m) % 5]
        args, xv, wv = _linear_case(hip, m, n, k, kind, seed=m * 31 + n)
        for out in (torch.float32, torch.bfloat16):
            _check_product(hip.linear_fp8(*args, y_dtype=out), xv, wv)


@pytest.mark.parametrize("kind", ["tiles", "rows", "f32"])
@pytest.mark.parametrize("m,n", [(1, 4097), (3, 5003), (16, 13824), (7, 8200)])
def test_linear_few_rows_many_columns(hip, m, n, kind):
    """Workgroups whose columns are not 16, and lie in two scale blocks."""
    args, xv, wv = _linear_case(hip, m, n, 384, kind, seed=n)
    for out in (torch.float32, torch.bfloat16):
        _check_product(hip.linear_fp8(*args, y_dtype=out), xv, wv)


@pytest.mark.parametrize("kind", ["tiles", "rows", "f32"])
@pytest.mark.parametrize("m,n,k", [(4100, 4099, 128), (4352, 4096, 640), (2048, 9000, 384), (2300, 4099, 256),
                                   (2100, 1300, 512), (1400, 3001, 640), (1290, 1700, 896), (650, 330, 4224)])
def test_linear_many_tiles(hip, m, n, k, kind):
    """Every tile kernel (256, 128 by two and by one a CU, 64 whole and with K split),
    ragged at both ends."""
    args, xv, wv = _linear_case(hip, m, n, k, kind, seed=3)
    y = hip.linear_fp8(*args)
    rows = torch.tensor([0, 1, 31, 32, 127, 128, 255, 256, min(1000, m - 3), m // 2, m - 2, m - 1])
    _check_product(y[rows.cuda()], xv[rows], wv)
    cols = torch.tensor([0, 5, 63, 64, 255, 256, n // 2, min(4000, n - 2), n - 1])
    _check_product(y[:, cols.cuda()], xv, wv[cols])


@pytest.mark.parametrize("n", [5248, 5121, 5250])
def test_linear_float_scales_end_inside_a_tile(hip, n):
    """Tiles of 256 columns of which the last block row of scales covers only the first half:
    the rows behind it belong to others."""
    m, k = 2048, 256
    (xc, xs, wc, ws), xv, wv = _linear_case(hip, m, n, k, "f32", seed=n)
    more = torch.full((ws.shape[0] + 4, ws.shape[1]), float("nan"), device="cuda")
    more[:ws.shape[0]] = ws
    rows = torch.tensor([0, 255, 256, 1000, m - 1])
    for out in (torch.float32, torch.bfloat16):
        y = hip.linear_fp8(xc, xs, wc, more[:ws.shape[0]], y_dtype=out)
        _check_product(y[rows.cuda()], xv[rows], wv)


def test_linear_few_rows_more_columns_than_a_grid(hip):
    """More columns than workgroups of 1024 threads for 16 columns can be launched for."""
    m, n = 3, (1 << 26) + 5
    xc, xs = hip.quantize_fp8(_x(m, 128, 1).cuda())
    wc = torch.randint(0, 0x70, (n, 128), dtype=torch.uint8, device="cuda")
    ws = torch.full(((n + 127) // 128, 4), 120, dtype=torch.uint8, device="cuda")
    f8, e8 = torch.float8_e4m3fn, torch.float8_e8m0fnu
    y = hip.linear_fp8(xc, xs, wc.view(f8), ws.view(e8)[:, :1], y_dtype=torch.bfloat16)
    cols = torch.tensor([0, 1, 1 << 20, (1 << 25) + 77, (1 << 26) - 1, 1 << 26, n - 1]).cuda()
    wv = ref64.fp8_values(wc[cols].cpu(), ws[:len(cols), :1].cpu())
    _check_product(y[:, cols], ref64.fp8_values(_bytes(xc), _bytes(xs)), wv)


@pytest.mark.parametrize("m,n,k", [(1, 5120, 13824), (16, 1280, 13824), (300, 700, 13824)])
def test_linear_long_sum(hip, m, n, k):
    args, xv, wv = _linear_case(hip, m, n, k, "tiles", seed=9)
    _check_product(hip.linear_fp8(*args), xv, wv)


@pytest.mark.parametrize("m", [3, 70, 300])
def test_linear_same_sign_sum_keeps_fp32(hip, m):
    """All products positive: the error of the sum stays that of fp32 additions."""
    k = 5120
    xc, xs = hip.quantize_fp8(_x(m, k, 1).abs().cuda())
    wc, ws = hip.quantize_fp8(_x(96, k, 2, spread=0.2).abs().cuda(), block_rows=128)
    y = hip.linear_fp8(xc, xs, wc, ws).double().cpu()
    want = ref64.fp8_values(_bytes(xc), _bytes(xs)) @ ref64.fp8_values(_bytes(wc), _bytes(ws), 128).T
    rel = ((y - want).abs() / want).max()
    # k additions that round by U each: a kernel that accumulated in fewer bits
    # would be off by 2^-13 and more
    assert float(rel) <= k * U, float(rel)


def test_linear_scales_far_apart(hip):
    """Scales near both ends of E8M0 whose product is an ordinary number."""
    m, n, k = 20, 40, 256
    for mm in (m, 300):
        x = _x(mm, k, 1).float() * 2.0 ** -110
        w = _x(n, k, 2, spread=0.1).float() * 2.0 ** 110
        xc, xs = hip.quantize_fp8(x.cuda())
        wc, ws = hip.quantize_fp8(w.cuda(), block_rows=128)
        xv = ref64.fp8_values(_bytes(xc), _bytes(xs))
        wv = ref64.fp8_values(_bytes(wc), _bytes(ws), 128)
        _check_product(hip.linear_fp8(xc, xs, wc, ws), xv, wv)


@pytest.mark.parametrize("m", [5, 150])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_linear_nan_scale(hip, m, out):
    """Scale byte 255 is NaN whatever the codes are."""
    xc, xs = hip.quantize_fp8(_x(m, 512, 4).cuda())
    wc, ws = hip.quantize_fp8(_x(70, 512, 5).cuda(), block_rows=128)
    xs.view(torch.uint8)[3, 2] = 255
    y = hip.linear_fp8(xc, xs, wc, ws, y_dtype=out).cpu()
    assert bool(torch.isnan(y[3]).all()) and bool(torch.isfinite(y[:3]).all()) and bool(torch.isfinite(y[4:]).all())
    assert bool(torch.isnan(hip.dequantize_fp8(xc, xs)[3, 256:384]).all())


@pytest.mark.parametrize("m", [5, 150])
def test_linear_nan_block_stays_in_its_row(hip, m):
    x = _x(m, 256, 4).float()
    x[2, 130] = float("nan")
    x[4, 1] = float("inf")
    xc, xs = hip.quantize_fp8(x.cuda())
    wc, ws = hip.quantize_fp8(_x(70, 256, 5).cuda(), block_rows=128)
    y = hip.linear_fp8(xc, xs, wc, ws).cpu()
    bad = torch.zeros(m, dtype=torch.bool)
    bad[[2, 4]] = True
    assert bool(torch.isnan(y[bad]).all()) and bool(torch.isfinite(y[~bad]).all())


def test_linear_empty(hip):
    e8 = torch.float8_e8m0fnu
    w, ws = hip.quantize_fp8(_x(40, 128).cuda(), block_rows=128)
    x = torch.empty((0, 128), dtype=torch.float8_e4m3fn, device="cuda")
    assert hip.linear_fp8(x, torch.empty((0, 1), dtype=e8, device="cuda"), w, ws).shape == (0, 40)
    x0 = torch.empty((3, 0), dtype=torch.float8_e4m3fn, device="cuda")
    w0 = torch.empty((4, 0), dtype=torch.float8_e4m3fn, device="cuda")
    y = torch.full((3, 4), 9.0, device="cuda")
    hip.linear_fp8(x0, torch.empty((3, 0), dtype=e8, device="cuda"), w0,
                   torch.empty((4, 0), dtype=e8, device="cuda"), y=y)
    assert bool((y == 0).all())
    codes, scales = hip.quantize_fp8(torch.empty((0, 200), device="cuda"))
    assert codes.shape == (0, 256) and scales.shape == (0, 2)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,n,k", [(1, 130, 70), (100, 257, 300), (385, 640, 129), (1001, 200, 384)])
def test_linear_backward(hip, m, n, k, dtype):
    dy = _x(m, n, 3, dtype=dtype) * 1e-3
    xt = hip.quantize_fp8(_x(m, k, 4).cuda(), transposed=True)
    wt = hip.quantize_fp8(_x(n, k, 5, spread=0.2).cuda(), block_rows=128, transposed=True)
    dx, dw = hip.linear_fp8_backward(dy.cuda(), *xt, *wt)
    assert dx.dtype == dtype and dx.shape == (m, k) and dw.dtype == torch.float32 and dw.shape == (n, k)
    _check_product(dx, ref64.fp8_values(*ref64.fp8_quantize(dy)),
                   ref64.fp8_values(_bytes(wt[0]), _bytes(wt[1]), 128))
    _check_product(dw, ref64.fp8_values(*ref64.fp8_quantize(dy.T)),
                   ref64.fp8_values(_bytes(xt[0]), _bytes(xt[1])))


@pytest.mark.parametrize("m,n,k", [(0, 40, 64), (30, 0, 64), (30, 40, 0)])
def test_linear_backward_empty(hip, m, n, k):
    dy = torch.ones((m, n), device="cuda")
    xt = hip.quantize_fp8(torch.ones((m, k), device="cuda"), transposed=True)
    wt = hip.quantize_fp8(torch.ones((n, k), device="cuda"), block_rows=128, transposed=True)
    dx, dw = hip.linear_fp8_backward(dy, *xt, *wt)
    assert dx.shape == (m, k) and dw.shape == (n, k)
    assert bool((dx == 0).all()) and bool((dw == 0).all())


def test_linear_backward_with_float_scales(hip):
    """W^T as a checkpoint's codes and float32 scales transposed."""
    m, n, k = 70, 300, 260
    dy = _x(m, n, 3) * 1e-3
    xt = hip.quantize_fp8(_x(m, k, 4).cuda(), transposed=True)
    wc, ws = hip.quantize_fp8(_x(n, k, 5, spread=0.2).cuda(), block_rows=128, transposed=True)
    s32 = torch.rand(ws.shape, device="cuda") + 0.5
    dx, _ = hip.linear_fp8_backward(dy.cuda(), *xt, wc, s32, dx_dtype=torch.float32)
    _check_product(dx, ref64.fp8_values(*ref64.fp8_quantize(dy)), ref64.fp8_values(_bytes(wc), s32.cpu(), 128))


def test_linear_backward_against_differences(hip):
    """With a dY that the format holds exactly, the gradients are those of
    sum(Y dY) for Y = X W^T on the quantized values: differences of a form that is
    linear in X and in W have no truncation error."""
    m, n, k = 50, 60, 256
    g = torch.Generator().manual_seed(1)
    dy = torch.randint(-7, 8, (m, n), generator=g).float()
    x, w = _x(m, k, 2), _x(n, k, 3, spread=0.2)
    xt = hip.quantize_fp8(x.cuda(), transposed=True)
    wt = hip.quantize_fp8(w.cuda(), block_rows=128, transposed=True)
    dx, dw = hip.linear_fp8_backward(dy.cuda(), *xt, *wt)
    xv = ref64.fp8_values(_bytes(xt[0]), _bytes(xt[1])).T[:m]
    wv = ref64.fp8_values(_bytes(wt[0]), _bytes(wt[1]), 128).T[:n]

    def loss(a, b):
        return float(((a @ b.T) * dy.double()).sum())

    for _ in range(4):
        v = torch.randn(xv.shape, generator=g).double()
        u = torch.randn(wv.shape, generator=g).double()
        want = (loss(xv + v, wv) - loss(xv - v, wv)) / 2
        got = float((dx.double().cpu() * v).sum())
        assert abs(got - want) <= n * U * float((dy.abs().double() @ wv.abs() * v.abs()).sum()) + 1e-9 * abs(want)
        want = (loss(xv, wv + u) - loss(xv, wv - u)) / 2
        got = float((dw.double().cpu() * u).sum())
        assert abs(got - want) <= m * U * float((dy.abs().double().T @ xv.abs() * u.abs()).sum()) + 1e-9 * abs(want)


def test_runs_are_identical(hip):
    args, _, _ = _linear_case(hip, 300, 520, 1152, "tiles", seed=1)
    first = hip.linear_fp8(*args)
    for _ in range(3):
        assert torch.equal(hip.linear_fp8(*args), first)


def test_outputs_leave_their_surroundings(hip):
    """Codes, scales and Y written into the middle of larger buffers."""
    m, n, k = 37, 45, 200
    x = _x(m, k, 1).cuda()
    sc = torch.full((m + 2, 8), 99, dtype=torch.uint8, device="cuda")
    cd = torch.full((m + 2, 256), 99, dtype=torch.uint8, device="cuda")
    codes, scales = hip.quantize_fp8(x, codes=cd[1:-1].view(torch.float8_e4m3fn),
                                     scales=sc[1:-1].view(torch.float8_e8m0fnu)[:, :2])
    _check_quantized(x.cpu(), codes, scales, 1)
    assert bool((cd[[0, -1]] == 99).all()) and bool((sc[[0, -1]] == 99).all()) and bool((sc[:, 2:] == 99).all())
    w = hip.quantize_fp8(_x(n, k, 2).cuda(), block_rows=128)
    for rows in (m, 200):
        xq = hip.quantize_fp8(_x(rows, k, 1).cuda())
        buf = torch.full(((rows + 2) * n + 64,), 99.0, device="cuda")
        y = buf[64:64 + rows * n].view(rows, n)
        hip.linear_fp8(*xq, *w, y=y)
        _check_product(y, ref64.fp8_values(_bytes(xq[0]), _bytes(xq[1])),
                       ref64.fp8_values(_bytes(w[0]), _bytes(w[1]), 128))
        assert bool((buf[:64] == 99).all()) and bool((buf[64 + rows * n:] == 99).all())


def test_stream_of_its_own(hip):
    s = torch.cuda.Stream()
    x = _x(300, 640, 1).cuda()
    w = hip.quantize_fp8(_x(200, 640, 2).cuda(), block_rows=128)
    want = hip.linear_fp8(*hip.quantize_fp8(x), *w)
    torch.cuda.synchronize()
    for _ in range(20):
        xq = hip.quantize_fp8(x, stream=s)
        y = hip.linear_fp8(*xq, *w, stream=s)
        del xq
    s.synchronize()
    assert torch.equal(y, want)


@pytest.mark.parametrize("m,n,k,dtype", [(4100, 4196, 4097, torch.bfloat16), (4224, 4096, 4099, torch.float32),
                                         (2100, 2200, 2111, torch.bfloat16), (2176, 2200, 2112, torch.float32),
                                         (1400, 1300, 1500, torch.bfloat16), (1401, 1300, 1501, torch.float32),
                                         (500, 450, 300, torch.bfloat16), (70, 33, 129, torch.float32)])
def test_linear_backward_in_one_launch(hip, m, n, k, dtype):
    """Both products by one kernel (each kind of tile): the same as one by one."""
    g = torch.Generator(device="cuda").manual_seed(5)
    dy = (1e-3 * torch.randn((m, n), generator=g, device="cuda")).to(dtype)
    xt = hip.quantize_fp8(torch.randn((m, k), generator=g, device="cuda"), transposed=True)
    wt = hip.quantize_fp8(0.02 * torch.randn((n, k), generator=g, device="cuda"), block_rows=128, transposed=True)
    dx, dw = hip.linear_fp8_backward(dy, *xt, *wt)
    codes, scales, codes_t, scales_t = hip.quantize_fp8_both(dy)
    assert torch.equal(dx, hip.linear_fp8(codes, scales, *wt, y_dtype=dtype))
    assert torch.equal(dw, hip.linear_fp8(codes_t, scales_t, *xt))
    rows = torch.tensor([0, 31, 64, m // 4, m // 2, m - 1])
    _check_product(dx[rows.cuda()], ref64.fp8_values(_bytes(codes), _bytes(scales))[rows],
                   ref64.fp8_values(_bytes(wt[0]), _bytes(wt[1]), 128))
    rows = torch.tensor([0, 32, n // 4, n // 2 - 1, n - 1])
    _check_product(dw[rows.cuda()], ref64.fp8_values(_bytes(codes_t), _bytes(scales_t))[rows],
                   ref64.fp8_values(_bytes(xt[0]), _bytes(xt[1])))
