"""The 8-bit linear layer on the GPU where its kernels and formats end: the largest
grids, exact sums, extreme scales, rounding next to ties."""
import pytest
import torch

import fp8_cases
import ref64
from test_gpu_fp8 import _check_product, _linear_case

pytestmark = pytest.mark.gpu

U = 2.0 ** -24  # half a step of fp32
F8, E8 = torch.float8_e4m3fn, torch.float8_e8m0fnu


def _bytes(t):
    return t.contiguous().view(torch.uint8).cpu()


@pytest.mark.parametrize("n", [(1 << 26) - 16, (1 << 26) - 15, (1 << 26) - 1])
def test_linear_few_rows_up_to_the_largest_grid(hip, n):
    """The last column count of the kernel for few rows (2^22 - 1 workgroups of 1024
    threads), and the first ones that take tiles. Small whole numbers: the sums are
    exact in either output type."""
    m = 3
    wc = torch.zeros((n, 128), dtype=torch.uint8, device="cuda")
    wc[:, 5] = 0x38 + (torch.arange(n, device="cuda") % 5 * 8).to(torch.uint8)  # 1, 2, 4, 8, 16
    xc = torch.zeros((m, 128), dtype=torch.uint8, device="cuda")
    xc[:, 5] = torch.tensor([0x38, 0x40, 0xC0], dtype=torch.uint8)  # 1, 2, -2
    xs = torch.full((m, 4), 127, dtype=torch.uint8, device="cuda")
    ws = torch.full(((n + 127) // 128, 4), 127, dtype=torch.uint8, device="cuda")
    y = hip.linear_fp8(xc.view(F8), xs.view(E8)[:, :1], wc.view(F8), ws.view(E8)[:, :1], y_dtype=torch.bfloat16)
    want = torch.exp2((torch.arange(n, device="cuda") % 5).float()).to(torch.bfloat16)
    assert torch.equal(y, torch.stack([want, 2 * want, -2 * want]))


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_more_row_tiles_than_a_grid(hip, block_rows):
    """The most rows there are, of one column: 2^24 row tiles, over several launches."""
    rows = (1 << 31) - 1
    x = torch.zeros((rows, 1), dtype=torch.bfloat16, device="cuda")
    at = torch.tensor([0, 127, 128, (1 << 30) - 1, 1 << 30, (1 << 30) + 1, rows - 128, rows - 2, rows - 1])
    vals = torch.tensor([1.0, -2.0, 3.0, 448.0, 0.5, -7.0, 5.0, 1.5, -0.375], dtype=torch.bfloat16)
    x[at.cuda(), 0] = vals.cuda()
    codes, scales = hip.quantize_fp8(x, block_rows=block_rows, transposed=True)
    want = torch.zeros(rows, dtype=torch.bfloat16, device="cuda")
    want[at.cuda()] = vals.cuda()
    for t in sorted({int(i) // 128 for i in at}):
        part = slice(128 * t, min(128 * t + 128, rows))
        rc, rs = ref64.fp8_quantize(want[part][None].cpu(), block_rows)
        assert torch.equal(_bytes(codes[:, 128 * t:128 * t + 128]), rc)
        assert torch.equal(_bytes(scales[:, t:t + 1]), rs)
    # everything else is zero
    assert int(torch.count_nonzero(codes.view(torch.uint8).view(torch.int64))) == len(
        {int(i) // 8 for i in at})
    assert int(torch.count_nonzero(scales.contiguous().view(torch.uint8))) == len({int(i) // 128 for i in at})


def _nearest_bf16(v):
    """float64 v at the nearest bf16 value (ties to even), as float64."""
    step = torch.exp2((torch.frexp(v)[1].clamp(min=-125) - 8).double())
    return torch.round(v / step) * step


@pytest.mark.parametrize("power", [0, -100, -122, -126, -131, -135, 100])
def test_dequantize_rounds_once(hip, power):
    """Every code times float32 scales that bring products next to the middle between two
    bf16 values (also where they are subnormal): the nearest one, of the exact product."""
    blocks = 512
    g = torch.Generator().manual_seed(3)
    middle = (2 * torch.randint(128, 256, (blocks,), generator=g) + 1).double()
    code = torch.randint(8, 16, (blocks,), generator=g).double()
    s = (middle / code).float().view(torch.int32) + torch.randint(-2, 3, (blocks,), generator=g, dtype=torch.int32)
    s = (s.view(torch.float32) * 2.0 ** power)[None]
    s[0, 0] = (0x815555 / 2 ** 23) * 2.0 ** power  # times 1.125 just above a middle
    codes = torch.arange(256, dtype=torch.uint8).view(2, 128).repeat(1, blocks)
    want = ref64.fp8_values(codes, s, 128)
    for out, rounded in ((torch.bfloat16, _nearest_bf16(want)), (torch.float32, want.float().double())):
        got = hip.dequantize_fp8(codes.cuda().view(F8), s.cuda(), out_dtype=out).double().cpu()
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(rounded)), power


def _extreme(m, n, k, side, byte, codes, seed):
    """x and w codes and E8M0 bytes: `byte` for one side's every block, the other's such
    that sums are ordinary numbers; and the 64-bit product. Whole numbers of one unit:
    every sum of up to 2^24 units is exact in fp32, in any order."""
    g = torch.Generator().manual_seed(seed)
    few = torch.tensor(codes, dtype=torch.uint8)[torch.randint(0, len(codes), ((m if side == "x" else n), k), generator=g)]
    small = torch.tensor([0, 0x38, 0x40, 0xC0], dtype=torch.uint8)  # 0, 1, 2, -2
    other = small[torch.randint(0, 4, ((n if side == "x" else m), k), generator=g)]
    kp = (k // 128 + 3) // 4 * 4
    back = 200 if byte < 127 else 20
    one = lambda rows, b: torch.full((rows, kp), b, dtype=torch.uint8)
    if side == "x":
        return few, one(m, byte), other, one(n, back)
    return other, one(m, back), few, one(n, byte)


TILES = [(3, 40, 256), (20, 70, 384), (300, 96, 4224), (1408, 1536, 128), (2176, 2304, 128), (2048, 5248, 128)]


@pytest.mark.parametrize("side", ["x", "w"])
@pytest.mark.parametrize("byte", [0, 1, 2, 3, 4, 246, 247])
@pytest.mark.parametrize("m,n,k", TILES)
def test_linear_extreme_scales(hip, m, n, k, byte, side):
    """Every kernel, one operand at either end of E8M0: its smallest codes (k 2^-9) under the
    lowest scales, its largest under the highest (up to 240 under 247: 2^128 - 2^124)."""
    codes = [0, 1, 2, 3, 7, 0x83] if byte < 127 else [0, 0x70, 0x74, 0x77, 0xF7] + ([0x7C, 0x7E] if byte < 247 else [])
    xc, xs, wc, ws = _extreme(m, n, k, side, byte, codes, byte)
    kb = k // 128
    rows = torch.tensor([0, 1, m // 2, m - 1])
    xv, wv = ref64.fp8_values(xc[rows], xs[rows, :kb]), ref64.fp8_values(wc, ws[:, :kb])
    want, size = xv @ wv.T, xv.abs() @ wv.abs().T
    # bytes 0 to 2: the operand is off by half of 2^-133 at most
    off = torch.zeros_like(want)
    if byte < 3:
        off = 2.0 ** -134 * (wv.abs().sum(1)[None, :] if side == "x" else xv.abs().sum(1)[:, None]).expand_as(want)
    xd, xsd, wd, wsd = xc.cuda().view(F8), xs.cuda().view(E8)[:, :kb], wc.cuda().view(F8), ws.cuda().view(E8)[:, :kb]
    kinds = [wsd]
    if side == "x" and byte < 127:  # float32 scales come after a block's sum, which has to stay in range
        kinds.append(torch.full(((n + 127) // 128, kb), 2.0 ** (int(ws[0, 0]) - 127), device="cuda"))
    for w_scales in kinds:
        y = hip.linear_fp8(xd, xsd, wd, w_scales)[rows.cuda()].double().cpu()
        assert bool(((y - want).abs() <= off).all()), (byte, side, w_scales.dtype, float(((y - want).abs() / size).max()))
        y = hip.linear_fp8(xd, xsd, wd, w_scales, y_dtype=torch.bfloat16)[rows.cuda()].double().cpu()
        tol = 7 * 2.0 ** -13 * size * (1 + 2.0 ** -8) + 2.0 ** -8 * want.abs()
        assert bool(((y - want).abs() <= tol).all()), (byte, side, "bf16")


@pytest.mark.parametrize("kind", ["tiles", "rows", "f32"])
@pytest.mark.parametrize("m,n,k", fp8_cases.KERNELS)
def test_linear_float32_sums_are_exact(hip, m, n, k, kind):
    """Every kernel: runs of products that cancel but for small ones. fp32 sums hold them
    exactly (tests/test_fp8_cases.py: the fp8 instructions would keep none); a bf16 Y is
    within what those may lose."""
    x, w = fp8_cases.cancelling(m, n, k)
    kb, kp, tiles = k // 128, (k // 128 + 3) // 4 * 4, (n + 127) // 128
    one = lambda rows: torch.full((rows, kp), 127, dtype=torch.uint8, device="cuda").view(E8)[:, :kb]
    ws = {"tiles": one(tiles), "rows": one(n), "f32": torch.ones((tiles, kb), device="cuda")}[kind]
    rows = torch.tensor([0, 1, 2, m // 2, m - 2, m - 1])
    xv, wv = fp8_cases.values(x[rows]), fp8_cases.values(w)
    want = xv @ wv.T
    xd, wd = x.cuda().view(F8), w.cuda().view(F8)
    y = hip.linear_fp8(xd, one(m), wd, ws)[rows.cuda()].double().cpu()
    assert torch.equal(y, want)
    y = hip.linear_fp8(xd, one(m), wd, ws, y_dtype=torch.bfloat16)[rows.cuda()].double().cpu()
    assert bool(((y - want).abs() <= 7 * 2.0 ** -13 * (xv.abs() @ wv.abs().T)).all())


@pytest.mark.parametrize("m,n,k", [(70, 300, 513), (1400, 1300, 257), (2176, 2300, 257), (4224, 4096, 257)])
def test_backward_float32_sums_are_exact(hip, m, n, k):
    """dX in float32 from a dY whose runs of 8 along n cancel against W^T's."""
    np_ = (n + 127) // 128 * 128
    dy, wt = fp8_cases.cancelling(m, k, np_)
    dy = fp8_cases.values(dy)[:, :n].float()
    wt[:, n:] = 0
    unit = torch.full(((k + 127) // 128, (np_ // 128 + 3) // 4 * 4), 127, dtype=torch.uint8, device="cuda")
    xt = hip.quantize_fp8(torch.ones((m, k), device="cuda"), transposed=True)
    # 256 is each block's largest: dY's own scales are 1 and its codes exact
    dx, _ = hip.linear_fp8_backward(dy.cuda(), *xt, wt.cuda().view(F8), unit.view(E8)[:, :np_ // 128])
    rows = torch.tensor([0, 1, m // 2, m - 1])
    assert torch.equal(dx[rows.cuda()].double().cpu(), dy[rows].double() @ fp8_cases.values(wt)[:, :n].T)


@pytest.mark.parametrize("kind", ["tiles", "rows", "f32"])
@pytest.mark.parametrize("m,n,k", [(301, 701, 4224), (17, 3, 8192), (301, 701, 13824), (650, 330, 4224),
                                   (1408, 1536, 256), (1409, 1535, 384), (2176, 2304, 256), (2177, 2303, 384),
                                   (2049, 5003, 256)])
def test_linear_both_types_by_every_kernel(hip, m, n, k, kind):
    """K split with an odd count of results, and every tile kernel, to both types."""
    args, xv, wv = _linear_case(hip, m, n, k, kind, seed=3)
    rows = torch.tensor([0, 1, 2, 15, 16, m // 2, m - 2, m - 1])
    for out in (torch.float32, torch.bfloat16):
        _check_product(hip.linear_fp8(*args, y_dtype=out)[rows.cuda()], xv[rows], wv)


@pytest.mark.parametrize("x_byte,w_byte", [(0, 127), (1, 200), (2, 120), (127, 0), (0, 254), (254, 0), (254, 1), (1, 254),
                                           (247, 20), (130, 3), (127, 127)])
@pytest.mark.parametrize("m,n,k", [(1, 130, 384), (3, 41, 5120), (16, 300, 640)])
def test_linear_few_rows_are_exact_under_every_scale(hip, m, n, k, x_byte, w_byte):
    """Up to 16 rows: runs of products that cancel but for small ones, at every end of
    E8M0. float32: the exact sum; bfloat16: the nearest value to it."""
    x, w = fp8_cases.cancelling(m, n, k)
    kb, kp, tiles = k // 128, (k // 128 + 3) // 4 * 4, (n + 127) // 128
    scales = lambda rows, b: torch.full((rows, kp), b, dtype=torch.uint8, device="cuda").view(E8)[:, :kb]
    want = (fp8_cases.values(x) @ fp8_cases.values(w).T) * 2.0 ** (x_byte - 127) * 2.0 ** (w_byte - 127)
    kinds = [scales(tiles, w_byte), scales(n, w_byte)]
    if 3 <= w_byte <= 253:
        kinds.append(torch.full((tiles, kb), 2.0 ** (w_byte - 127), device="cuda"))
    for ws in kinds:
        for out in (torch.float32, torch.bfloat16):
            y = hip.linear_fp8(x.cuda().view(F8), scales(m, x_byte), w.cuda().view(F8), ws, y_dtype=out)
            assert torch.equal(y.double().cpu(), want if out == torch.float32 else _nearest_bf16(want)), (ws.shape, out)


@pytest.mark.parametrize("m", [1, 16])
def test_linear_few_rows_differing_scales(hip, m):
    """Every column and block under a scale of its own, also beside others that are NaN."""
    n, k = 37, 1280
    g = torch.Generator().manual_seed(m)
    xc = torch.randint(0, 120, (m, k), generator=g, dtype=torch.uint8)
    wc = torch.randint(0, 120, (n, k), generator=g, dtype=torch.uint8)
    xs = torch.randint(60, 190, (m, 12), generator=g, dtype=torch.uint8)
    ws = torch.randint(60, 190, (n, 12), generator=g, dtype=torch.uint8)
    xv, wv = ref64.fp8_values(xc, xs[:, :10]), ref64.fp8_values(wc, ws[:, :10])
    args = xc.cuda().view(F8), xs.cuda().view(E8)[:, :10], wc.cuda().view(F8)
    # scales up to 2^62 each: some columns' sums of up to 2^124 448^2 1280 leave fp32's range
    inside = (xv.abs() @ wv.abs().T).amax(0) < 2.0 ** 127
    assert int(inside.sum()) >= n // 2
    for out in (torch.float32, torch.bfloat16):
        y = hip.linear_fp8(*args, ws.cuda().view(E8)[:, :10], y_dtype=out).cpu()
        _check_product(y[:, inside], xv, wv[inside])
    bad = ws.clone()
    bad[5, 3] = 255
    y = hip.linear_fp8(*args, bad.cuda().view(E8)[:, :10]).cpu()
    assert bool(torch.isnan(y[:, 5]).all())
    inside[5] = False
    _check_product(y[:, inside], xv, wv[inside])


def test_offsets_beyond_32_bits(hip):
    """More than 2^31 elements of x, of codes both ways, and of Y."""
    rows, k = 270001, 8192
    x = torch.zeros((rows, k), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator().manual_seed(6)
    last = torch.randn((300, k), generator=g).to(torch.bfloat16).cuda()
    x[-300:] = last
    codes, scales, codes_t, scales_t = hip.quantize_fp8_both(x)
    c2, s2 = hip.quantize_fp8(last)
    assert torch.equal(codes[-300:].view(torch.uint8), c2.view(torch.uint8))
    assert torch.equal(scales[-300:].view(torch.uint8), s2.view(torch.uint8))
    tail = rows // 128 * 128  # the last block along the rows, 49 of them
    t2, u2 = hip.quantize_fp8(x[tail:], transposed=True)
    assert torch.equal(codes_t[:, tail:].contiguous().view(torch.uint8), t2.view(torch.uint8))
    assert torch.equal(scales_t[:, -1:].contiguous().view(torch.uint8), u2.contiguous().view(torch.uint8))
    back = hip.dequantize_fp8(codes, scales, out_dtype=torch.bfloat16)
    assert torch.equal(back[-300:], hip.dequantize_fp8(c2, s2, out_dtype=torch.bfloat16))
    del back, codes_t, scales_t, x
    n = 8000
    wq = hip.quantize_fp8(torch.randn((n, k), generator=g).cuda(), block_rows=128)
    for out in (torch.bfloat16, torch.float32):
        y = hip.linear_fp8(codes, scales, *wq, y_dtype=out)
        assert y.numel() > 1 << 31 and not bool(y[:-300].any())
        xv = ref64.fp8_values(_bytes(c2[:3]), _bytes(s2[:3]))
        _check_product(y[-300:-297], xv, ref64.fp8_values(_bytes(wq[0]), _bytes(wq[1]), 128))
        assert torch.equal(y[-256:], hip.linear_fp8(codes[-8192:], scales[-8192:], *wq, y_dtype=out)[-256:])
        del y


@pytest.mark.parametrize("power,x_byte", [(-90, 82), (-95, 79), (-126, 247), (-140, 200), (120, 27), (126, 1), (-60, 60), (0, 127)])
@pytest.mark.parametrize("m", [1, 16])
def test_linear_few_rows_float_scales_of_any_size(hip, m, power, x_byte):
    """Float32 weight scales whose product with X's leaves the normal numbers, while the
    results do not: only the results have to be in range."""
    n, k = 300, 640
    g = torch.Generator().manual_seed(m)
    xc = torch.randint(0, 120, (m, k), generator=g, dtype=torch.uint8)
    wc = torch.randint(0, 120, (n, k), generator=g, dtype=torch.uint8)
    xs = torch.full((m, 8), x_byte, dtype=torch.uint8)
    s32 = ((1 + torch.rand((3, 5), generator=g)).double() * 2.0 ** power).float()
    xv, wv = ref64.fp8_values(xc, xs[:, :5]), ref64.fp8_values(wc, s32, 128)
    size = xv.abs() @ wv.abs().T
    # (additions below 2^-126 are exact: U times a size above it counts every rounding)
    assert 2.0 ** -126 < float(size.min()) and float(size.max()) < 2.0 ** 127
    args = xc.cuda().view(F8), xs.cuda().view(E8)[:, :5], wc.cuda().view(F8), s32.cuda()
    for out in (torch.float32, torch.bfloat16):
        y = hip.linear_fp8(*args, y_dtype=out)
        want = xv @ wv.T
        # k additions, a rounding a block, one of the result: nothing is cut for either type
        tol = (k + k // 128 + 1) * U * size
        if out == torch.bfloat16:
            tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * want.abs()
        assert bool(((y.double().cpu() - want).abs() <= tol).all()), out
