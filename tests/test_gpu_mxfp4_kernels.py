"""Every kernel of the 4-bit products in every mode, at sizes that reach it (tests/mx4_cases.py;
tests/test_mxfp4_choices.py holds the choice of a kernel to them): within the bound that counts
the fp32 additions, exactly where every sum is representable, with every scale byte, and with
nothing written beside the result."""
import pytest
import torch

import mx4_cases
import mx4_ref

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float32]
GUARD = 4096  # elements before and behind a result: 16-byte aligned


def _random(rows, k, seed, lo=119, hi=135):
    """Code and scale bytes, scales in lo .. hi."""
    g = torch.Generator().manual_seed(seed)
    return (torch.randint(0, 256, (rows, k // 2), generator=g, dtype=torch.uint8),
            torch.randint(lo, hi + 1, (rows, k // 32), generator=g).to(torch.uint8))


def _experts(count, n, k, seed, lo=119, hi=135):
    c = [_random(n, k, seed + 10 * e, lo, hi) for e in range(count)]
    return torch.stack([a for a, _ in c]), torch.stack([b for _, b in c])


def _cuda(c):
    return c[0].cuda(), c[1].cuda().view(torch.float8_e8m0fnu)


def _x(rows, k, seed, dtype, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((rows, k), generator=g) * torch.exp(spread * torch.randn((1, k), generator=g))).to(dtype)


def _near(y, xv, wv, what):
    """Within the fp32 additions of a product: 64 parts of K at most (a split has 16 stages or more a part, so
    8 of them at k = 2^15, and a workgroup's are counted by the bound itself)."""
    ref, s = xv @ wv.T, xv.abs() @ wv.abs().T
    err = (y.double().cpu() - ref).abs()
    tol = mx4_ref.bound(xv.shape[1], s, y.dtype, 64)
    assert bool((err <= tol).all()), (what, tuple(y.shape), y.dtype, float((err / tol).max()))


class _Guarded:
    """A result [m][n] between elements that have to keep their value."""

    def __init__(self, m, n, dtype):
        self.held = torch.full((m * n + 2 * GUARD,), 3.0, dtype=dtype, device="cuda")
        self.y = self.held[GUARD:GUARD + m * n].view(m, n)

    def check(self):
        torch.cuda.synchronize()
        assert bool((self.held[:GUARD] == 3).all()) and bool((self.held[-GUARD:] == 3).all())


def _cases(cases):
    return pytest.mark.parametrize("case", cases, ids=mx4_cases.case_ids(cases))


def _exact_scales(k):
    """Scale bytes whose products are multiples of 2^-6 (0.25 by 2^-4) and whose sums of magnitudes stay
    below 2^18 (at most 36 * 2^4 of k <= 2^14 products at 36 / 4 in the mean): every partial sum, in any
    order, is a multiple of 2^-6 below 2^18, so fp32 holds it."""
    assert k <= 1 << 14
    return 125, 126


# ---------------------------------------------------------------- one weight


@pytest.mark.parametrize("y_dtype", DTYPES)
@_cases(mx4_cases.LINEAR)
def test_linear(hip, case, y_dtype):
    _, m, n, k = case
    x, w = _random(m, k, seed=m + k), _random(n, k, seed=n + k + 1)
    g = _Guarded(m, n, y_dtype)
    hip.linear_mxfp4(*_cuda(x), *_cuda(w), y_dtype=y_dtype, y=g.y)
    g.check()
    _near(g.y, mx4_ref.values(*x), mx4_ref.values(*w), case)


@_cases(mx4_cases.LINEAR)
def test_linear_exact_sums(hip, case):
    _, m, n, k = case
    lo, hi = _exact_scales(k)
    x, w = _random(m, k, m + k + 5, lo, hi), _random(n, k, n + k + 6, lo, hi)
    xv, wv = mx4_ref.values(*x), mx4_ref.values(*w)
    assert float((xv.abs() @ wv.abs().T).max()) < 2.0 ** 18
    ref = xv @ wv.T
    xd, wd = _cuda(x), _cuda(w)
    assert torch.equal(hip.linear_mxfp4(*xd, *wd).double().cpu(), ref)
    assert torch.equal(hip.linear_mxfp4(*xd, *wd, y_dtype=torch.bfloat16).cpu(), ref.float().to(torch.bfloat16))


@_cases([c for c in mx4_cases.LINEAR if c[3] <= 2304])
def test_linear_keeps_small_products_beside_large_ones_that_cancel(hip, case):
    """In every run of 8 along k 36 2^12 and -36 2^12, next to each other, beside six products of 2^10, or
    all of these 2^-12 of that. The large ones' pairs cancel wherever a sum ends between two pairs; inside,
    at most 16 pairs of an instruction are open, 2^21.2, beside 2304 * 3 / 4 * 2^10 = 2^20.8 of the small: below
    2^22, so multiples of 2^-2 are exact in fp32."""
    _, m, n, k = case
    x, w = _random(m, k, 1, 127, 127), _random(n, k, 2, 127, 127)
    for c, large in ((x, 0x77), (w, 0xF7)):
        c[0][:] = (c[0] & 0x88) | 0x11
        c[0][:, ::4] = large
    big = torch.zeros(k // 32, dtype=torch.bool)
    big[::2] = True
    x[1][:, big] = 133
    w[1][:, big] = 133
    want = mx4_ref.values(*x) @ mx4_ref.values(*w).T
    assert bool(want.any())
    assert torch.equal(hip.linear_mxfp4(*_cuda(x), *_cuda(w)).double().cpu(), want)


@_cases(mx4_cases.LINEAR)
def test_linear_every_scale_byte(hip, case):
    """Scales 0 to 254 whose products stay in range; NaN where one is 255, and nowhere else."""
    _, m, n, k = case
    x, w = _random(m, k, 1, 127, 127), _random(n, k, 2, 127, 127)
    b = torch.arange(k // 32) * 254 // max(k // 32 - 1, 1)
    x[1][:] = b.to(torch.uint8)
    w[1][:] = (254 - b).to(torch.uint8)
    # products are multiples of 0.25, at most 36: sums below 2^19 of k <= 2^14
    want = mx4_ref.values(*x) @ mx4_ref.values(*w).T
    assert torch.equal(hip.linear_mxfp4(*_cuda(x), *_cuda(w)).double().cpu(), want)
    x[1][m - 1, k // 32 - 1] = 255  # the last block
    x[1][m // 2, 3] = 255
    w[1][n - 1, 0] = 255
    w[1][n // 3, k // 32 - 1] = 255
    for dtype in DTYPES:
        y = hip.linear_mxfp4(*_cuda(x), *_cuda(w), y_dtype=dtype).double().cpu()
        bad = torch.zeros((m, n), dtype=torch.bool)
        bad[[m - 1, m // 2], :] = True
        bad[:, [n - 1, n // 3]] = True
        assert torch.equal(torch.isnan(y), bad)
        assert torch.equal(y[~bad], want.float().to(dtype).double()[~bad])


@_cases([c for c in mx4_cases.LINEAR if c[0][0] in (mx4_cases.T256, mx4_cases.T128)])
def test_linear_does_not_change_from_run_to_run(hip, case):
    _, m, n, k = case
    x, w = _cuda(_random(m, k, 1)), _cuda(_random(n, k, 2))
    first = hip.linear_mxfp4(*x, *w)
    for _ in range(3):
        assert torch.equal(hip.linear_mxfp4(*x, *w), first)


@_cases([c for c in mx4_cases.LINEAR if c[3] <= 1152])
def test_linear_sums_beyond_the_range_are_not_finite(hip, case):
    """Products of 2^122 to 2^127.2 whose sums pass 2^128: infinite, or NaN where parts of either sign meet; a
    row and a column of zeros stay zero beside them."""
    _, m, n, k = case
    x, w = _random(m, k, 1, 189, 189), _random(n, k, 2, 187, 187)
    x[0][0], w[0][n - 1] = 0, 0
    want = mx4_ref.values(*x) @ mx4_ref.values(*w).T
    past = want.abs() >= 2.0 ** 128
    assert bool(past.any()) or m == 1
    for dtype in DTYPES:
        y = hip.linear_mxfp4(*_cuda(x), *_cuda(w), y_dtype=dtype).float().cpu()
        assert not bool(torch.isfinite(y[past]).any())
        assert not y[0].any() and not y[:, n - 1].any()


# ---------------------------------------------------------------- a weight for each group of rows


def _groups(offsets):
    return list(enumerate(zip(offsets[:-1], offsets[1:])))


@pytest.mark.parametrize("y_dtype", DTYPES)
@_cases(mx4_cases.GROUPED)
def test_grouped(hip, case, y_dtype):
    _, rows, offsets, n, k = case
    x, w = _random(rows, k, rows), _experts(len(offsets) - 1, n, k, 7)
    g = _Guarded(rows, n, y_dtype)
    hip.linear_mxfp4_grouped(*_cuda(x), *_cuda(w), torch.tensor(offsets, device="cuda"), y_dtype=y_dtype, y=g.y)
    g.check()
    xv = mx4_ref.values(*x)
    for e, (b, t) in _groups(offsets):
        if t > b:
            _near(g.y[b:t], xv[b:t], mx4_ref.values(w[0][e], w[1][e]), (case, e))
    assert bool((g.y[:offsets[0]] == 3).all()) and bool((g.y[offsets[-1]:] == 3).all())


@_cases(mx4_cases.GROUPED)
def test_grouped_exact_sums_and_nan_scales(hip, case):
    _, rows, offsets, n, k = case
    lo, hi = _exact_scales(k)
    x, w = _random(rows, k, rows + 1, lo, hi), _experts(len(offsets) - 1, n, k, 9, lo, hi)
    xv = mx4_ref.values(*x)
    want = torch.full((rows, n), 3.0, dtype=torch.float64)
    for e, (b, t) in _groups(offsets):
        want[b:t] = xv[b:t] @ mx4_ref.values(w[0][e], w[1][e]).T
    off = torch.tensor(offsets, device="cuda")
    y = torch.full((rows, n), 3.0, device="cuda")
    hip.linear_mxfp4_grouped(*_cuda(x), *_cuda(w), off, y=y)
    assert torch.equal(y.double().cpu(), want)
    # the last row of the last group and, of the first group's weight, the last row: those alone
    first, last = next(e for e, (b, t) in _groups(offsets) if t > b), offsets[-1] - 1
    x[1][last, k // 32 - 1] = 255
    w[1][first, n - 1, 0] = 255
    bad = torch.zeros((rows, n), dtype=torch.bool)
    bad[last] = True
    bad[offsets[first]:offsets[first + 1], n - 1] = True
    y = torch.full((rows, n), 3.0, dtype=torch.bfloat16, device="cuda")
    hip.linear_mxfp4_grouped(*_cuda(x), *_cuda(w), off, y_dtype=torch.bfloat16, y=y)
    y = y.cpu()
    assert torch.equal(torch.isnan(y), bad)
    assert torch.equal(y[~bad], want.float().to(torch.bfloat16)[~bad])


# ---------------------------------------------------------------- gradients


_q = mx4_cases.rounded


class _C:
    """One gradient or both by the C entry points, whose other one is NULL."""

    def __init__(self, hip, dy, xt, wt, n, k, which, off=None):
        m, g = dy.shape[0], 0 if off is None else off.numel() - 1
        lead = () if off is None else (g,)
        self.dx = _Guarded(m, k, dy.dtype) if which & 1 else None
        self.dw = _Guarded(lead[0] * n if lead else n, k, torch.float32) if which & 2 else None
        L, st = hip.lib(), torch.cuda.current_stream().cuda_stream
        need = (L.hif4_linear_mxfp4_backward_workspace_bytes(m, n, k) if off is None
                else L.hif4_linear_mxfp4_grouped_backward_workspace_bytes(g, m, n, k))
        ws = torch.empty((need,), dtype=torch.uint8, device="cuda")
        p = lambda t: None if t is None else t.data_ptr()  # noqa: E731
        dt = {torch.float32: 0, torch.bfloat16: 1}[dy.dtype]
        xt, wt = xt if which & 2 else (None, None), wt if which & 1 else (None, None)
        args = [p(dy), dt, dy.stride(0), p(xt[0]), p(xt[1]), p(wt[0]), p(wt[1])]
        out = [p(self.dx.y if which & 1 else None), dt, p(self.dw.y if which & 2 else None), 0, p(ws), need, st]
        if off is None:
            assert L.hif4_linear_mxfp4_backward(*args, m, n, k, *out) == 0
        else:
            assert L.hif4_linear_mxfp4_grouped_backward(*args, p(off), g, m, n, k, *out) == 0
        for t in (self.dx, self.dw):
            if t is not None:
                t.check()


@pytest.mark.parametrize("dtype", DTYPES)
@_cases(mx4_cases.BACKWARD)
def test_backward(hip, case, dtype):
    _, m, n, k, which = case
    dy, x, w = _x(m, n, 1, dtype), _x(m, k, 2, dtype), _x(n, k, 3, dtype, 0.2)
    xt, wt = hip.quantize_mxfp4(x.cuda(), transposed=True), hip.quantize_mxfp4(w.cuda(), transposed=True)
    got = _C(hip, dy.cuda(), xt, wt, n, k, which)
    if which & 1:
        _near(got.dx.y, _q(dy), _q(w.T.contiguous()), case)
    if which & 2:
        _near(got.dw.y, _q(dy.T), _q(x.T.contiguous()), case)


@pytest.mark.parametrize("dtype", DTYPES)
@_cases(mx4_cases.GROUPED_BACKWARD)
def test_grouped_backward(hip, case, dtype):
    _, rows, offsets, n, k, which = case
    groups = len(offsets) - 1
    off = torch.tensor(offsets, device="cuda")
    dy, x = _x(rows, n, 1, dtype), _x(rows, k, 2, dtype)
    w = torch.stack([_x(n, k, 3 + e, dtype, 0.2) for e in range(groups)])
    xt = hip.quantize_mxfp4(x.cuda(), transposed=True, offsets=off)
    wt = hip.quantize_mxfp4(w.cuda(), transposed=True)
    got = _C(hip, dy.cuda(), xt, wt, n, k, which, off)
    for e, (b, t) in _groups(offsets):
        if which & 1 and t > b:
            _near(got.dx.y[b:t], _q(dy[b:t]), _q(w[e].T.contiguous()), (case, e))
        if which & 2:
            dw = got.dw.y[e * n:(e + 1) * n]
            if t > b:
                _near(dw, _q(dy[b:t].T), _q(x[b:t].T.contiguous()), (case, e))
            else:
                assert not dw.any()
    if which & 1:
        assert bool((got.dx.y[:offsets[0]] == 3).all()) and bool((got.dx.y[offsets[-1]:] == 3).all())


@pytest.mark.parametrize("groups", [False, True])
def test_one_gradient_by_the_binding(hip, groups):
    """The gradient that is asked for, as the C entry point gives it, without the other's operands."""
    m, n, k = 300, 333, 200
    off = torch.tensor([3, 100, 100, 299], device="cuda") if groups else None
    dy = torch.nn.functional.pad(_x(m, n, 1, torch.bfloat16), (2, 3)).cuda()[:, 2:2 + n]  # rows of its own stride
    xt = hip.quantize_mxfp4(_x(m, k, 2, torch.bfloat16).cuda(), transposed=True, offsets=off)
    w = torch.stack([_x(n, k, 3 + e, torch.float32, 0.2) for e in range(3)]).cuda()
    wt = hip.quantize_mxfp4(w if groups else w[0], transposed=True)
    call = hip.linear_mxfp4_grouped_backward if groups else hip.linear_mxfp4_backward
    tail = (off,) if groups else ()
    rows = slice(3, 299) if groups else slice(0, m)
    dx, dw = call(dy, None, None, *wt, *tail, need_dw=False)
    assert dw is None and torch.equal(dx[rows], _C(hip, dy, xt, wt, n, k, 1, off).dx.y[rows])
    dx, dw = call(dy, *xt, None, None, *tail, dw_dtype=torch.float32, need_dx=False)
    assert dx is None and torch.equal(dw.flatten(0, -2), _C(hip, dy, xt, wt, n, k, 2, off).dw.y)
    both = call(dy, *xt, *wt, *tail)
    want = _C(hip, dy, xt, wt, n, k, 3, off)
    assert torch.equal(both[0][rows], want.dx.y[rows]) and torch.equal(both[1].flatten(0, -2), want.dw.y)
