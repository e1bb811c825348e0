"""Refusals and size queries of the 4-bit microscaled layers, on the CPU: the C entry points
return their documented status before any device work, the binding raises before any call."""
import os

import pytest
import torch

OK, NULL, SHAPE, ALIGN, WORKSPACE, DTYPE, DEVICE, LAUNCH, ARG, SCRATCH = range(10)
A = 0x100000  # a 256-byte-aligned stand-in address; never dereferenced here
BIG = 1 << 50


@pytest.fixture(scope="module")
def L():
    from bit_block_float_amd import build, hif4
    if not os.path.exists(hif4.LIB_PATH):
        build.build()
    return hif4.lib()


def _quantize(L, x=A, dt=0, batch=1, rows=4, k=40, ld=40, t=0, off=None, groups=0, codes=A, scales=A):
    return L.hif4_quantize_mxfp4(x, dt, batch, rows, k, ld, t, off, groups, codes, scales, None)


def test_quantize(L):
    assert _quantize(L, x=None) == NULL and _quantize(L, codes=None) == NULL and _quantize(L, scales=None) == NULL
    assert _quantize(L, rows=-1) == SHAPE and _quantize(L, k=-1) == SHAPE and _quantize(L, batch=-1) == SHAPE
    assert _quantize(L, ld=39) == SHAPE and _quantize(L, rows=1 << 31) == SHAPE
    assert _quantize(L, batch=1 << 20, rows=1 << 11) == SHAPE
    assert _quantize(L, k=(1 << 22) + 1, ld=1 << 23) == SHAPE
    assert _quantize(L, dt=2) == DTYPE and _quantize(L, t=2) == ARG
    assert _quantize(L, x=A + 2) == ALIGN and _quantize(L, codes=A + 8) == ALIGN and _quantize(L, scales=A + 2) == ALIGN
    assert _quantize(L, x=A + 1, dt=1) == ALIGN
    assert _quantize(L, off=A, groups=1) == ARG                    # groups go along the rows
    assert _quantize(L, t=1, off=None, groups=2) == NULL
    assert _quantize(L, t=1, off=A, groups=0) == ARG
    assert _quantize(L, t=1, off=A, groups=2, batch=2) == ARG
    assert _quantize(L, t=1, off=A, groups=(1 << 16) + 1) == SHAPE and _quantize(L, t=1, off=A, groups=-1) == SHAPE
    assert _quantize(L, t=1, off=A + 4, groups=2) == ALIGN
    assert _quantize(L, t=1, off=A, groups=1 << 16, rows=(1 << 31) - 1) == SHAPE  # too many columns
    # nothing to do: no device needed
    assert _quantize(L, rows=0, x=None, codes=None, scales=None) == OK
    assert _quantize(L, k=0, ld=0, x=None, codes=None, scales=None) == OK
    assert _quantize(L, batch=0, x=None, codes=None, scales=None) == OK
    assert _quantize(L, rows=0, t=1, x=None, codes=None, scales=None) == OK
    # groups of no rows still have columns
    assert _quantize(L, rows=0, t=1, off=A, groups=200, x=None, codes=None) == NULL


def test_quantize_both(L):
    def call(x=A, rows=4, k=40, off=None, groups=0, codes=A, scales=A, codes_t=A, scales_t=A, batch=1):
        return L.hif4_quantize_mxfp4_both(x, 0, batch, rows, k, 40, off, groups, codes, scales, codes_t, scales_t, None)
    for name in ("codes", "scales", "codes_t", "scales_t", "x"):
        assert call(**{name: None}) == NULL
    for name in ("codes", "codes_t"):
        assert call(**{name: A + 8}) == ALIGN
    for name in ("scales", "scales_t", "x"):
        assert call(**{name: A + 2}) == ALIGN
    assert call(k=41) == SHAPE and call(groups=1) == NULL and call(off=A) == ARG and call(off=A, groups=1, batch=3) == ARG
    assert call(rows=0, codes=None, scales=None, codes_t=None, scales_t=None, x=None) == OK


def test_columns(L):
    from bit_block_float_amd import hif4
    for rows, groups, want in ((0, 0, 0), (1, 0, 128), (128, 0, 128), (129, 0, 256), (10, 1, 128), (0, 1, 0), (1, 2, 128),
                               (2, 2, 256), (300, 6, 1024), (1000, 3, 1280)):
        assert hif4.mxfp4_columns(rows, groups) == want, (rows, groups)
    # no split of the rows takes more
    for parts in ((1, 1, 1, 297), (300, 0, 0), (129, 129, 42), (1, 128, 171)):
        assert sum(-(-p // 128) * 128 for p in parts) <= hif4.mxfp4_columns(300, len(parts))
    assert L.hif4_mxfp4_columns(-1, 0) == 0 and L.hif4_mxfp4_columns(5, -1) == 0 and L.hif4_mxfp4_columns(1 << 31, 0) == 0


def test_dequantize(L):
    def call(codes=A, scales=A, rows=4, k=40, out=A, dt=0):
        return L.hif4_dequantize_mxfp4(codes, scales, rows, k, out, dt, None)
    assert call(codes=None) == NULL and call(scales=None) == NULL and call(out=None) == NULL
    assert call(rows=-1) == SHAPE and call(k=-1) == SHAPE and call(k=1 << 31) == SHAPE and call(dt=5) == DTYPE
    assert call(codes=A + 4) == ALIGN and call(out=A + 2) == ALIGN and call(out=A + 1, dt=1) == ALIGN
    assert call(rows=0, codes=None) == OK and call(k=0, out=None) == OK


def test_linear(L):
    def call(x=A, xs=A, w=A, ws=A, m=4, n=5, k=128, y=A, dt=0, work=A, nbytes=BIG):
        return L.hif4_linear_mxfp4(x, xs, w, ws, m, n, k, y, dt, work, nbytes, None)
    for name in ("x", "xs", "w", "ws", "y"):
        assert call(**{name: None}) == NULL
        assert call(**{name: A + 2}) == ALIGN
    assert call(m=-1) == SHAPE and call(n=-1) == SHAPE and call(k=127) == SHAPE and call(k=64) == SHAPE
    assert call(m=1 << 31) == SHAPE and call(k=(1 << 22) + 128) == SHAPE and call(m=1 << 20, n=1 << 18) == SHAPE
    assert call(dt=2) == DTYPE
    assert call(m=0, y=None) == OK and call(n=0, y=None) == OK
    need = L.hif4_linear_mxfp4_workspace_bytes(300, 96, 13824)
    assert need > 0 and need % (300 * 96 * 4) == 0
    assert call(m=300, n=96, k=13824, work=None) == WORKSPACE
    assert call(m=300, n=96, k=13824, nbytes=need - 1) == WORKSPACE
    assert call(m=300, n=96, k=13824, work=A + 128, nbytes=need) == ALIGN
    for m, n, k in ((100, 100, 64), (-1, 4, 128), (1 << 30, 1 << 30, 128), (300, 300, 1)):
        assert L.hif4_linear_mxfp4_workspace_bytes(m, n, k) == 0


def test_linear_grouped(L):
    def call(x=A, xs=A, w=A, ws=A, off=A, groups=3, m=4, n=5, k=128, y=A, dt=0):
        return L.hif4_linear_mxfp4_grouped(x, xs, w, ws, off, groups, m, n, k, y, dt, None)
    for name in ("x", "xs", "w", "ws", "y", "off"):
        assert call(**{name: None}) == NULL
        assert call(**{name: A + 2}) == ALIGN
    assert call(m=-1) == SHAPE and call(n=-1) == SHAPE and call(k=127) == SHAPE and call(groups=-1) == SHAPE
    assert call(groups=(1 << 16) + 1) == SHAPE and call(groups=1 << 16, n=1 << 15) == SHAPE
    assert call(m=1 << 30, n=1 << 14) == SHAPE and call(dt=7) == DTYPE
    assert call(m=0, y=None) == OK and call(n=0, y=None) == OK and call(groups=0, off=None, y=None) == OK


def test_backwards(L):
    def plain(dy=A, ldy=5, xt=A, xts=A, wt=A, wts=A, m=4, n=5, k=6, dx=A, dxt=0, dw=A, dwt=0, work=A, nbytes=BIG, dt=0):
        return L.hif4_linear_mxfp4_backward(dy, dt, ldy, xt, xts, wt, wts, m, n, k, dx, dxt, dw, dwt, work, nbytes, None)

    def grouped(dy=A, ldy=5, xt=A, xts=A, wt=A, wts=A, m=4, n=5, k=6, dx=A, dxt=0, dw=A, dwt=0, work=A, nbytes=BIG, dt=0,
                off=A, groups=3):
        return L.hif4_linear_mxfp4_grouped_backward(dy, dt, ldy, xt, xts, wt, wts, off, groups, m, n, k, dx, dxt, dw, dwt,
                                                    work, nbytes, None)
    for call in (plain, grouped):
        for name in ("dy", "xt", "xts", "wt", "wts"):
            assert call(**{name: None}) == NULL
            assert call(**{name: A + 2}) == ALIGN
        assert call(dx=A + 8) == ALIGN and call(dw=A + 8) == ALIGN
        assert call(work=None) == WORKSPACE and call(nbytes=5) == WORKSPACE and call(work=A + 16) == ALIGN
        assert call(ldy=4) == SHAPE and call(m=-1) == SHAPE and call(k=-1) == SHAPE and call(n=(1 << 22) + 1, ldy=1 << 23) == SHAPE
        assert call(dt=2) == DTYPE and call(dxt=2) == DTYPE and call(dwt=-1) == DTYPE
        assert call(k=0, dx=None, dw=None) == OK and call(dx=None, dw=None, work=None) == OK
    assert plain(m=(1 << 22) + 1) == SHAPE
    assert grouped(m=1 << 22) == SHAPE  # its columns pass the limit
    assert grouped(groups=-1) == SHAPE and grouped(groups=1 << 17) == SHAPE and grouped(groups=(1 << 32) + 3) == SHAPE
    assert grouped(off=None) == NULL and grouped(off=A + 4) == ALIGN
    assert grouped(groups=0, off=None, dw=None) == OK
    a, b = L.hif4_linear_mxfp4_backward_workspace_bytes(1000, 700, 300), 1000 * 768 // 2 + 700 * 1024 // 2
    assert b < a < 3 * b + 40 * 1000 * 700 * 4
    assert L.hif4_linear_mxfp4_backward_workspace_bytes(-1, 4, 4) == 0
    assert L.hif4_linear_mxfp4_grouped_backward_workspace_bytes(4, 1 << 22, 4, 4) == 0
    assert L.hif4_linear_mxfp4_grouped_backward_workspace_bytes(-1, 4, 4, 4) == 0
    assert L.hif4_linear_mxfp4_grouped_backward_workspace_bytes(4, 100, 4, 4) > 0


def test_norm(L):
    def call(x=A, dt=0, rows=4, c=8, ld=8, w=A, b=A, wd=0, eps=1e-6, codes=A, scales=A):
        return L.hif4_layer_norm_quantize_mxfp4(x, dt, rows, c, ld, w, b, wd, eps, codes, scales, None)
    assert call(x=None) == NULL and call(codes=None) == NULL and call(scales=None) == NULL
    assert call(codes=A + 8) == ALIGN and call(scales=A + 1) == ALIGN and call(x=A + 2) == ALIGN
    assert call(ld=7) == SHAPE and call(c=0, ld=0) == SHAPE and call(rows=-1) == SHAPE and call(c=65537, ld=65537) == SHAPE
    assert call(eps=-1.0) == ARG and call(eps=1e39) == ARG and call(dt=3) == DTYPE and call(wd=3) == DTYPE
    assert call(rows=0, x=None, codes=None) == OK


def test_binding_checks_shapes_before_the_library():
    from bit_block_float_amd import hif4
    e8 = torch.float8_e8m0fnu
    c = lambda *s: torch.empty(s, dtype=torch.uint8)  # noqa: E731
    s = lambda *d: torch.empty(d, dtype=e8)  # noqa: E731
    off = torch.zeros(4, dtype=torch.int64)
    raises = lambda f, *a, **kw: pytest.raises(ValueError, f, *a, **kw)  # noqa: E731
    raises(hif4.quantize_mxfp4, torch.empty((4, 8), dtype=torch.float16))
    raises(hif4.quantize_mxfp4, torch.empty((2, 4, 8)).transpose(1, 2))
    raises(hif4.quantize_mxfp4, torch.empty((4, 8)), offsets=off)                            # not transposed
    raises(hif4.quantize_mxfp4, torch.empty((4, 8)), transposed=True, offsets=off.int())
    raises(hif4.quantize_mxfp4, torch.empty((2, 4, 8)), transposed=True, offsets=off)
    raises(hif4.quantize_mxfp4, torch.empty((4, 8)), transposed=True, offsets=off[:1])
    raises(hif4.quantize_mxfp4, torch.empty((4, 8)))                                         # not on the GPU
    raises(hif4.dequantize_mxfp4, c(4, 60), s(4, 4))
    raises(hif4.dequantize_mxfp4, c(4, 64), s(4, 3))
    raises(hif4.dequantize_mxfp4, c(4, 64), s(4, 4), k=129)
    raises(hif4.dequantize_mxfp4, c(4, 64), s(4, 4), k=-1)
    raises(hif4.dequantize_mxfp4, c(4, 64), s(4, 4), out_dtype=torch.float16)
    raises(hif4.linear_mxfp4, c(4, 64), s(4, 4), c(5, 128), s(5, 8))
    raises(hif4.linear_mxfp4, c(4, 64), c(4, 4), c(5, 64), s(5, 4))
    raises(hif4.linear_mxfp4, c(4, 128)[:, :64], s(4, 4), c(5, 64), s(5, 4))
    raises(hif4.linear_mxfp4_grouped, c(4, 64), s(4, 4), c(5, 64), s(5, 4), off)             # one weight
    raises(hif4.linear_mxfp4_grouped, c(4, 64), s(4, 4), c(2, 5, 64), s(2, 5, 4), off)       # three groups
    raises(hif4.linear_mxfp4_grouped, c(4, 64), s(4, 4), c(3, 5, 128), s(3, 5, 8), off)
    dy = torch.empty((4, 5))
    raises(hif4.linear_mxfp4_backward, dy, c(6, 64), s(6, 4), c(7, 64), s(7, 4))
    raises(hif4.linear_mxfp4_backward, dy, c(6, 128), s(6, 8), c(6, 64), s(6, 4))
    raises(hif4.linear_mxfp4_backward, dy, c(6, 64), s(6, 4), c(6, 64), s(6, 4), dx_dtype=torch.float16)
    raises(hif4.linear_mxfp4_grouped_backward, dy, c(6, 64), s(6, 4), c(3, 6, 64), s(3, 6, 4), off)  # 3 x 128 columns
    raises(hif4.linear_mxfp4_grouped_backward, dy, c(6, 192), s(6, 12), c(2, 6, 64), s(2, 6, 4), off)
    raises(hif4.layer_norm_quantize_mxfp4, torch.empty((4, 8)), weight=torch.empty(7))


def test_one_gradient_checks_what_it_needs():
    from bit_block_float_amd import hif4
    e8 = torch.float8_e8m0fnu
    c = lambda *s: torch.empty(s, dtype=torch.uint8)  # noqa: E731
    s = lambda *d: torch.empty(d, dtype=e8)  # noqa: E731
    off = torch.zeros(4, dtype=torch.int64)
    dy, none = torch.empty((4, 5)), (None, None)
    raises = lambda f, *a, **kw: pytest.raises(ValueError, f, *a, **kw)  # noqa: E731
    xt, wt, wte, xtg = (c(6, 64), s(6, 4)), (c(6, 64), s(6, 4)), (c(3, 6, 64), s(3, 6, 4)), (c(6, 192), s(6, 12))
    raises(hif4.linear_mxfp4_backward, dy, *xt, *wt, need_dx=False, need_dw=False)
    raises(hif4.linear_mxfp4_backward, dy, *none, c(6, 128), s(6, 8), need_dw=False)
    raises(hif4.linear_mxfp4_backward, dy, c(6, 128), s(6, 8), *none, need_dx=False)
    raises(hif4.linear_mxfp4_grouped_backward, dy, *xtg, *wte, off, need_dx=False, need_dw=False)
    raises(hif4.linear_mxfp4_grouped_backward, dy, *none, c(2, 6, 64), s(2, 6, 4), off, need_dw=False)
    raises(hif4.linear_mxfp4_grouped_backward, dy, *xt, *none, off, need_dx=False)
    # what is not needed is not looked at: these get as far as the tensors' device
    for call in (lambda: hif4.linear_mxfp4_backward(dy, *none, *wt, need_dw=False),
                 lambda: hif4.linear_mxfp4_backward(dy, *xt, *none, need_dx=False),
                 lambda: hif4.linear_mxfp4_grouped_backward(dy, *none, *wte, off, need_dw=False),
                 lambda: hif4.linear_mxfp4_grouped_backward(dy, *xtg, *none, off, need_dx=False)):
        with pytest.raises(ValueError, match="must be on the GPU"):
            call()
