"""Refused calls of the 8-bit linear layer and the layer norm, on the CPU: status
codes of the C ABI (no call reaches a device) and the binding's ValueErrors."""
import ctypes

import pytest
import torch

OK, NULL, SHAPE, ALIGN, WORKSPACE, DTYPE, DEVICE, LAUNCH, ARG = range(9)
A = 0x100000  # a 256-byte-aligned stand-in address; never dereferenced here
BIG = 1 << 31


@pytest.fixture(scope="module")
def L():
    import os

    from bit_block_float_amd import build, hif4
    if not os.path.exists(hif4.LIB_PATH):
        build.build()
    return hif4.lib()


def test_quantize_fp8(L):
    def q(x=A, dt=1, rows=4, k=200, ld=200, br=1, t=0, c=A, s=A, lds=4):
        return L.hif4_quantize_fp8(x, dt, rows, k, ld, br, t, c, s, lds, None)

    assert q(rows=-1) == SHAPE and q(k=-1) == SHAPE and q(ld=199) == SHAPE
    assert q(rows=BIG) == SHAPE and q(k=(1 << 22) + 1, ld=1 << 23) == SHAPE
    assert q(dt=2) == DTYPE and q(br=2) == ARG and q(t=2) == ARG
    assert q(rows=0, x=None, c=None, s=None) == OK and q(k=0, x=None) == OK
    assert q(x=None) == NULL and q(c=None) == NULL and q(s=None) == NULL
    assert q(lds=1) == SHAPE                       # two blocks a row
    assert q(lds=2) == ALIGN and q(lds=5) == ALIGN  # whole words
    assert q(t=1, rows=600, lds=4) == SHAPE        # five blocks along the rows
    assert q(x=A + 1) == ALIGN and q(x=A + 2, dt=0) == ALIGN
    assert q(c=A + 8) == ALIGN and q(s=A + 2) == ALIGN


def test_quantize_fp8_both(L):
    def q(x=A, dt=1, rows=300, k=200, ld=200, br=1, c=A, s=A, lds=4, ct=A, st=A, ldt=4):
        return L.hif4_quantize_fp8_both(x, dt, rows, k, ld, br, c, s, lds, ct, st, ldt, None)

    assert q(rows=-1) == SHAPE and q(lds=1) == SHAPE and q(ldt=2) == SHAPE
    assert q(ct=None) == NULL and q(st=None) == NULL and q(c=None) == NULL
    assert q(ct=A + 4) == ALIGN and q(ldt=6) == ALIGN and q(br=64) == ARG
    assert q(rows=0, x=None) == OK


def test_dequantize_fp8(L):
    def d(c=A, s=A, kind=0, br=1, lds=4, rows=4, k=200, o=A, dt=0):
        return L.hif4_dequantize_fp8(c, s, kind, br, lds, rows, k, o, dt, None)

    assert d(rows=-1) == SHAPE and d(lds=1) == SHAPE and d(dt=5) == DTYPE and d(kind=2) == DTYPE
    assert d(br=3) == ARG and d(c=None) == NULL and d(o=None) == NULL
    assert d(c=A + 8) == ALIGN and d(o=A + 2) == ALIGN and d(s=A + 2, kind=1) == ALIGN
    assert d(rows=0, c=None) == OK


def test_linear_fp8(L):
    def f(x=A, xs=A, ldxs=4, w=A, ws=A, ldws=4, kind=0, br=128, m=8, n=8, k=512, y=A, dt=0, wsp=A, nb=1 << 40):
        return L.hif4_linear_fp8(x, xs, ldxs, w, ws, ldws, kind, br, m, n, k, y, dt, wsp, nb, None)

    assert f(m=-1) == SHAPE and f(n=-1) == SHAPE and f(k=200) == SHAPE and f(k=-128) == SHAPE
    assert f(m=BIG) == SHAPE and f(n=BIG) == SHAPE and f(k=1 << 23) == SHAPE
    assert f(m=BIG - 1, n=BIG - 1) == SHAPE
    assert f(dt=2) == DTYPE and f(kind=2) == DTYPE and f(br=64) == ARG
    assert f(kind=1, br=1) == ARG                  # float scales are per 128 x 128
    assert f(m=0, x=None, y=None) == OK and f(n=0, w=None, y=None) == OK
    assert f(x=None) == NULL and f(xs=None) == NULL and f(w=None) == NULL and f(ws=None) == NULL
    assert f(y=None) == NULL and f(y=A + 8) == ALIGN
    assert f(ldxs=3) == SHAPE and f(ldws=3) == SHAPE
    assert f(ldxs=5) == ALIGN and f(ldws=6) == ALIGN
    assert f(x=A + 8) == ALIGN and f(w=A + 4) == ALIGN and f(xs=A + 1) == ALIGN and f(ws=A + 2) == ALIGN
    for args in ((-1, 8, 128), (8, BIG, 128), (8, 8, 1 << 23)):
        assert L.hif4_linear_fp8_workspace_bytes(*args) == 0


def test_linear_fp8_backward(L):
    ws = L.hif4_linear_fp8_backward_workspace_bytes(300, 200, 640)
    # dY's codes and scales along both sides at least
    assert ws >= 300 * 256 + 300 * 4 + 200 * 384 + 200 * 4 and ws % 256 == 0
    for args in ((-1, 8, 128), (8, -1, 128), (1 << 23, 8, 8), (8, 8, BIG)):
        assert L.hif4_linear_fp8_backward_workspace_bytes(*args) == 0

    def f(dy=A, dt=1, ld=200, xc=A, xs=A, ldx=4, wc=A, wsc=A, ldw=4, kind=0, br=128, m=300, n=200, k=640, dx=A,
          dxt=1, dw=A, dwt=0, wsp=A, nb=ws):
        return L.hif4_linear_fp8_backward(dy, dt, ld, xc, xs, ldx, wc, wsc, ldw, kind, br, m, n, k, dx, dxt, dw, dwt,
                                          wsp, nb, None)

    assert f(m=-1) == SHAPE and f(k=-1) == SHAPE and f(ld=199) == SHAPE and f(k=BIG) == SHAPE
    assert f(dt=2) == DTYPE and f(dxt=2) == DTYPE and f(dwt=2) == DTYPE and f(kind=2) == DTYPE
    assert f(br=2) == ARG and f(kind=1, br=1) == ARG
    for name in ("dy", "xc", "xs", "wc", "wsc"):
        assert f(**{name: None}) == NULL
    assert f(wsp=None) == WORKSPACE and f(nb=ws - 1) == WORKSPACE and f(wsp=A + 128) == ALIGN
    assert f(ldx=2) == SHAPE and f(ldw=1) == SHAPE and f(ldx=6) == ALIGN
    assert f(dx=A + 8) == ALIGN and f(dw=A + 4) == ALIGN and f(dy=A + 1) == ALIGN
    assert f(dx=None, dw=None, dy=A, wsp=None) == OK


def test_layer_norm(L):
    def f(x=A, dt=1, rows=4, c=100, ld=100, w=A, b=A, wd=0, eps=1e-6, y=A, ldy=100, mean=A, rstd=A):
        return L.hif4_layer_norm(x, dt, rows, c, ld, w, b, wd, eps, y, ldy, mean, rstd, None)

    assert f(rows=-1) == SHAPE and f(c=0) == SHAPE and f(c=65537, ld=1 << 20) == SHAPE
    assert f(ld=99) == SHAPE and f(ldy=99) == SHAPE and f(rows=BIG) == SHAPE
    assert f(dt=3) == DTYPE and f(wd=3) == DTYPE
    assert f(eps=-1e-6) == ARG and f(eps=float("nan")) == ARG and f(eps=float("inf")) == ARG
    assert f(rows=0, x=None, y=None) == OK
    assert f(x=None) == NULL and f(y=None) == NULL
    assert f(x=A + 1) == ALIGN and f(y=A + 1) == ALIGN and f(w=A + 2) == ALIGN and f(mean=A + 2) == ALIGN


def test_layer_norm_quantize(L):
    def f(x=A, dt=1, rows=4, c=128, ld=128, w=A, b=A, wd=0, eps=1e-6, mask=None, nm=0, kept=None, codes=A, meta=A):
        return L.hif4_layer_norm_quantize(x, dt, rows, c, ld, w, b, wd, eps, mask, nm, kept, codes, meta, None)

    assert f(c=100) == SHAPE and f(nm=-1) == SHAPE and f(mask=A, nm=129, kept=A) == SHAPE
    assert f(codes=None) == NULL and f(meta=None) == NULL and f(mask=A, nm=3) == NULL
    assert f(codes=A + 8) == ALIGN and f(meta=A + 2) == ALIGN and f(mask=A + 8, nm=1, kept=A) == ALIGN
    assert f(eps=-1.0) == ARG and f(rows=0, x=None) == OK


def test_layer_norm_quantize_fp8(L):
    def f(x=A, dt=1, rows=4, c=200, ld=200, w=A, b=A, wd=0, eps=1e-6, codes=A, scales=A, lds=4):
        return L.hif4_layer_norm_quantize_fp8(x, dt, rows, c, ld, w, b, wd, eps, codes, scales, lds, None)

    assert f(lds=1) == SHAPE and f(lds=6) == ALIGN and f(codes=None) == NULL and f(scales=None) == NULL
    assert f(codes=A + 4) == ALIGN and f(scales=A + 2) == ALIGN and f(rows=0, x=None) == OK


def test_layer_norm_backward(L):
    ws = L.hif4_layer_norm_backward_workspace_bytes(4, 100)
    assert ws >= 2 * 100 * 4 and ws % 256 == 0
    assert L.hif4_layer_norm_backward_workspace_bytes(-1, 100) == 0
    assert L.hif4_layer_norm_backward_workspace_bytes(4, 65537) == 0

    def f(dy=A, lddy=100, x=A, ldx=100, dt=1, rows=4, c=100, mean=A, rstd=A, w=A, wd=0, dx=A, lddx=100, dw=A,
          db=A, wsp=A, nb=ws):
        return L.hif4_layer_norm_backward(dy, lddy, x, ldx, dt, rows, c, mean, rstd, w, wd, dx, lddx, dw, db, wsp,
                                          nb, None)

    assert f(lddy=99) == SHAPE and f(ldx=99) == SHAPE and f(lddx=99) == SHAPE and f(c=0) == SHAPE
    assert f(dt=2) == DTYPE and f(wd=2) == DTYPE
    for name in ("dy", "x", "mean", "rstd", "dx"):
        assert f(**{name: None}) == NULL
    assert f(wsp=None) == WORKSPACE and f(nb=ws - 1) == WORKSPACE and f(wsp=A + 16) == ALIGN
    assert f(dx=A + 1) == ALIGN and f(dw=A + 2) == ALIGN
    assert f(rows=0, dw=None, db=None, wsp=None, dy=None, x=None) == OK


def test_binding_refuses():
    from bit_block_float_amd import hif4
    x = torch.zeros((4, 200))
    f8, e8 = torch.float8_e4m3fn, torch.float8_e8m0fnu
    bad = [
        lambda: hif4.quantize_fp8(x),                                    # not on a GPU
        lambda: hif4.quantize_fp8(x.half()),
        lambda: hif4.quantize_fp8(x[0]),
        lambda: hif4.quantize_fp8(x.T),
        lambda: hif4.quantize_fp8(x, block_rows=64),
        lambda: hif4.quantize_fp8_both(x, block_rows=0),
        lambda: hif4.dequantize_fp8(x, x),
        lambda: hif4.dequantize_fp8(torch.zeros((4, 256), dtype=f8), x, k=100),
        lambda: hif4.linear_fp8(torch.zeros((4, 200), dtype=f8), x, torch.zeros((4, 200), dtype=f8), x),
        lambda: hif4.linear_fp8(torch.zeros((4, 128), dtype=f8), x, torch.zeros((4, 256), dtype=f8), x),
        lambda: hif4.linear_fp8(torch.zeros((4, 128), dtype=f8), x, torch.zeros((4, 128), dtype=f8), x,
                                y_dtype=torch.float16),
        lambda: hif4.linear_fp8_backward(x, torch.zeros((8, 256), dtype=f8), x, torch.zeros((8, 256), dtype=f8), x),
        lambda: hif4.layer_norm(x.double()),
        lambda: hif4.layer_norm(x, weight=torch.ones(199)),
        lambda: hif4.layer_norm(x, weight=torch.ones(200), bias=torch.ones(200, dtype=torch.bfloat16)),
        lambda: hif4.layer_norm(x),
        lambda: hif4.layer_norm_quantize(x),
        lambda: hif4.layer_norm_backward(x, x.bfloat16(), x[:, 0], x[:, 0]),
        lambda: hif4.layer_norm_backward(x, x, x[:3, 0], x[:, 0]),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was accepted")
    # scales: shape, type, and rows that are not whole words
    ok = torch.zeros((4, 4), dtype=torch.uint8).view(e8)
    hif4._check_scales(ok[:, :3], "s", 4, 3)
    for t, rows, blocks in ((ok, 4, 3), (ok.view(torch.uint8), 4, 4), (ok[:, :3].contiguous(), 4, 3)):
        with pytest.raises(ValueError):
            hif4._check_scales(t, "s", rows, blocks)
