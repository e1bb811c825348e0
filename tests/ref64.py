"""Plain 64-bit references of the 8-bit block format, its product and the layer
norm (CPU, torch float64; no library code)."""
import torch


def up128(v):
    return -(-v // 128) * 128


def fp8_quantize(x, block_rows=1):
    """(code bytes uint8 [rows][k up to 128s], E8M0 bytes uint8 [.][blocks]) of x."""
    x = x.double()
    rows, k = x.shape
    rp, kp = -(-rows // block_rows) * block_rows, up128(k)
    v = torch.zeros((rp, kp), dtype=torch.float64)
    v[:rows, :k] = x
    v = v.reshape(rp // block_rows, block_rows, kp // 128, 128)
    bad = ~torch.isfinite(v).all(3).all(1)
    a = torch.where(bad[:, None, :, None], torch.zeros_like(v), v)
    f, e = torch.frexp(a.abs().amax((1, 3)))
    e = torch.where(f == 0, torch.full_like(e, -127), (e - 9 + (f > 0.875).int()).clamp(min=-127))
    q = a / torch.exp2(e.double())[:, None, :, None]
    codes = e4m3_bits(q)
    codes = torch.where(bad[:, None, :, None], torch.full_like(codes, 0x7F), codes)
    scales = torch.where(bad, torch.full_like(e, 255), e + 127)
    return codes.reshape(rp, kp)[:rows].to(torch.uint8), scales.to(torch.uint8)


def e4m3_bits(q):
    """E4M3 code of |q| <= 448, round to nearest even; int32."""
    ex = torch.frexp(q)[1].clamp(min=-5) - 1           # exponent of the binade, -6 at least
    ex = torch.where(q == 0, torch.full_like(ex, -6), ex)  # frexp gives a zero exponent 0
    k = torch.round(q.abs() / torch.exp2((ex - 3).double()))  # steps of 2^(ex-3): 8..16, below 8 if subnormal
    bits = (k + torch.where(ex > -6, (ex + 6) * 8, torch.zeros_like(ex)).double()).int()
    return bits | torch.where(torch.signbit(q), 128, 0).int()


def fp8_values(codes, scales, block_rows=1):
    """float64 values of uint8 code bytes and scales (uint8 E8M0 bytes or float32)."""
    c = codes.to(torch.int32)
    ex, fr = (c >> 3) & 15, c & 7
    v = torch.where(ex == 0, fr.double() * 2.0 ** -9, (8 + fr).double() * torch.exp2((ex - 10).double()))
    v = torch.where((c & 127) == 127, torch.full_like(v, float("nan")), v)
    v = torch.where(c >= 128, -v, v)
    if scales.dtype == torch.uint8:
        s = torch.exp2(scales.double() - 127)
        s = torch.where(scales == 255, torch.full_like(s, float("nan")), s)
    else:
        s = scales.double()
    s = s.repeat_interleave(block_rows, 0)[: c.shape[0]].repeat_interleave(128, 1)
    return v * s


def layer_norm(x, w, b, eps):
    x = x.double()
    mean = x.mean(1, keepdim=True)
    var = (x - mean).square().mean(1, keepdim=True)
    rstd = (var + eps).rsqrt()
    y = (x - mean) * rstd
    if w is not None:
        y = y * w.double()
    if b is not None:
        y = y + b.double()
    return y, mean[:, 0], rstd[:, 0]


def layer_norm_backward(dy, x, mean, rstd, w):
    dy, x = dy.double(), x.double()
    xhat = (x - mean.double()[:, None]) * rstd.double()[:, None]
    g = dy if w is None else dy * w.double()
    m1, m2 = g.mean(1, keepdim=True), (g * xhat).mean(1, keepdim=True)
    return (g - m1 - xhat * m2) * rstd.double()[:, None], (dy * xhat).sum(0), dy.sum(0)
