"""Plain 64-bit references of the 4-bit microscaled format and its products, with one
weight and by groups of rows (CPU, torch float64; no library code)."""
import torch

MAGNITUDES = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)


def up128(v):
    return -(-v // 128) * 128


def quantize(x):
    """(code bytes uint8 [rows][kp/2], scale bytes uint8 [rows][kp/32]) of x along its rows."""
    x = x.double()
    rows, k = x.shape
    v = torch.zeros((rows, up128(k)), dtype=torch.float64)
    v[:, :k] = x
    v = v.reshape(rows, up128(k) // 32, 32)
    bad = ~torch.isfinite(v).all(2)
    a = torch.where(bad[:, :, None], torch.zeros_like(v), v)
    f, e = torch.frexp(a.abs().amax(2))
    e = torch.where(f == 0, torch.full_like(e, -127), (e - 3 + (f > 0.75).int()).clamp(min=-127))
    q = a.abs() / torch.exp2(e.double())[:, :, None]
    away = (q[..., None] - MAGNITUDES).abs()  # the nearest magnitude, the even code of two as near
    near = away == away.amin(-1, keepdim=True)
    odd_tie = near.sum(-1) > 1
    code = torch.where(odd_tie, (near * (torch.arange(8) % 2 == 0)).int().argmax(-1), near.int().argmax(-1))
    code = code | torch.where(torch.signbit(a), 8, 0)
    code = torch.where(bad[:, :, None], torch.full_like(code, 7), code).reshape(rows, up128(k)).to(torch.uint8)
    scales = torch.where(bad, torch.full_like(e, 255), e + 127).to(torch.uint8)
    return code[:, ::2] | (code[:, 1::2] << 4), scales


def values(codes, scales):
    """float64 values [rows][kp] of code and scale bytes."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
    v = MAGNITUDES[c & 7] * torch.where(c > 7, -1.0, 1.0).double()
    s = torch.exp2(scales.double() - 127)
    s = torch.where(scales == 255, torch.full_like(s, float("nan")), s)
    return v * s.repeat_interleave(32, -1)


def columns(rows, groups):
    return (rows + 127 * groups) // 128 * 128


def spaced(x, offsets):
    """The groups' rows of x, each group's from a multiple of 128 on, zeros between and behind."""
    out = torch.zeros((columns(x.shape[0], len(offsets) - 1), x.shape[1]), dtype=x.dtype)
    at = 0
    for b, e in zip(offsets[:-1], offsets[1:]):
        out[at:at + e - b] = x[b:e]
        at += up128(e - b)
    return out


def starts(offsets):
    """(first column, columns) of each group in what spaced() lays out."""
    at, out = 0, []
    for b, e in zip(offsets[:-1], offsets[1:]):
        out.append((at, up128(e - b)))
        at += up128(e - b)
    return out


def bound(k, s, dtype, parts=1):
    """How far a product's result may be from the real one, sums of magnitudes s: an instruction
    adds 64 exact products and the accumulator, rounding twice at most, and the K parts of a
    workgroup (16 at most) and of a split are added; then the rounding to dtype."""
    fp32 = (2 * -(-k // 64) + 16 + parts) * 2.0 ** -24
    half = 2.0 ** -8 if dtype == torch.bfloat16 else 0.0
    return (fp32 * (1 + half) + half) * s + 2.0 ** -149
