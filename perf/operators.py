"""The measured cases of the 8-bit linear layer and of the layer norm before it.

Six operators of the ``hif4`` binding, each in a plain form (elementary torch
operations in 32 bits, rounded once at the end) and as the library's call:

  quantize_fp8          real -> E4M3 codes + one power-of-two (E8M0) scale per
                        128 elements along the contraction (or per 128 x 128)
  linear_fp8            Y = X W^T on such codes
  linear_fp8_backward   dX = Q(dY) W and dW = Q(dY^T) X of that layer
  layer_norm            the norm in front of a linear layer
  layer_norm_quantize   the same, its result quantized on the way out (HiF4, or
                        E4M3 through layer_norm_quantize_fp8)
  layer_norm_backward   dX, dweight, dbias

Sizes are those of the repository's workloads (57,600 video tokens, hidden
5120, FFN 13,824, 8192-token attention projections) and generic odd ones.
"""
import math

import torch

own = False

F8, E8 = torch.float8_e4m3fn, torch.float8_e8m0fnu
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
TOKENS, HIDDEN, FFN = 57600, 5120, 13824
EPS = 1e-6


def listed():
    return [
        # the activation of a layer kept in 8 bits, quantized per token as it arrives
        dict(name="quantize activation", op="quantize", rows=TOKENS, k=HIDDEN, dtype="bf16", block=1,
             transposed=False),
        # a weight quantized in tiles for the input-gradient product, once per optimizer step
        dict(name="quantize weight transposed", op="quantize", rows=FFN, k=HIDDEN, dtype="bf16",
             block=128, transposed=True),
        # one row (a time embedding, a single new token) against a checkpoint's weight with its
        # float32 scale per 128 x 128: latency and the weight's bytes count
        dict(name="linear one token", op="linear", m=1, n=FFN, k=HIDDEN, scales="f32", y="bf16"),
        # the FFN-up layer over a whole video
        dict(name="linear ffn up", op="linear", m=TOKENS, n=FFN, k=HIDDEN, scales="e8m0", y="bf16"),
        # a training or calibration step's backward through an attention projection
        dict(name="backward attention", op="linear_backward", m=8192, n=HIDDEN, k=HIDDEN, dy="bf16"),
        # the same for a short, odd batch whose length ends inside a block, gradients in float32
        dict(name="backward odd batch", op="linear_backward", m=1001, n=1300, k=640, dy="f32"),
        # the norm before a block's linear layers, whole video
        dict(name="norm video", op="norm", rows=TOKENS, c=HIDDEN, dtype="bf16", weight="f32"),
        # a few rows of an odd width: launch and latency
        dict(name="norm few odd rows", op="norm", rows=77, c=1003, dtype="f32", weight="f32"),
        # norm and HiF4 quantization in one pass: what linear_w4a4 reads as codes
        dict(name="norm to HiF4 video", op="norm_hif4", rows=TOKENS, c=HIDDEN, dtype="bf16", weight="f32"),
        # norm and E4M3 quantization in one pass: an odd number of text tokens
        dict(name="norm to fp8 text", op="norm_fp8", rows=509, c=HIDDEN, dtype="bf16", weight="bf16"),
        # its backward over a whole video (modulation: weight = 1 + scale, bias = shift, in float32)
        dict(name="norm backward video", op="norm_backward", rows=TOKENS, c=HIDDEN, dtype="bf16", weight="f32"),
        # and over a few odd rows
        dict(name="norm backward odd", op="norm_backward", rows=777, c=1003, dtype="f32", weight="f32"),
    ]


def _spread(rng, lo, hi):
    """A whole number in lo..hi, uniform in its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantize", "linear", "linear", "linear_backward", "norm", "norm_hif4",
                     "norm_fp8", "norm_backward"])
    if op == "quantize":
        k = _spread(rng, 1, FFN)
        rows = _spread(rng, 1, min(TOKENS, TOKENS * HIDDEN // k))
        return dict(op=op, rows=rows, k=k, dtype=rng.choice(["bf16", "f32"]),
                    block=rng.choice([1, 128]), transposed=rng.random() < 0.5)
    if op == "linear":
        k = 128 * _spread(rng, 1, FFN // 128)
        n = _spread(rng, 1, FFN)
        m = _spread(rng, 1, TOKENS if n * k <= FFN * HIDDEN else 8192)
        return dict(op=op, m=m, n=n, k=k, scales=rng.choice(["e8m0", "f32"]), y=rng.choice(["bf16", "f32"]))
    if op == "linear_backward":
        return dict(op=op, m=_spread(rng, 1, 8192), n=_spread(rng, 1, HIDDEN), k=_spread(rng, 1, HIDDEN),
                    dy=rng.choice(["bf16", "f32"]))
    c = _spread(rng, 16, FFN)
    if op == "norm_hif4":
        c = 64 * _spread(rng, 1, FFN // 64)
    rows = _spread(rng, 1, min(TOKENS, TOKENS * HIDDEN // c))
    dtype = "bf16" if op == "norm_hif4" else rng.choice(["bf16", "f32"])
    return dict(op=op, rows=rows, c=c, dtype=dtype, weight=rng.choice(["f32", "bf16", "none"]))


# ---------------------------------------------------------------- inputs


def _activations(rows, c, gen, device):
    """Heavy-tailed rows: channel scales spread like a log-normal, a few channels far larger."""
    scale = torch.exp(torch.randn((c,), generator=gen, device=device))
    far = torch.rand((c,), generator=gen, device=device) < 0.001
    scale = torch.where(far, scale * 50.0, scale)
    x = torch.randn((rows, c), generator=gen, device=device)
    return x.mul_(scale).add_(0.1)


def prepare(case, seed):
    device = "cuda" if torch.cuda.is_available() else "cpu"
    gen = torch.Generator(device=device)
    gen.manual_seed(int(seed))
    op = case["op"]
    s = {"case": case}
    if op == "quantize":
        std = 1.0 if case["block"] == 1 else 0.02
        s["x"] = (_activations(case["rows"], case["k"], gen, device) * std).to(DTYPES[case["dtype"]])
    elif op == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        s["x_codes"], s["x_scales"] = _quantized(_activations(m, k, gen, device).to(torch.bfloat16), 1)
        w = torch.randn((n, k), generator=gen, device=device).mul_(0.02)
        s["w_codes"], s["w_scales"] = _quantized(w, 128)
        if case["scales"] == "f32":  # a checkpoint's scales are any float32, not powers of two
            t = 0.5 + 0.5 * torch.rand(s["w_scales"].shape, generator=gen, device=device)
            s["w_scales"] = s["w_scales"].float() * t
    elif op == "linear_backward":
        m, n, k = case["m"], case["n"], case["k"]
        s["dy"] = (_activations(m, n, gen, device) * 1e-3).to(DTYPES[case["dy"]])
        s["xt_codes"], s["xt_scales"] = _quantized(_activations(m, k, gen, device).T.contiguous(), 1)
        w = torch.randn((n, k), generator=gen, device=device).mul_(0.02)
        s["wt_codes"], s["wt_scales"] = _quantized(w.T.contiguous(), 128)
    else:
        rows, c = case["rows"], case["c"]
        dtype = DTYPES[case["dtype"]]
        s["x"] = _activations(rows, c, gen, device).to(dtype)
        s["w"] = s["b"] = None
        if case["weight"] != "none":
            wt = DTYPES[case["weight"]]
            s["w"] = (1.0 + 0.2 * torch.randn((c,), generator=gen, device=device)).to(wt)
            s["b"] = (0.2 * torch.randn((c,), generator=gen, device=device)).to(wt)
        if op == "norm_backward":
            s["dy"] = (1e-3 * torch.randn((rows, c), generator=gen, device=device)).to(dtype)
            xf = s["x"].float()
            s["mean"] = xf.mean(1)
            s["rstd"] = torch.rsqrt((xf - s["mean"][:, None]).square().mean(1) + EPS)
    return s


# ---------------------------------------------------------------- plain forms (32 bits)


def _scale_of(amax):
    """Smallest power of two s (2^-127 at least) with amax <= 448 s, and 1/s, in float32."""
    bits = amax.view(torch.int32)
    e = (bits >> 23) - 135 + ((bits & 0x7FFFFF) > 0x600000).int()
    e = e.clamp(-127, 127)
    one = torch.where(e == -127, torch.full_like(e, 0x400000), (e + 127) << 23)
    return one.view(torch.float32), ((127 - e) << 23).view(torch.float32)


def _pad128(x, rows):
    up = (lambda v: (v + 127) // 128 * 128)
    return torch.nn.functional.pad(x, (0, up(x.shape[1]) - x.shape[1], 0, (up(x.shape[0]) - x.shape[0]) if rows else 0))


def _quantized(x, block):
    """E4M3 codes [rows][k up to 128s] and E8M0 scales of x [rows][k] (block rows x 128)."""
    rows = x.shape[0]
    x = _pad128(x.float(), block == 128)
    r, k = x.shape
    v = x.view(r // block, block, k // 128, 128)
    s, inv = _scale_of(v.abs().amax((1, 3), keepdim=True))
    codes = (v * inv).to(F8).view(r, k)[:rows].contiguous()
    return codes, _e8m0(s.view(r // block, k // 128))


def _e8m0(s):
    """Float32 powers of two as E8M0 (the biased exponent), rows padded to 4 bytes."""
    e = ((s.view(torch.int32) >> 23) & 255).to(torch.uint8)
    out = torch.zeros((e.shape[0], (e.shape[1] + 3) // 4 * 4), dtype=torch.uint8, device=e.device)
    out[:, :e.shape[1]] = e
    return out.view(E8)[:, :e.shape[1]]


def _scales32(scales):
    if scales.dtype == torch.float32:
        return scales
    b = scales.view(torch.uint8).int()
    return torch.where(b == 0, torch.full_like(b, 0x400000), b << 23).view(torch.float32)


def _values(codes, scales):
    """What codes and scales stand for, in float32."""
    r, k = codes.shape
    s = _scales32(scales)
    if s.shape[0] != r:
        s = s.repeat_interleave(128, 0)[:r]
    return (codes.float().view(r, k // 128, 128) * s[:, :, None]).view(r, k)


def _norm(x, w, b):
    x = x.float()
    mean = x.mean(1, keepdim=True)
    d = x - mean
    rstd = torch.rsqrt(d.square().mean(1, keepdim=True) + EPS)
    y = d * rstd
    if w is not None:
        y = y * w.float() + b.float()
    return y, mean[:, 0], rstd[:, 0]


def _hif4_values(y):
    """The HiF4 values of bf16 y: level-1 code from the unit's maximum, one bit per 8 and per 4."""
    r, c = y.shape
    a = y.float().view(r, c // 64, 8, 2, 4)
    code = torch.arange(256, device=y.device)
    v = torch.exp2((code // 4 - 31).float()) * (1 + (code % 4).float() / 4)
    m4 = a.abs().amax(4, keepdim=True)
    m8 = m4.amax(3, keepdim=True)
    m64 = m8.amax(2, keepdim=True)
    v1 = v[torch.searchsorted(7 * v, m64).clamp(max=255)]
    d = v1 * torch.where(m8 > 3.5 * v1, 2.0, 1.0)
    d = d * torch.where(m4 > 1.75 * d, 2.0, 1.0)
    k = torch.round(4 * a.abs() / d).clamp(max=7)
    return (torch.sign(a) * k * d / 4).view(r, c).to(torch.bfloat16)


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "quantize":
        x = s["x"].T if case["transposed"] else s["x"]
        return list(_quantized(x, case["block"]))
    if op == "linear":
        y = _values(s["x_codes"], s["x_scales"]) @ _values(s["w_codes"], s["w_scales"]).T
        return y.to(DTYPES[case["y"]])
    if op == "linear_backward":
        n, k, m = case["n"], case["k"], case["m"]
        d = _values(*_quantized(s["dy"], 1))
        dx = d @ _values(s["wt_codes"], s["wt_scales"]).T
        dt = _values(*_quantized(s["dy"].T, 1))
        dw = dt @ _values(s["xt_codes"], s["xt_scales"]).T
        return [dx.to(DTYPES[case["dy"]]), dw]
    if op == "norm":
        y, mean, rstd = _norm(s["x"], s["w"], s["b"])
        return [y.to(s["x"].dtype), mean, rstd]
    if op == "norm_hif4":
        return _hif4_values(_norm(s["x"], s["w"], s["b"])[0].to(torch.bfloat16))
    if op == "norm_fp8":
        return list(_quantized(_norm(s["x"], s["w"], s["b"])[0].to(s["x"].dtype), 1))
    dy, w = s["dy"].float(), s["w"]
    xhat = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    g = dy if w is None else dy * w.float()
    dx = (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True)) * s["rstd"][:, None]
    out = [dx.to(s["x"].dtype)]
    return out if w is None else out + [(dy * xhat).sum(0).to(w.dtype), dy.sum(0).to(w.dtype)]


# ---------------------------------------------------------------- the library's calls


def _library(s):
    from bit_block_float_amd import hif4

    case = s["case"]
    op = case["op"]
    if op == "quantize":
        return list(hif4.quantize_fp8(s["x"], block_rows=case["block"], transposed=case["transposed"]))
    if op == "linear":
        return hif4.linear_fp8(s["x_codes"], s["x_scales"], s["w_codes"], s["w_scales"],
                               y_dtype=DTYPES[case["y"]])
    if op == "linear_backward":
        return list(hif4.linear_fp8_backward(s["dy"], s["xt_codes"], s["xt_scales"], s["wt_codes"],
                                             s["wt_scales"]))
    if op == "norm":
        return list(hif4.layer_norm(s["x"], s["w"], s["b"], eps=EPS))
    if op == "norm_hif4":
        codes, meta, _ = hif4.layer_norm_quantize(s["x"], s["w"], s["b"], eps=EPS)
        return hif4.dequantize(codes, meta, out_dtype=torch.bfloat16)
    if op == "norm_fp8":
        return list(hif4.layer_norm_quantize_fp8(s["x"], s["w"], s["b"], eps=EPS))
    dx, dw, db = hif4.layer_norm_backward(s["dy"], s["x"], s["mean"], s["rstd"], weight=s["w"])
    return [dx] if s["w"] is None else [dx, dw, db]


def run(state):
    return _library(state) if own else _plain(state)


# ---------------------------------------------------------------- what a pass cannot do without


def work(case):
    op = case["op"]
    up = (lambda v: (v + 127) // 128 * 128)
    size = (lambda t: {"bf16": 2, "f32": 4, "none": 0}[t])
    if op == "quantize":
        r, k = case["rows"], case["k"]
        out, length = (k, up(r)) if case["transposed"] else (r, up(k))
        scales = (out if case["block"] == 1 else up(out) // 128) * (length // 128)
        return {"bytes": r * k * size(case["dtype"]) + out * length + scales, "flops": 2 * r * k}
    if op == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        scales = m * k // 128 + up(n) // 128 * (k // 128) * (4 if case["scales"] == "f32" else 1)
        return {"bytes": (m + n) * k + scales + m * n * size(case["y"]), "flops": 2 * m * n * k}
    if op == "linear_backward":
        m, n, k = case["m"], case["n"], case["k"]
        codes = k * (up(m) + up(n))
        return {"bytes": m * n * size(case["dy"]) + codes + codes // 128 + m * k * size(case["dy"]) + n * k * 4,
                "flops": 4 * m * n * k}
    r, c = case["rows"], case["c"]
    e, w = size(case["dtype"]), size(case["weight"])
    if op == "norm":
        return {"bytes": r * c * 2 * e + 2 * c * w + 8 * r, "flops": 8 * r * c}
    if op == "norm_hif4":  # the values come back in bf16
        return {"bytes": r * c * (e + 2) + 2 * c * w, "flops": 14 * r * c}
    if op == "norm_fp8":
        return {"bytes": r * (c * e + up(c) + up(c) // 128) + 2 * c * w, "flops": 10 * r * c}
    return {"bytes": r * c * 3 * e + 3 * c * w + 8 * r, "flops": 14 * r * c}


# ---------------------------------------------------------------- the definition, in 64 bits


def _exact_fp8(x, block):
    """Codes and scales of float64 x: the exponent by frexp, each quotient rounded to the 3-bit
    significand (steps of 2^-9 below 2^-6), half to even."""
    rows, k = x.shape
    rp, kp = -(-rows // block) * block, -(-k // 128) * 128
    v = x.new_zeros((rp, kp))
    v[:rows, :k] = x
    v = v.reshape(rp // block, block, kp // 128, 128)
    f, e = torch.frexp(v.abs().amax(3).amax(1))
    e = e - 9 + (f > 0.875).to(e.dtype)
    s = torch.exp2(e.double().clamp(min=-127))
    s = torch.where(f == 0, torch.full_like(s, 2.0 ** -127), s)
    q = v / s[:, None, :, None]
    step = torch.exp2(torch.frexp(q)[1].double().clamp(min=-5) - 4)
    return (torch.round(q / step) * step).reshape(rp, kp)[:rows], s


def _exact_values(codes, scales):
    s = scales.double() if scales.dtype == torch.float32 else torch.exp2(scales.view(torch.uint8).double() - 127)
    rows, k = codes.shape
    at = torch.arange(rows, device=codes.device)
    s = s[at if s.shape[0] == rows else at // 128]
    v = codes.double().reshape(rows, k // 128, 128)
    return v.mul_(s.unsqueeze(2)).reshape(rows, k)


def _exact_norm(x, w, b):
    x = x.double()
    var, mean = torch.var_mean(x, 1, correction=0, keepdim=True)
    rstd = (var + EPS) ** -0.5
    y = (x - mean) * rstd
    return (y if w is None else y * w.double() + b.double()), mean.squeeze(1), rstd.squeeze(1)


def _exact_hif4(y):
    rows, c = y.shape
    a = y.double().abs().reshape(rows, c // 64, 64)
    f, e = torch.frexp(a.amax(2) / 7)
    code = (4 * (e.double() + 30) + torch.ceil(8 * f - 4)).clamp(0, 255)
    code = torch.where(f == 0, torch.zeros_like(code), code)
    top = torch.exp2(torch.floor(code / 4) - 31) * (1 + torch.remainder(code, 4) / 4)
    g = a.reshape(rows, c // 64, 8, 8).amax(3)
    e2 = (g > 3.5 * top.unsqueeze(2)).double()
    q = a.reshape(rows, c // 64, 16, 4).amax(3)
    level = top.unsqueeze(2) * torch.exp2(e2.repeat_interleave(2, 2))
    level = (level * torch.exp2((q > 1.75 * level).double())).repeat_interleave(4, 2)
    k = torch.round(a / level * 4).clamp(max=7)
    return torch.copysign(k * level / 4, y.double().reshape_as(a)).reshape(rows, c)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        x = s["x"].double()
        return list(_exact_fp8(x.T if case["transposed"] else x, case["block"]))
    if op == "linear":
        return torch.mm(_exact_values(s["x_codes"], s["x_scales"]), _exact_values(s["w_codes"], s["w_scales"]).T)
    if op == "linear_backward":
        def gradient(d, codes, scales):
            q, t = _exact_fp8(d.double(), 1)
            q = (q.reshape(q.shape[0], -1, 128) * t.unsqueeze(2)).reshape(q.shape)
            return torch.mm(q, _exact_values(codes, scales).T)
        return [gradient(s["dy"], s["wt_codes"], s["wt_scales"]), gradient(s["dy"].T, s["xt_codes"], s["xt_scales"])]
    if op == "norm":
        return list(_exact_norm(s["x"], s["w"], s["b"]))
    if op == "norm_hif4":  # the norm's result is a bf16 value before it is quantized
        return _exact_hif4(_exact_norm(s["x"], s["w"], s["b"])[0].to(torch.bfloat16))
    if op == "norm_fp8":
        return list(_exact_fp8(_exact_norm(s["x"], s["w"], s["b"])[0].to(s["x"].dtype).double(), 1))
    x, dy = s["x"].double(), s["dy"].double()
    n = case["c"]
    rstd = s["rstd"].double().unsqueeze(1)
    xhat = (x - s["mean"].double().unsqueeze(1)) * rstd
    g = dy if s["w"] is None else dy * s["w"].double()
    dx = rstd / n * (n * g - g.sum(1, keepdim=True) - xhat * (g * xhat).sum(1, keepdim=True))
    return [dx] if s["w"] is None else [dx, (dy * xhat).sum(0), dy.sum(0)]
