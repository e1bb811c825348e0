"""The measured cases of the microscaled 4-bit (MXFP4) linear layers and their grouped form.

Six operators of the ``hif4`` binding, each in a plain form (elementary torch
operations in 32 bits, rounded once at the end) and as the library's call:

  quantize_mxfp4                real -> E2M1 codes + one power-of-two (E8M0) scale per 32 elements
  linear_mxfp4                  Y = X W^T on such codes
  linear_mxfp4_backward         dX = Q(dY) W and dW = Q(dY^T) X of that layer
  linear_mxfp4_grouped          the same product, each run of rows with its own expert's weight
  linear_mxfp4_grouped_backward its two gradients
  layer_norm_quantize_mxfp4     the norm in front of such a layer, quantized on the way out

Sizes are those of the repository's workloads (57,600 video tokens, hidden
5120, FFN 13,824, 8192-token attention projections) and generic ones.
"""
import math

import torch

own = False

E8 = torch.float8_e8m0fnu
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
TOKENS, HIDDEN, FFN = 57600, 5120, 13824
EPS = 1e-6


def listed():
    return [
        # the activation of a 4-bit layer, quantized per token as it arrives (and decoded: fake quantization)
        dict(name="quantize activation", op="quantize", rows=TOKENS, k=HIDDEN, dtype="bf16", transposed=False,
             groups=0),
        # a routed batch quantized along its tokens, expert by expert, for the weight gradients
        dict(name="quantize routed transposed", op="quantize", rows=4099, k=1300, dtype="f32", transposed=True,
             groups=7),
        # one row (a time embedding, a single new token): latency and the weight's bytes count
        dict(name="linear one token", op="linear", m=1, n=FFN, k=HIDDEN, y="bf16"),
        # the FFN-up layer over a whole video
        dict(name="linear ffn up", op="linear", m=TOKENS, n=FFN, k=HIDDEN, y="bf16"),
        # a training or calibration step's backward through an attention projection
        dict(name="backward attention", op="linear_backward", m=8192, n=HIDDEN, k=HIDDEN, dy="bf16"),
        # the same for a short, odd batch whose length ends inside a block, gradients in float32
        dict(name="backward odd batch", op="linear_backward", m=1001, n=1300, k=640, dy="f32"),
        # new tokens of a serving batch over many experts, few rows each or none: the weights' bytes
        dict(name="experts few tokens", op="grouped", rows=96, groups=32, n=HIDDEN, k=2048, y="bf16"),
        # a batch of videos at several timesteps, the FFN-up layers of the two experts that share it
        dict(name="experts two timesteps", op="grouped", rows=TOKENS, groups=2, n=FFN, k=HIDDEN, y="bf16"),
        # a training step's backward through routed experts of a usual size
        dict(name="experts backward", op="grouped_backward", rows=16384, groups=16, n=2048, k=HIDDEN, dy="bf16"),
        # and of a short odd batch, gradients in float32
        dict(name="experts backward odd", op="grouped_backward", rows=1001, groups=5, n=1300, k=640, dy="f32"),
        # norm and quantization in one pass before a 4-bit layer, whole video
        dict(name="norm to mxfp4 video", op="norm", rows=TOKENS, c=HIDDEN, dtype="bf16", weight="f32"),
        # and over a few rows of an odd width: launch and latency
        dict(name="norm to mxfp4 odd", op="norm", rows=77, c=1003, dtype="f32", weight="f32"),
    ]


def _spread(rng, lo, hi):
    """A whole number in lo..hi, uniform in its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantize", "linear", "linear", "linear_backward", "grouped", "grouped",
                     "grouped_backward", "norm"])
    if op == "quantize":
        k = _spread(rng, 1, FFN)
        rows = _spread(rng, 1, min(TOKENS, TOKENS * HIDDEN // k))
        transposed = rng.random() < 0.5
        return dict(op=op, rows=rows, k=k, dtype=rng.choice(["bf16", "f32"]), transposed=transposed,
                    groups=rng.choice([0, _spread(rng, 1, 64)]) if transposed and k * rows < 1 << 27 else 0)
    if op == "linear":
        k = 128 * _spread(rng, 1, FFN // 128)
        n = _spread(rng, 1, FFN)
        m = _spread(rng, 1, TOKENS if n * k <= FFN * HIDDEN else 8192)
        return dict(op=op, m=m, n=n, k=k, y=rng.choice(["bf16", "f32"]))
    if op == "linear_backward":
        return dict(op=op, m=_spread(rng, 1, 8192), n=_spread(rng, 1, HIDDEN), k=_spread(rng, 1, HIDDEN),
                    dy=rng.choice(["bf16", "f32"]))
    if op in ("grouped", "grouped_backward"):
        groups = _spread(rng, 1, 128)
        rows = _spread(rng, 1, 32768)
        n = _spread(rng, 1, HIDDEN)
        k = _spread(rng, 1, HIDDEN)
        if op == "grouped":
            return dict(op=op, rows=rows, groups=groups, n=n, k=128 * ((k + 127) // 128), y=rng.choice(["bf16", "f32"]))
        return dict(op=op, rows=rows, groups=groups, n=n, k=min(k, max(1, (1 << 28) // (n * groups))),
                    dy=rng.choice(["bf16", "f32"]))
    c = _spread(rng, 16, FFN)
    rows = _spread(rng, 1, min(TOKENS, TOKENS * HIDDEN // c))
    return dict(op=op, rows=rows, c=c, dtype=rng.choice(["bf16", "f32"]), weight=rng.choice(["f32", "bf16", "none"]))


# ---------------------------------------------------------------- inputs


def _activations(rows, c, gen, device):
    """Heavy-tailed rows: channel scales spread like a log-normal, a few channels far larger."""
    scale = torch.exp(torch.randn((c,), generator=gen, device=device))
    far = torch.rand((c,), generator=gen, device=device) < 0.001
    scale = torch.where(far, scale * 50.0, scale)
    x = torch.randn((rows, c), generator=gen, device=device)
    return x.mul_(scale).add_(0.1)


def _routed(rows, groups, seed, device):
    """Rows of each group, drawn row by row from a skewed popularity: (counts on the host, offsets)."""
    gen = torch.Generator()
    gen.manual_seed(int(seed) + 1)
    popular = torch.exp(torch.randn((groups,), generator=gen))
    counts = torch.bincount(torch.multinomial(popular, rows, replacement=True, generator=gen), minlength=groups)
    offsets = torch.zeros((groups + 1,), dtype=torch.int64)
    torch.cumsum(counts, 0, out=offsets[1:])
    return counts.tolist(), offsets.to(device)


def prepare(case, seed):
    device = "cuda" if torch.cuda.is_available() else "cpu"
    gen = torch.Generator(device=device)
    gen.manual_seed(int(seed))
    op = case["op"]
    s = {"case": case}
    if op == "quantize":
        s["x"] = _activations(case["rows"], case["k"], gen, device).to(DTYPES[case["dtype"]])
        if case["groups"]:
            s["counts"], s["offsets"] = _routed(case["rows"], case["groups"], seed, device)
    elif op == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        s["x_codes"], s["x_scales"] = _packed(_activations(m, k, gen, device).to(torch.bfloat16))
        s["w_codes"], s["w_scales"] = _packed(torch.randn((n, k), generator=gen, device=device).mul_(0.02))
    elif op == "linear_backward":
        m, n, k = case["m"], case["n"], case["k"]
        s["dy"] = (_activations(m, n, gen, device) * 1e-3).to(DTYPES[case["dy"]])
        s["xt_codes"], s["xt_scales"] = _packed(_activations(m, k, gen, device).T)
        s["wt_codes"], s["wt_scales"] = _packed(torch.randn((n, k), generator=gen, device=device).mul_(0.02).T)
    elif op == "grouped":
        rows, groups, n, k = case["rows"], case["groups"], case["n"], case["k"]
        s["counts"], s["offsets"] = _routed(rows, groups, seed, device)
        s["x_codes"], s["x_scales"] = _packed(_activations(rows, k, gen, device).to(torch.bfloat16))
        w = [_packed(torch.randn((n, k), generator=gen, device=device).mul_(0.02)) for _ in range(groups)]
        s["w_codes"], s["w_scales"] = torch.stack([c for c, _ in w]), _stack_scales([t for _, t in w])
    elif op == "grouped_backward":
        rows, groups, n, k = case["rows"], case["groups"], case["n"], case["k"]
        s["counts"], s["offsets"] = _routed(rows, groups, seed, device)
        s["dy"] = (_activations(rows, n, gen, device) * 1e-3).to(DTYPES[case["dy"]])
        s["xt_codes"], s["xt_scales"] = _packed(_spaced(_activations(rows, k, gen, device), s["counts"]).T)
        w = [_packed(torch.randn((k, n), generator=gen, device=device).mul_(0.02)) for _ in range(groups)]
        s["wt_codes"], s["wt_scales"] = torch.stack([c for c, _ in w]), _stack_scales([t for _, t in w])
    else:
        rows, c = case["rows"], case["c"]
        s["x"] = _activations(rows, c, gen, device).to(DTYPES[case["dtype"]])
        s["w"] = s["b"] = None
        if case["weight"] != "none":
            wt = DTYPES[case["weight"]]
            s["w"] = (1.0 + 0.2 * torch.randn((c,), generator=gen, device=device)).to(wt)
            s["b"] = (0.2 * torch.randn((c,), generator=gen, device=device)).to(wt)
    return s


def _stack_scales(scales):
    return torch.stack([t.view(torch.uint8) for t in scales]).view(E8)


# ---------------------------------------------------------------- plain forms (32 bits)


def _up128(v):
    return (v + 127) // 128 * 128


def _spaced(x, counts):
    """The groups' rows, each group's rounded up to a multiple of 128 with zeros; behind them zeros up
    to the most that any groups of as many rows can take."""
    most = (x.shape[0] + 127 * len(counts)) // 128 * 128
    ends = torch.tensor([0] + counts).cumsum(0).tolist()
    starts = torch.tensor([0] + [_up128(v) for v in counts]).cumsum(0).tolist()
    at = torch.cat([torch.arange(v) + t for v, t in zip(counts, starts)])
    out = x.new_zeros((most, x.shape[1]))
    out[at.to(x.device)] = x[:ends[-1]]
    return out


def _scale_of(amax):
    """Smallest power of two s (2^-127 at least) with amax <= 6 s, and 1/s, in float32."""
    bits = amax.view(torch.int32)
    e = ((bits >> 23) - 129 + ((bits & 0x7FFFFF) > 0x400000).int()).clamp(min=-127)
    one = torch.where(e == -127, torch.full_like(e, 0x400000), (e + 127) << 23)
    return one.view(torch.float32), ((127 - e) << 23).view(torch.float32)


def _quantized(x):
    """E2M1 magnitudes with sign [rows][k up to 128s] and scales [rows][blocks of 32], float32."""
    rows, k = x.shape
    v = torch.nn.functional.pad(x.float(), (0, _up128(k) - k)).view(rows, _up128(k) // 32, 32)
    s, inv = _scale_of(v.abs().amax(2, keepdim=True))
    v = v * inv
    a = v.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return (torch.round(v / step) * step).view(rows, -1), s.view(rows, -1)


def _times(q, s):
    return (q.view(q.shape[0], -1, 32) * s.unsqueeze(2)).view(q.shape)


def _packed(x):
    """Codes uint8 [rows][k up to 128s / 2], the even element in the low half, and E8M0 scales."""
    q, s = _quantized(x)
    a = q.abs()
    bits = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    bits = bits | (torch.signbit(q).to(torch.uint8) << 3)
    codes = bits[:, ::2] | (bits[:, 1::2] << 4)
    return codes.contiguous(), ((s.view(torch.int32) >> 23) & 255).to(torch.uint8).view(E8)


def _values(codes, scales):
    """What codes and scales stand for, in float32."""
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    q = table[torch.stack([codes & 15, codes >> 4], -1).int()].view(*codes.shape[:-1], -1)
    b = scales.view(torch.uint8).int()
    s = torch.where(b == 0, torch.full_like(b, 0x400000), b << 23).view(torch.float32)
    return (q.view(*s.shape, 32) * s.unsqueeze(-1)).view(q.shape)


def _norm(x, w, b):
    x = x.float()
    d = x - x.mean(1, keepdim=True)
    y = d * torch.rsqrt(d.square().mean(1, keepdim=True) + EPS)
    return y if w is None else y * w.float() + b.float()


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "quantize":
        x = s["x"]
        if case["transposed"]:
            x = (_spaced(x, s["counts"]) if case["groups"] else x).T
        q, t = _quantized(x)
        return [_times(q, t)[:, :x.shape[1]].to(torch.bfloat16), _e8m0(t)]
    if op == "linear":
        y = _values(s["x_codes"], s["x_scales"]) @ _values(s["w_codes"], s["w_scales"]).T
        return y.to(DTYPES[case["y"]])
    if op == "linear_backward":
        dx = _times(*_quantized(s["dy"])) @ _values(s["wt_codes"], s["wt_scales"]).T
        dw = _times(*_quantized(s["dy"].T)) @ _values(s["xt_codes"], s["xt_scales"]).T
        return [dx.to(DTYPES[case["dy"]]), dw]
    if op == "grouped":
        x = _values(s["x_codes"], s["x_scales"]).split(s["counts"])
        y = [v @ _values(c, t).T for v, c, t in zip(x, s["w_codes"], s["w_scales"])]
        return torch.cat(y).to(DTYPES[case["y"]])
    if op == "grouped_backward":
        counts = s["counts"]
        d = _times(*_quantized(s["dy"])).split(counts)
        dx = [v @ _values(c, t).T for v, c, t in zip(d, s["wt_codes"], s["wt_scales"])]
        padded = [_up128(v) for v in counts]
        dt = _times(*_quantized(_spaced(s["dy"], counts).T))[:, :sum(padded)].split(padded, 1)
        xt = _values(s["xt_codes"], s["xt_scales"])[:, :sum(padded)].split(padded, 1)
        return [torch.cat(dx).to(DTYPES[case["dy"]]), torch.stack([a @ b.T for a, b in zip(dt, xt)])]
    y = _norm(s["x"], s["w"], s["b"]).to(s["x"].dtype)
    return _times(*_quantized(y))[:, :case["c"]].to(torch.bfloat16)


def _e8m0(s):
    return ((s.view(torch.int32) >> 23) & 255).to(torch.uint8).view(E8)


# ---------------------------------------------------------------- the library's calls


def _library(s):
    from bit_block_float_amd import hif4

    case = s["case"]
    op = case["op"]
    if op == "quantize":
        codes, scales = hif4.quantize_mxfp4(s["x"], transposed=case["transposed"], offsets=s.get("offsets"))
        k = None if case["groups"] else s["x"].shape[0 if case["transposed"] else 1]
        return [hif4.dequantize_mxfp4(codes, scales, k=k, out_dtype=torch.bfloat16), scales]
    if op == "linear":
        return hif4.linear_mxfp4(s["x_codes"], s["x_scales"], s["w_codes"], s["w_scales"],
                                 y_dtype=DTYPES[case["y"]])
    if op == "linear_backward":
        return list(hif4.linear_mxfp4_backward(s["dy"], s["xt_codes"], s["xt_scales"], s["wt_codes"],
                                               s["wt_scales"]))
    if op == "grouped":
        return hif4.linear_mxfp4_grouped(s["x_codes"], s["x_scales"], s["w_codes"], s["w_scales"], s["offsets"],
                                         y_dtype=DTYPES[case["y"]])
    if op == "grouped_backward":
        return list(hif4.linear_mxfp4_grouped_backward(s["dy"], s["xt_codes"], s["xt_scales"], s["wt_codes"],
                                                       s["wt_scales"], s["offsets"]))
    codes, scales = hif4.layer_norm_quantize_mxfp4(s["x"], s["w"], s["b"], eps=EPS)
    return hif4.dequantize_mxfp4(codes, scales, k=case["c"], out_dtype=torch.bfloat16)


def run(state):
    return _library(state) if own else _plain(state)


# ---------------------------------------------------------------- what a pass cannot do without


def work(case):
    op = case["op"]
    size = (lambda t: {"bf16": 2, "f32": 4, "none": 0}[t])
    held = (lambda v: v // 2 + v // 32)  # codes and scales of v elements
    if op == "quantize":  # the values come back in bf16, the scales as they are
        r, k = case["rows"], case["k"]
        along = r + 64 * case["groups"] if case["transposed"] else k
        return {"bytes": r * k * size(case["dtype"]) + r * k * 2 + (k if case["transposed"] else r) * along // 32,
                "flops": 2 * r * k}
    if op == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": held((m + n) * k) + m * n * size(case["y"]), "flops": 2 * m * n * k}
    if op == "linear_backward":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": m * n * size(case["dy"]) + held(k * (m + n)) + m * k * size(case["dy"]) + n * k * 4,
                "flops": 4 * m * n * k}
    if op == "grouped":
        r, g, n, k = case["rows"], case["groups"], case["n"], case["k"]
        return {"bytes": held(r * k + min(r, g) * n * k) + r * n * size(case["y"]), "flops": 2 * r * n * k}
    if op == "grouped_backward":
        r, g, n, k = case["rows"], case["groups"], case["n"], case["k"]
        return {"bytes": r * n * size(case["dy"]) + held(r * k + min(r, g) * n * k) + r * k * size(case["dy"]) +
                g * n * k * 4, "flops": 4 * r * n * k}
    r, c = case["rows"], case["c"]
    return {"bytes": r * c * (size(case["dtype"]) + 2) + 2 * c * size(case["weight"]), "flops": 12 * r * c}


# ---------------------------------------------------------------- the definition, in 64 bits


def _exact_quantized(x):
    """Values and scales of float64 x: the exponent by frexp, each quotient to the nearest of the
    format's magnitudes by its distance, the one with the even code where two are as near."""
    rows, k = x.shape
    kp = -(-k // 128) * 128
    v = x.new_zeros((rows, kp))
    v[:, :k] = x
    v = v.reshape(rows, kp // 32, 32)
    f, e = torch.frexp(v.abs().amax(2))
    e = e - 3 + (f > 0.75).to(e.dtype)
    s = torch.exp2(e.double().clamp(min=-127))
    s = torch.where(f == 0, torch.full_like(s, 2.0 ** -127), s)
    a = v.abs() / s[:, :, None]
    q = torch.zeros_like(a)
    for low, high, up in ((0, .5, False), (.5, 1, True), (1, 1.5, False), (1.5, 2, True), (2, 3, False), (3, 4, True),
                          (4, 6, False)):
        mid = (low + high) / 2
        q = torch.where((a >= mid) if up else (a > mid), torch.full_like(q, high), q)
    return torch.copysign(q, v).mul_(s[:, :, None]).reshape(rows, kp), s


def _exact_values(codes, scales):
    c = codes.to(torch.int32)
    c = torch.stack((c.remainder(16), c.div(16, rounding_mode="floor")), 2).flatten(1)
    m, e = (c & 1).double(), (c >> 1 & 3)
    v = torch.where(e == 0, m / 2, (1 + m / 2) * torch.exp2(e.double() - 1))
    v = torch.where(c > 7, -v, v)
    return v * torch.exp2(scales.view(torch.uint8).double() - 127).repeat_interleave(32, 1)


def _exact_norm(x, w, b):
    x = x.double()
    var, mean = torch.var_mean(x, 1, correction=0, keepdim=True)
    y = (x - mean) * (var + EPS) ** -0.5
    return y if w is None else y * w.double() + b.double()


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        x = s["x"].double()
        if case["groups"]:
            wide = x.new_zeros(((case["rows"] + 127 * case["groups"]) // 128 * 128, case["k"]))
            at = row = 0
            for n in s["counts"]:
                wide[at:at + n] = x[row:row + n]
                at, row = at + -(-n // 128) * 128, row + n
            x = wide
        x = x.T if case["transposed"] else x
        v, t = _exact_quantized(x)
        return [v[:, :x.shape[1]], t]
    if op == "linear":
        return torch.mm(_exact_values(s["x_codes"], s["x_scales"]), _exact_values(s["w_codes"], s["w_scales"]).T)
    if op == "linear_backward":
        dy = s["dy"].double()
        return [torch.mm(_exact_quantized(dy)[0], _exact_values(s["wt_codes"], s["wt_scales"]).T),
                torch.mm(_exact_quantized(dy.T)[0], _exact_values(s["xt_codes"], s["xt_scales"]).T)]
    if op == "grouped":
        y = torch.zeros((case["rows"], case["n"]), dtype=torch.float64, device=s["x_codes"].device)
        row = 0
        for e, n in enumerate(s["counts"]):
            if n:
                x = _exact_values(s["x_codes"][row:row + n], s["x_scales"].view(torch.uint8)[row:row + n].view(E8))
                torch.mm(x, _exact_values(s["w_codes"][e], s["w_scales"][e]).T, out=y[row:row + n])
            row += n
        return y
    if op == "grouped_backward":
        dy = s["dy"].double()
        dx = dy.new_zeros((case["rows"], case["k"]))
        dw = dy.new_zeros((case["groups"], case["n"], case["k"]))
        row = at = 0
        for e, n in enumerate(s["counts"]):
            if n:
                d, wide = dy[row:row + n], -(-n // 128) * 128
                dx[row:row + n] = torch.mm(_exact_quantized(d)[0], _exact_values(s["wt_codes"][e], s["wt_scales"][e]).T)
                xt = _exact_values(s["xt_codes"][:, at // 2:(at + wide) // 2],
                                   s["xt_scales"].view(torch.uint8)[:, at // 32:(at + wide) // 32].contiguous())
                dw[e] = torch.mm(_exact_quantized(d.T)[0], xt.T)
                at += wide
            row += n
        return [dx, dw]
    y = _exact_norm(s["x"], s["w"], s["b"]).to(s["x"].dtype)  # what is quantized is a value of x's type
    return _exact_quantized(y.double())[0][:, :case["c"]]
