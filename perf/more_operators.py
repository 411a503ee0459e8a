"""The operators on the way into an 8-bit LM head, as cases to measure: layer norm with its backward pass, the
quantiser with a scale for each block of 128, the 8-bit matrix product (forward alone, and a training step's
three products), and the sampler over an 8-bit head.

``run`` computes an operator in elementary torch operations, or, with ``own`` set, through the library."""

import math

import torch

own = False

DEV = "cuda"
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
LARGEST = {E4M3: 448.0, E5M2: 57344.0}
EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # one decode step's hidden states, normed and quantised for what multiplies them: latency
        dict(name="norm_decode", op="norm8", n=16, d=4096, rms=True, type="bf16"),
        # the hidden states of a long batch of prompts
        dict(name="norm_rows", op="norm", n=16384, d=4096, rms=False, type="bf16"),
        # a toy model's training step, odd sizes, everything in 32 bits
        dict(name="normgrad_small", op="normgrad", n=257, d=521, rms=False, type="fp32", wtype="fp32"),
        # the norm's part of a training step of an 8B-class body
        dict(name="normgrad_step", op="normgrad", n=16384, d=4096, rms=False, type="bf16", wtype="bf16"),
        # a quarter of an LM head laid out in 8 bits
        dict(name="quant_weight", op="quant", rows=32064, cols=4096, block=128, transpose=False, fmt="e4m3", type="bf16"),
        # the gradients of a ragged micro-batch, quantised along its tokens for the weight's gradient
        dict(name="quant_grad", op="quant", rows=2043, cols=14336, block=1, transpose=True, fmt="e5m2", type="bf16"),
        # query, key and value projections of one decode step: bound by reading the weights
        dict(name="product_decode", op="product", T=16, k=4096, n=6144, type="bf16"),
        # the way back to the model width for a ragged batch of prompts
        dict(name="product_prompts", op="product", T=517, k=14336, n=4096, type="bf16"),
        # a small layer's training step, odd sizes
        dict(name="linear_small", op="linear", T=65, k=136, n=257),
        # a wide layer's training step on one micro-batch: forward, gradient of the inputs, gradient of the weights
        dict(name="linear_step", op="linear", T=2048, k=4096, n=14336),
        # one decode step through an 8-bit head: bound by reading it once
        dict(name="sample_decode", op="sample", B=16, d=4096, V=128256, bias="none"),
        # a larger batch with some vocabulary entries forbidden
        dict(name="sample_batch", op="sample", B=64, d=4096, V=151936, bias="shared"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm8", "norm", "normgrad", "quant", "product", "linear", "sample"))
    kind = rng.choice(("bf16", "bf16", "fp16", "fp32"))
    if op in ("norm8", "norm", "normgrad"):
        n, d = _log_int(rng, 1, 16384), _log_int(rng, 64, 8192)
        n = max(1, min(n, 16384 * 4096 // d // (2 if kind == "fp32" else 1)))
        case = dict(op=op, n=n, d=d, rms=rng.random() < 0.5, type=kind)
        return dict(case, wtype=rng.choice((kind, "fp32"))) if op == "normgrad" else case
    if op == "quant":
        return dict(op=op, rows=_log_int(rng, 1, 16384), cols=_log_int(rng, 64, 8000), block=rng.choice((1, 128)),
                    transpose=rng.random() < 0.4, fmt=rng.choice(("e4m3", "e5m2")), type=kind)
    if op == "product":
        return dict(op=op, T=_log_int(rng, 1, 2048), k=_log_int(rng, 64, 12000), n=_log_int(rng, 64, 12000), type=kind)
    if op == "linear":
        return dict(op=op, T=_log_int(rng, 1, 2048), k=_log_int(rng, 64, 4096), n=_log_int(rng, 64, 14336))
    return dict(op=op, B=_log_int(rng, 1, 128), d=_log_int(rng, 64, 4096), V=_log_int(rng, 1000, 152000),
                bias=rng.choice(("none", "shared", "rows")))


# ------------------------------------------------------------------ blocks of 128, in elementary operations
def _blocks(x, block):
    """x [r, c] as [r / block, block, c / 128, 128], zeros behind its ends."""
    r, c = x.shape
    R, C = -(-r // block), -(-c // 128)
    wide = torch.zeros((R * block, C * 128), dtype=torch.float32, device=x.device)
    wide[:r, :c] = x
    return wide.view(R, block, C, 128)


def _quantised(x, block, fmt):
    """(q, scale) of x: a scale for `block` rows by 128 columns; rows of q lie a multiple of 16 bytes apart."""
    r, c = x.shape
    b = _blocks(x, block)
    largest = torch.tensor(LARGEST[fmt], device=x.device)
    scale = (b.abs().amax((1, 3)) / largest).clamp(min=2.0 ** -100)
    q = (b * (1.0 / scale)[:, None, :, None]).to(fmt).view(b.shape[0] * block, -1)
    wide = torch.zeros((r, -(-c // 16) * 16), dtype=torch.uint8, device=x.device).view(fmt)
    wide[:, :c] = q[:r, :c]
    return wide[:, :c], scale


def _values(q, scale):
    """What q and its scales stand for, in 32 bits."""
    block = 1 if scale.shape[0] == q.shape[0] else 128
    r, c = q.shape
    return (_blocks(q.float(), block) * scale[:, None, :, None]).view(scale.shape[0] * block, -1)[:r, :c]


# ------------------------------------------------------------------ inputs
def _rand(gen, *shape):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32)


def _hidden(gen, n, d, dtype):
    """Hidden states: rows of different sizes, a few columns that stand out, some drift from zero."""
    x = _rand(gen, n, d) * (0.5 + torch.rand((n, 1), generator=gen, device=DEV)) + 0.1
    x[:, ::97] *= 8.0
    return x.to(dtype)


def _prepare_norm(case, gen):
    n, d = case["n"], case["d"]
    dtype = TYPES[case["type"]]
    wtype = TYPES[case.get("wtype", "fp32")]
    s = dict(op=case["op"], rms=case["rms"], x=_hidden(gen, n, d, dtype), w=(1.0 + 0.2 * _rand(gen, d)).to(wtype),
             b=None if case["rms"] else (0.2 * _rand(gen, d)).to(wtype))
    if case["op"] == "normgrad":
        s["g"] = (_rand(gen, n, d) * 1e-3).to(dtype)
    return s


def _prepare_quant(case, gen):
    x = _hidden(gen, case["rows"], case["cols"], TYPES[case["type"]])
    return dict(op="quant", x=x, block=case["block"], transpose=case["transpose"], fmt=E4M3 if case["fmt"] == "e4m3" else E5M2)


def _prepare_product(case, gen):
    T, k, n = case["T"], case["k"], case["n"]
    W = _rand(gen, n, k) / math.sqrt(k)
    s = dict(op=case["op"], x=_hidden(gen, T, k, TYPES[case.get("type", "bf16")]), W=_quantised(W, 128, E4M3))
    if case["op"] == "linear":
        s["Wt"] = _quantised(W.t(), 128, E4M3)                  # the same blocks, laid out for the gradient of x
        s["g"] = (_rand(gen, T, n) * 1e-3).bfloat16()
    return s


def _prepare_sample(case, gen):
    B, d, V = case["B"], case["d"], case["V"]
    h, W = _quantised(_hidden(gen, B, d, torch.bfloat16), 1, E4M3), _quantised(_rand(gen, V, d) * (0.5 / math.sqrt(d)), 128, E4M3)
    bias = None
    if case["bias"] == "shared":                                # some entries forbidden
        bias = torch.where(torch.rand(V, generator=gen, device=DEV) < 0.1, -math.inf, 0.0)
    elif case["bias"] == "rows":                                # a dense adjustment for each row
        bias = 0.5 * _rand(gen, B, V)
    temp = 0.6 + 0.6 * torch.rand(B, generator=gen, device=DEV)
    draw_seed = int(torch.randint(0, 1 << 40, (1,), generator=gen, device=DEV))
    return dict(op="sample", h=h, W=W, bias=bias, temp=temp, seed=draw_seed, step=draw_seed % 1000)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    make = {"quant": _prepare_quant, "sample": _prepare_sample, "product": _prepare_product, "linear": _prepare_product}
    return make.get(case["op"], _prepare_norm)(case, gen)


# ------------------------------------------------------------------ plain forms
def _plain_stats(s):
    x = s["x"].float()
    if s["rms"]:
        return x, None, (x.square().mean(1) + EPS).rsqrt()
    mean = x.mean(1)
    return x, mean, ((x - mean[:, None]).square().mean(1) + EPS).rsqrt()


def _plain_hat(x, mean, rstd):
    return (x if mean is None else x - mean[:, None]) * rstd[:, None]


def _plain_norm(s):
    x, mean, rstd = _plain_stats(s)
    y = _plain_hat(x, mean, rstd) * s["w"].float()
    if s["b"] is not None:
        y = y + s["b"].float()
    if s["op"] == "norm8":
        return _quantised(y, 1, E4M3)
    return (y.to(s["x"].dtype),) + (() if mean is None else (mean,)) + (rstd,)


def _plain_normgrad(s):
    x, mean, rstd = _plain_stats(s)
    hat = _plain_hat(x, mean, rstd)
    g = s["g"].float()
    a = g * s["w"].float()
    y = hat * s["w"].float()
    if s["b"] is not None:
        y = y + s["b"].float()
    gx = a - hat * (a * hat).mean(1, keepdim=True)
    if mean is not None:
        gx = gx - a.mean(1, keepdim=True)
    gx = (gx * rstd[:, None]).to(s["x"].dtype)
    gw = (g * hat).sum(0, dtype=torch.float64).to(s["w"].dtype)                 # long sums
    if s["b"] is None:
        return y.to(s["x"].dtype), gx, gw
    return y.to(s["x"].dtype), gx, gw, g.sum(0, dtype=torch.float64).to(s["w"].dtype)


def _plain_quant(s):
    return _quantised(s["x"].t() if s["transpose"] else s["x"], s["block"], s["fmt"])


def _plain_product(s):
    return (_values(*_quantised(s["x"], 1, E4M3)) @ _values(*s["W"]).t()).bfloat16()


def _plain_linear(s):
    y = _plain_product(s)
    gx = _values(*_quantised(s["g"], 1, E5M2)) @ _values(*s["Wt"]).t()
    gW = _values(*_quantised(s["g"].t(), 1, E5M2)) @ _values(*_quantised(s["x"].t(), 1, E4M3)).t()
    return y, gx.bfloat16(), gW


def _plain_words(s, B, V):
    """The draws of (row, id): Philox-4x32-10 under the key (seed), counter (id / 4, row, step)."""
    low = 0xFFFFFFFF
    c = [torch.arange(-(-V // 4), device=DEV)[None, :].expand(B, -1), torch.arange(B, device=DEV)[:, None],
         torch.full((1, 1), s["step"] & low, device=DEV), torch.full((1, 1), s["step"] >> 32, device=DEV)]
    k0, k1 = s["seed"] & low, s["seed"] >> 32
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57             # (the low 64 bits, whatever their sign)
        c = [(b >> 32 & low) ^ c[1] ^ k0, b & low, (a >> 32 & low) ^ c[3] ^ k1, a & low]
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    return torch.stack([v.expand(B, -1) for v in c], 2).view(B, -1)[:, :V]


def _plain_sample(s):
    x = _values(*s["h"]) @ _values(*s["W"]).t()
    if s["bias"] is not None:
        x = x + s["bias"]
    u = ((_plain_words(s, *x.shape) >> 9).double() + 0.5) * 2.0 ** -23          # scores next to one another
    z = x.double() / s["temp"].double()[:, None] - torch.log(-torch.log(u))
    best, ids = z.max(1)
    return ids, best.float()


def run(s):
    if own:
        return _run_own(s)
    plain = {"normgrad": _plain_normgrad, "quant": _plain_quant, "product": _plain_product, "linear": _plain_linear,
             "sample": _plain_sample}
    return plain.get(s["op"], _plain_norm)(s)


# ------------------------------------------------------------------ through the library
def _run_own(s):
    from lm_head_exact_gb300 import binding as fs
    op = s["op"]
    if op == "norm8":
        return fs.layer_norm_fp8(s["x"], s["w"], s["b"], eps=EPS, rms=s["rms"])
    if op == "norm":
        return tuple(v for v in fs.layer_norm(s["x"], s["w"], s["b"], eps=EPS, rms=s["rms"]) if v is not None)
    if op == "normgrad":
        y, mean, rstd = fs.layer_norm(s["x"], s["w"], s["b"], eps=EPS, rms=s["rms"])
        gx, gw, gb = fs.layer_norm_backward(s["g"], s["x"], s["w"], mean, rstd, need_bias=s["b"] is not None)
        return (y, gx, gw) if gb is None else (y, gx, gw, gb)
    if op == "quant":
        return fs.quantize_fp8(s["x"], block_rows=s["block"], dtype=s["fmt"], transpose=s["transpose"])
    if op == "product":
        return fs.fp8_matmul(*fs.quantize_fp8(s["x"]), *s["W"])
    if op == "linear":
        y = fs.fp8_matmul(*fs.quantize_fp8(s["x"]), *s["W"])
        gx = fs.fp8_matmul(*fs.quantize_fp8(s["g"], dtype=E5M2), *s["Wt"])
        gW = fs.fp8_matmul(*fs.quantize_fp8(s["g"], dtype=E5M2, transpose=True), *fs.quantize_fp8(s["x"], transpose=True),
                           out_dtype=torch.float32)
        return y, gx, gW
    return fs.sample_fp8(*s["h"], *s["W"], s["temp"], s["seed"], s["step"], bias=s["bias"])


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op, width = case["op"], {"bf16": 2, "fp16": 2, "fp32": 4}
    if op in ("norm8", "norm", "normgrad"):
        n, d, w = case["n"], case["d"], width[case["type"]]
        vectors = (1 if case["rms"] else 2) * d * width[case.get("wtype", "fp32")]
        stats = (4 if case["rms"] else 8) * n
        if op == "norm8":
            return dict(bytes=n * d * (w + 1) + vectors + 4 * n * -(-d // 128), flops=6 * n * d)
        if op == "norm":
            return dict(bytes=2 * n * d * w + vectors + stats, flops=6 * n * d)
        return dict(bytes=4 * n * d * w + 2 * vectors, flops=18 * n * d)
    if op == "quant":
        r, c = (case["cols"], case["rows"]) if case["transpose"] else (case["rows"], case["cols"])
        return dict(bytes=r * c * (width[case["type"]] + 1) + 4 * -(-r // case["block"]) * -(-c // 128), flops=3 * r * c)
    if op in ("product", "linear"):
        T, k, n = case["T"], case["k"], case["n"]
        scales = 4 * -(-k // 128) * -(-n // 128)
        if op == "product":
            return dict(bytes=width[case["type"]] * T * k + n * k + scales + 2 * T * n, flops=2 * T * n * k)
        return dict(bytes=2 * T * k + 2 * T * n + n * k + scales + 2 * T * n + 2 * T * k + 4 * n * k, flops=6 * T * n * k)
    B, d, V = case["B"], case["d"], case["V"]
    bias = {"none": 0, "shared": 4 * V, "rows": 4 * B * V}[case["bias"]]
    scales = 4 * -(-d // 128) * (B + -(-V // 128))
    return dict(bytes=V * d + B * d + scales + bias + 16 * B, flops=2 * B * V * d)


# ------------------------------------------------------------------ by definition, in 64 bits
def _exact_round(v, fmt):
    """The nearest values of an 8-bit type to v (fp64, within its range), ties to even."""
    bits, lowest = (3, -6) if fmt == E4M3 else (2, -14)
    power = torch.frexp(v)[1].sub(1).clamp(min=lowest) - bits
    step = (power.long() + 1023 << 52).view(torch.float64)                      # two to this power
    return torch.round(v / step) * step


def _exact_quantised(x, block, fmt):
    """(values of q, scales, what they stand for): scale and reciprocal rounded to 32 bits, as they are kept."""
    r, c = x.shape
    rows, cols = torch.arange(r, device=DEV) // block, torch.arange(c, device=DEV) // 128
    size = torch.nn.functional.pad(x.double().abs(), (0, -c % 128, 0, -r % block))
    top = size.unflatten(1, (-1, 128)).amax(2).unflatten(0, (-1, block)).amax(1)
    scale = torch.clamp((top / LARGEST[fmt]).float(), min=2.0 ** -100).double()
    inverse = (1.0 / scale).float().double()
    q = _exact_round((x.double() * inverse[rows][:, cols]).float().double(), fmt)
    return q, scale, q * scale[rows][:, cols]


def _exact_values(pair):
    q, scale = pair
    rows = torch.arange(q.shape[0], device=DEV) * scale.shape[0] // q.shape[0] if scale.shape[0] == q.shape[0] \
        else torch.arange(q.shape[0], device=DEV) // 128
    return q.double() * scale.double()[rows].repeat_interleave(128, 1)[:, :q.shape[1]]


def _exact_norm(s):
    x = s["x"].double()
    centre = torch.zeros(x.shape[0], dtype=torch.float64, device=DEV) if s["rms"] else x.mean(1)
    spread = torch.linalg.vector_norm(x - centre.unsqueeze(1), dim=1).square() / x.shape[1]
    rstd = 1.0 / torch.sqrt(spread + EPS)
    hat = torch.einsum("nd,n->nd", x - centre.unsqueeze(1), rstd)
    y = hat * s["w"].double() + (0.0 if s["b"] is None else s["b"].double())
    if s["op"] == "norm8":
        return _exact_quantised(y.float(), 1, E4M3)[:2]
    if s["op"] == "norm":
        return (y, rstd) if s["rms"] else (y, centre, rstd)
    g = s["g"].double()
    a = g * s["w"].double()
    d = x.shape[1]
    gx = a - hat * (torch.einsum("nd,nd->n", a, hat) / d).unsqueeze(1)
    if not s["rms"]:
        gx = gx - (a.sum(1) / d).unsqueeze(1)
    out = (y, gx * rstd.unsqueeze(1), torch.einsum("nd,nd->d", g, hat))
    return out if s["rms"] else out + (g.sum(0),)


def _exact_sample(s):
    logits = _exact_values(s["h"]).matmul(_exact_values(s["W"]).T)
    if s["bias"] is not None:
        logits = logits + s["bias"].double()
    B, V = logits.shape
    v = torch.arange(V, device=DEV).repeat(B, 1)
    x0, x1 = v // 4, torch.arange(B, device=DEV).unsqueeze(1).expand(B, V).clone()
    x2, x3 = torch.full_like(v, s["step"] % 2 ** 32), torch.full_like(v, s["step"] // 2 ** 32)

    def product(m, x):
        """(high, low) 32 bits of m x, by halves of 16 bits."""
        lo, hi = m * (x % 65536), m * (x // 65536)
        total = lo // 65536 + hi
        return total // 65536, total % 65536 * 65536 + lo % 65536

    for i in range(10):
        ka, kb = (s["seed"] + i * 0x9E3779B9) % 2 ** 32, (s["seed"] // 2 ** 32 + i * 0xBB67AE85) % 2 ** 32
        (ha, la), (hb, lb) = product(0xD2511F53, x0), product(0xCD9E8D57, x2)
        x0, x1, x2, x3 = hb.bitwise_xor(x1).bitwise_xor(ka), lb, ha.bitwise_xor(x3).bitwise_xor(kb), la
    word = torch.stack((x0, x1, x2, x3)).gather(0, (v % 4).unsqueeze(0)).squeeze(0)
    u = (2 * (word // 512) + 1).double() / 2 ** 24
    z = logits / s["temp"].double().unsqueeze(1) - (-u.log()).log()
    top = z.argmax(1)
    return top, z.gather(1, top.unsqueeze(1)).squeeze(1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("norm8", "norm", "normgrad"):
        return _exact_norm(s)
    if op == "sample":
        return _exact_sample(s)
    if op == "quant":
        return _exact_quantised(s["x"].T if s["transpose"] else s["x"], s["block"], s["fmt"])[:2]
    x, W = s["x"], _exact_values(s["W"])
    y = _exact_quantised(x, 1, E4M3)[2].matmul(W.T)
    if op == "product":
        return y
    gx = _exact_quantised(s["g"], 1, E5M2)[2].matmul(_exact_values(s["Wt"]).T)
    gW = _exact_quantised(s["g"].T, 1, E5M2)[2].matmul(_exact_quantised(x.T, 1, E4M3)[2].T)
    return y, gx, gW
