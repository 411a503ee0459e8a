"""The 8-bit path on the GPU against its fp64 forms.

Tolerances (u = 2^-24, half a step of fp32 relative to the value; 2^-8 and 2^-11
for bf16 and fp16):

* quantising is defined by roundings that are each to nearest: bits agree;
* a product's block of 128 products, each exact in fp32, is summed in the tensor
  cores, where an addition may be cut: 128 x 2u of the sum of its terms'
  magnitudes; its scale is rounded once, multiplied in and added to nearest, once for each block:
  (2 + blocks) u of them; then the result's own rounding.
"""

import numpy as np
import pytest

from _helpers import to_device
from lm_head_exact_gb300 import synthetic
from oracle import fp8, sampler

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {"fp32": 2.0 ** -24, "bf16": 2.0 ** -8, "fp16": 2.0 ** -11}


def dtype_of(torch, name):
    return {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16, fp8.E4M3: torch.float8_e4m3fn,
            fp8.E5M2: torch.float8_e5m2}[name]


def values(rng, rows, cols, kind):
    """Random values of a type, as fp32: rows of very different sizes, some
    zeros, a block of zeros."""
    x = (rng.standard_normal((rows, cols)) * np.exp2(rng.integers(-8, 5, (rows, 1)))).astype(np.float32)
    x[rng.random((rows, cols)) < 0.05] = 0.0
    x[0, :min(cols, 128)] = 0.0
    if kind == "bf16":
        return synthetic.bf16_bits_to_f32(synthetic.bf16_bits(x))
    return x.astype(np.float16).astype(np.float32) if kind == "fp16" else x


def on_device(torch, x, kind, pad=0, shift=0):
    """x as a tensor of a type whose rows lie `pad` elements further apart than
    they are long, `shift` elements into its memory."""
    rows, cols = x.shape
    flat = torch.full((rows * (cols + pad) + shift,), float("nan"), dtype=dtype_of(torch, kind), device="cuda")
    view = flat[shift:].view(rows, cols + pad)[:, :cols]
    view.copy_(to_device(x, torch))
    return view


def f64(t):
    return t.detach().cpu().to(dtype=__import__("torch").float64).numpy()


QUANT_SHAPES = [(1, 1), (1, 128), (2, 17), (3, 4096), (16, 130), (127, 129), (128, 128), (129, 1000), (300, 264),
                (2047, 72)]


@pytest.mark.parametrize("fmt", [fp8.E4M3, fp8.E5M2])
@pytest.mark.parametrize("kind,pad,shift", [("bf16", 0, 0), ("bf16", 3, 1), ("fp16", 8, 8), ("fp32", 0, 0), ("fp32", 1, 2)])
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("rows,cols", QUANT_SHAPES)
def test_quantise_bits(fs, torch_cuda, rows, cols, block, transpose, kind, pad, shift, fmt):
    torch = torch_cuda
    x = values(np.random.default_rng(rows * 7 + cols), rows, cols, kind)
    q, scale = fs.quantize_fp8(on_device(torch, x, kind, pad, shift), block_rows=block, dtype=dtype_of(torch, fmt),
                               transpose=transpose)
    want = fp8.quantise(x.T if transpose else x, block, fmt)
    assert q.shape == want.q.shape and q.dtype == dtype_of(torch, fmt) and q.stride(0) % 16 == 0 or q.shape[0] == 1
    np.testing.assert_array_equal(f64(scale), want.scale)
    np.testing.assert_array_equal(f64(q.float()), want.q)


def test_quantise_many_rows(fs, torch_cuda):
    """Rows beyond what one launch's grid takes (65535 tiles of 16 or 128)."""
    torch = torch_cuda
    n = 65535 * 128 + 77
    x = torch.zeros((n, 8), dtype=torch.bfloat16, device="cuda")
    x[:, 3] = (torch.arange(n, device="cuda") % 251 + 1).bfloat16()
    for block in (1, 128):
        q, scale = fs.quantize_fp8(x, block_rows=block)
        got = q[:, 3].float() * scale[:, 0].repeat_interleave(block)[:n]
        assert bool(((got - x[:, 3].float()).abs() <= x[:, 3].float() * 0.0626).all())
    q, scale = fs.quantize_fp8(x, transpose=True)
    got = q[3].float() * scale[3].repeat_interleave(128)[:n]
    assert bool(((got - x[:, 3].float()).abs() <= x[:, 3].float() * 0.0626).all())
    assert bool((scale[0] == 2.0 ** -100).all())


def test_quantise_ends(fs, torch_cuda):
    torch = torch_cuda
    x = np.zeros((4, 130), np.float32)
    x[1, 5], x[2, 5], x[3, :2] = np.nan, np.inf, (1e-38, -3e38)
    x[1, 6] = 2.0
    for transpose in (False, True):
        q, scale = fs.quantize_fp8(to_device(x.T if transpose else x, torch), transpose=transpose)
        want = fp8.quantise(x)
        np.testing.assert_array_equal(f64(scale), want.scale)
        np.testing.assert_array_equal(f64(q.float()), want.q)


def test_quantise_leaves_what_lies_behind_rows(fs, torch_cuda):
    torch = torch_cuda
    x = torch.randn((37, 77), device="cuda").bfloat16()
    for transpose, (R, C) in ((False, (37, 77)), (True, (77, 37))):
        memory = torch.full((R + 2, 96), 0x55, dtype=torch.uint8, device="cuda")
        scale = torch.full((R, 3), -1.0, device="cuda")
        q = memory.view(torch.float8_e4m3fn)[1:-1, :C]
        fs.quantize_fp8(x, transpose=transpose, out=(q, scale[:, :1]))
        after = memory.clone()
        after[1:-1, :C] = 0x55
        assert bool((after == 0x55).all()) and bool((scale[:, 1:] == -1).all()) and bool((scale[:, 0] > 0).all())


class Operand:
    """A quantised matrix, on the device and as the oracle's."""

    def __init__(self, torch, rows, cols, block=1, fmt=fp8.E4M3, seed=0, spread=2):
        rng = np.random.default_rng(seed + rows * 31 + cols)
        x = (rng.standard_normal((rows, cols)) * np.exp2(rng.integers(-spread, spread + 1, (rows, 1)))).astype(np.float32)
        self.ref = fp8.quantise(x, block, fmt)
        pitch = (cols + 15) // 16 * 16 + 16 * (seed % 2)
        memory = torch.full((rows, pitch), 0x7f, dtype=torch.uint8, device="cuda")   # NaNs behind the rows
        self.q = memory.view(dtype_of(torch, fmt))[:, :cols]
        self.q.copy_(torch.from_numpy(self.ref.q).float().to(dtype_of(torch, fmt)).cuda())
        self.scale = torch.from_numpy(self.ref.scale.astype(np.float32)).cuda()
        if seed % 2 == 0 and block == 1:
            self.scale = self.scale.t().contiguous().t()


def check_product(got, a, b, kind, what):
    out, size = fp8.product(a.ref, b.ref)
    blocks = a.ref.scale.shape[1]
    tol = (2 * 128 + 2 + blocks) * U * size * 1.01 + HALF[kind] * np.abs(out)
    err = np.abs(f64(got) - out)
    over = err / np.maximum(tol, 1e-300)
    assert np.all(err <= tol), f"{what}: {over.max():.3g} times the tolerance at {np.unravel_index(over.argmax(), over.shape)}"


PRODUCT_SHAPES = [(1, 1, 1), (1, 64, 128), (2, 5, 33), (16, 256, 512), (17, 130, 200), (31, 300, 129), (64, 1000, 1024),
                  (127, 129, 640), (128, 128, 128), (129, 257, 384), (300, 1001, 1000), (16, 6144, 256), (1, 4100, 2050),
                  (600, 520, 264), (5, 64, 16384)]


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("m,n,k", PRODUCT_SHAPES)
def test_product(fs, torch_cuda, m, n, k, block, kind):
    torch = torch_cuda
    a = Operand(torch, m, k, seed=k % 2)
    b = Operand(torch, n, k, block, seed=(n + 1) % 2)
    got = fs.fp8_matmul(a.q, a.scale, b.q, b.scale, out_dtype=dtype_of(torch, kind))
    check_product(got, a, b, kind, f"{m} x {n} x {k} block {block}")
    assert fs.device_error() == 0


@pytest.mark.parametrize("fa,fb", [(fp8.E4M3, fp8.E5M2), (fp8.E5M2, fp8.E4M3), (fp8.E5M2, fp8.E5M2)])
def test_product_types(fs, torch_cuda, fa, fb):
    torch = torch_cuda
    for m, n, k in ((40, 200, 300), (3, 70, 1000)):
        a, b = Operand(torch, m, k, fmt=fa), Operand(torch, n, k, 128, fmt=fb)
        check_product(fs.fp8_matmul(a.q, a.scale, b.q, b.scale, out_dtype=torch.float32), a, b, "fp32", f"{fa} {fb}")


@pytest.mark.parametrize("m,n,k", [(2048, 2176, 512), (1500, 4099, 384), (4000, 300, 1000)])
def test_product_of_many_tiles(fs, torch_cuda, m, n, k):
    """More tiles than the GPU holds at a time."""
    torch = torch_cuda
    a, b = Operand(torch, m, k), Operand(torch, n, k, 128)
    check_product(fs.fp8_matmul(a.q, a.scale, b.q, b.scale, out_dtype=torch.float32), a, b, "fp32", f"{m} x {n} x {k}")
    c = Operand(torch, n, k, 1)
    check_product(fs.fp8_matmul(a.q, a.scale, c.q, c.scale), a, c, "bf16", f"{m} x {n} x {k} by rows")


@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("m,n,k", [(1, 33000, 4200), (9, 8200, 4100), (16, 6145, 4112), (31, 4100, 4200), (20, 3000, 8200),
                                   (64, 1000, 16400), (33, 130, 80000), (64, 7, 1000003), (7, 10, 300000), (65, 20000, 1100)])
def test_product_of_few_rows(fs, torch_cuda, m, n, k, block):
    """Few rows of a, with more of b to read than the smallest products have."""
    torch = torch_cuda
    a, b = Operand(torch, m, k, seed=k % 2), Operand(torch, n, k, block, seed=n % 2)
    for kind in ("fp32", "bf16"):
        check_product(fs.fp8_matmul(a.q, a.scale, b.q, b.scale, out_dtype=dtype_of(torch, kind)), a, b, kind, f"{m} x {n} x {k}")
    assert fs.device_error() == 0


def test_product_into_a_view(fs, torch_cuda):
    """Rows further apart than they are long, off any alignment; nothing else is
    written."""
    torch = torch_cuda
    for kind in ("bf16", "fp32"):
        for m, n, k in ((33, 75, 200), (200, 300, 512), (7, 1, 64)):
            a, b = Operand(torch, m, k), Operand(torch, n, k, 128)
            memory = torch.full((m + 2, n + 9), 7.0, dtype=dtype_of(torch, kind), device="cuda")
            out = memory[1:-1, 5:5 + n]
            fs.fp8_matmul(a.q, a.scale, b.q, b.scale, out=out)
            check_product(out, a, b, kind, "view")
            memory[1:-1, 5:5 + n] = 7.0
            assert bool((memory == 7.0).all())


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("m,n,k", [(65, 193, 128), (129, 71, 200), (300, 1000, 256), (257, 6, 100), (70, 449, 17),
                                   (1500, 2049, 128)])
def test_product_into_an_aligned_view(fs, torch_cuda, m, n, k, block, kind):
    """Rows on 16-byte boundaries that end anywhere: nothing behind them, or
    behind the last one, is written."""
    torch = torch_cuda
    a, b = Operand(torch, m, k, seed=n % 2), Operand(torch, n, k, block, seed=m % 2)
    memory = torch.full((m + 2, (n + 31) // 16 * 16), 7.0, dtype=dtype_of(torch, kind), device="cuda")
    out = memory[1:-1, 8:8 + n]
    fs.fp8_matmul(a.q, a.scale, b.q, b.scale, out=out)
    check_product(out, a, b, kind, "aligned view")
    memory[1:-1, 8:8 + n] = 7.0
    assert bool((memory == 7.0).all()) and fs.device_error() == 0


def test_product_keeps_nan_and_infinity_in_their_rows(fs, torch_cuda):
    torch = torch_cuda
    a, b = Operand(torch, 20, 300), Operand(torch, 140, 300, 128)
    clean = fs.fp8_matmul(a.q, a.scale, b.q, b.scale, out_dtype=torch.float32)
    bits = a.q.view(torch.uint8).clone()
    bits[3, 290] = 0x7f                                        # a NaN in one row of a
    scale = a.scale.clone()
    scale[5, 1] = float("inf")
    got = fs.fp8_matmul(bits.view(torch.float8_e4m3fn) if bits.stride(0) % 16 == 0 else _pitched(torch, bits), scale,
                        b.q, b.scale, out_dtype=torch.float32)
    assert bool(got[3].isnan().all()) and not bool(got[5].isfinite().any())
    rows = [i for i in range(20) if i not in (3, 5)]
    assert bool((got[rows] == clean[rows]).all())


def test_large_product_of_few_rows_keeps_nan_and_infinity_in_their_rows(fs, torch_cuda):
    torch = torch_cuda
    a, b = Operand(torch, 20, 4300), Operand(torch, 4200, 4300, 128)
    clean = fs.fp8_matmul(a.q, a.scale, b.q, b.scale, out_dtype=torch.float32)
    bits = a.q.view(torch.uint8).clone()
    bits[3, 4290] = 0x7f
    scale = a.scale.clone()
    scale[5, 1] = float("inf")
    got = fs.fp8_matmul(_pitched(torch, bits), scale, b.q, b.scale, out_dtype=torch.float32)
    assert bool(got[3].isnan().all()) and not bool(got[5].isfinite().any())
    rows = [i for i in range(20) if i not in (3, 5)]
    assert bool((got[rows] == clean[rows]).all())


def _pitched(torch, bits):
    wide = torch.zeros((bits.shape[0], (bits.shape[1] + 15) // 16 * 16), dtype=torch.uint8, device="cuda")
    wide[:, :bits.shape[1]] = bits
    return wide.view(torch.float8_e4m3fn)[:, :bits.shape[1]]


def test_product_of_nothing(fs, torch_cuda):
    torch = torch_cuda
    f8 = torch.float8_e4m3fn
    empty = lambda r, c: (torch.empty((r, c), dtype=f8, device="cuda"), torch.empty((r, -(-c // 128)), device="cuda"))  # noqa: E731
    assert fs.fp8_matmul(*empty(0, 64), *empty(5, 64)).shape == (0, 5)
    assert fs.fp8_matmul(*empty(5, 64), *empty(0, 64)).shape == (5, 0)
    assert bool((fs.fp8_matmul(*empty(5, 0), *empty(3, 0)) == 0).all())
    memory = torch.full((4, 6), 3.0, device="cuda")
    fs.fp8_matmul(*empty(4, 0), *empty(5, 0), out=memory[:, :5])
    assert bool((memory[:, :5] == 0).all()) and bool((memory[:, 5] == 3).all())
    q, s = fs.quantize_fp8(torch.empty((0, 40), device="cuda"))
    assert q.shape == (0, 40) and s.shape == (0, 1)


def test_linear_layer_gradients(fs, torch_cuda):
    """The three products of a linear layer's training step on the values that
    its operands stand for: W laid out twice from the same blocks."""
    torch = torch_cuda
    T, k, n = 77, 200, 300
    rng = np.random.default_rng(0)
    x, W, g = (values(rng, *s, "bf16") for s in ((T, k), (n, k), (T, n)))
    X, Wd, G = (on_device(torch, v, "bf16") for v in (x, W, g))
    e5 = torch.float8_e5m2
    W8, Wt8 = fs.quantize_fp8(Wd, block_rows=128), fs.quantize_fp8(Wd, block_rows=128, transpose=True)
    assert bool((W8[0].float().t() == Wt8[0].float()).all()) and bool((W8[1].t() == Wt8[1]).all())
    gx = fs.fp8_matmul(*fs.quantize_fp8(G, dtype=e5), *Wt8, out_dtype=torch.float32)
    gW = fs.fp8_matmul(*fs.quantize_fp8(G, dtype=e5, transpose=True), *fs.quantize_fp8(X, transpose=True), out_dtype=torch.float32)
    pairs = ((gx, fp8.quantise(g, 1, fp8.E5M2), fp8.quantise(W.T, 128)),
             (gW, fp8.quantise(g.T, 1, fp8.E5M2), fp8.quantise(x.T)))
    for got, a, b in pairs:
        out, size = fp8.product(a, b)
        assert np.all(np.abs(f64(got) - out) <= (2 * 128 + 2 + a.scale.shape[1]) * U * size * 1.01 + U * np.abs(out))


# ---------------------------------------------------------------- sampling
def sample_case(torch, B, d, V, block=128, bias=None, seed=0):
    rng = np.random.default_rng(seed + B + V)
    h = Operand(torch, B, d, 1, seed=seed, spread=0)
    W = Operand(torch, V, d, block, seed=seed + 1, spread=0)
    W.scale *= 1.5 / np.sqrt(d)
    W.ref = fp8.Quantised(W.ref.q, f64(W.scale), W.ref.q * fp8._spread(f64(W.scale), V, d, block))
    temp = rng.uniform(0.5, 1.5, B).astype(np.float32)
    if B > 3:
        temp[1], temp[2], temp[3] = 0.0, -1.0, np.nan
    b = None
    if bias == "shared":
        b = np.where(rng.random(V) < 0.3, -np.inf, rng.standard_normal(V)).astype(np.float32)
    elif bias == "rows":
        b = rng.standard_normal((B, V)).astype(np.float32)
        b[0] = -np.inf
    logits = fp8.product(h.ref, W.ref)[0]
    if b is not None:
        logits = logits + b
    return h, W, temp, b, logits


@pytest.mark.parametrize("bias", [None, "shared", "rows"])
@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("B,d,V", [(1, 64, 1000), (4, 200, 257), (5, 129, 4097), (33, 384, 3000), (128, 256, 1001),
                                   (200, 130, 600), (300, 512, 2049), (2, 16, 1)])
def test_samples(fs, torch_cuda, B, d, V, block, bias):
    from _helpers import compare
    torch = torch_cuda
    h, W, temp, b, logits = sample_case(torch, B, d, V, block, bias)
    bias_t = None if b is None else to_device(b, torch)
    for step in (0, 5):
        ids, mx = fs.sample_fp8(h.q, h.scale, W.q, W.scale, to_device(temp, torch), 1234, step, bias=bias_t)
        ref = sampler.sample_from_logits(logits, temp, 1234, step, np.arange(B), np.arange(V))
        compare(ids.cpu().numpy(), mx.cpu().numpy(), ref, what=f"8-bit head B={B} d={d} V={V}")
    assert fs.device_error() == 0


@pytest.mark.parametrize("B", [4, 40, 130, 300])
@pytest.mark.parametrize("what", ["flat", "peaked", "forbidden", "shifted"])
def test_samples_of_extreme_rows(fs, torch_cuda, B, what):
    """Rows whose scores are all noise, none, or far from zero: what is left
    out early does not change a sample."""
    from _helpers import compare
    torch = torch_cuda
    d, V = 128, 21001
    h, W, _, _, logits = sample_case(torch, B, d, V)
    rng = np.random.default_rng(B)
    temp = np.array([1.0, 0.0, 0.1, 1e3, 0.5, 30.0], np.float32)[np.arange(B) % 6]
    bias = np.zeros(V, np.float32)
    if what == "flat":
        h.scale.zero_()                                        # every logit 0: greedy takes the smallest id
        logits = np.zeros_like(logits)
    elif what == "peaked":
        bias[rng.integers(0, V, 5)] = 25.0
    elif what == "forbidden":
        bias[:] = -np.inf
        bias[rng.integers(0, V, 3)] = -4.0
    else:
        bias[:] = -60.0 + 40.0 * (rng.random(V) < 1e-3)
    ids, mx = fs.sample_fp8(h.q, h.scale, W.q, W.scale, to_device(temp, torch), 99, 7, bias=to_device(bias, torch))
    ref = sampler.sample_from_logits(logits + bias, temp, 99, 7, np.arange(B), np.arange(V))
    compare(ids.cpu().numpy(), mx.cpu().numpy(), ref, what=f"8-bit head, {what} rows, B={B}")
    if what == "flat":
        assert bool((ids.cpu()[torch.from_numpy(temp) == 0] == 0).all())
    assert fs.device_error() == 0


def test_samples_of_a_large_head(fs, torch_cuda):
    """All SMs with several tiles each, over a vocabulary that ends inside one."""
    from _helpers import compare
    torch = torch_cuda
    B, d, V = 20, 256, 128256 + 13
    h, W, temp, _, logits = sample_case(torch, B, d, V)
    ids, mx = fs.sample_fp8(h.q, h.scale, W.q, W.scale, to_device(temp, torch), 7, 3)
    compare(ids.cpu().numpy(), mx.cpu().numpy(), sampler.sample_from_logits(logits, temp, 7, 3, np.arange(B), np.arange(V)),
            what="large head")


def test_samples_of_no_vocabulary(fs, torch_cuda):
    torch = torch_cuda
    h, _ = Operand(torch, 3, 64), None
    W = torch.empty((0, 64), dtype=torch.float8_e4m3fn, device="cuda")
    ids, mx = fs.sample_fp8(h.q, h.scale, W, torch.empty((0, 1), device="cuda"), torch.ones(3, device="cuda"), 0, 0)
    assert ids.tolist() == [-1] * 3 and mx.tolist() == [-float("inf")] * 3
    ids, _ = fs.sample_fp8(h.q[:0], h.scale[:0], W, torch.empty((0, 1), device="cuda"), torch.ones(0, device="cuda"), 0, 0)
    assert ids.shape == (0,)


def test_samples_are_those_of_the_product(fs, torch_cuda):
    """The sampler scans the logits that the product forms: greedy rows return
    its largest, bit for bit."""
    torch = torch_cuda
    for B, d, V in ((16, 512, 3001), (140, 300, 5000)):
        h, W, _, _, _ = sample_case(torch, B, d, V)
        logits = fs.fp8_matmul(h.q, h.scale, W.q, W.scale, out_dtype=torch.float32)
        ids, mx = fs.sample_fp8(h.q, h.scale, W.q, W.scale, torch.zeros(B, device="cuda"), 0, 0)
        assert (mx - logits.max(1).values).abs().max().item() <= 1e-5
