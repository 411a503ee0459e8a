"""Layer norm and its backward pass on the GPU against their fp64 forms.

Tolerances (u = 2^-24, half a step of fp32 relative to the value; 2^-8 and 2^-11 for
bf16 and fp16).  A thread adds up to 32 terms in turn, then threads are joined
in at most 10 + 1 steps: a sum of terms t has an error of at most
S = (32 + 11 + 2) u of sum |t|.

* mean: S mean|x| + u |mean|.  A centred value: u |x - mean| beside that.
* rstd: half the relative error of its square sum (that of the squares: twice a
  centred value's, S, 2u) and 3 steps for the root and the product by 1 / d.
* y = xh w + b: the errors of xh, 2u |xh w|, u |y|, and the result's rounding.
* gradients: a = g w is rounded once (u |a|); its two means have errors of
  S mean|a| and S mean|a xh| + mean(|a| err(xh)); the three terms of grad_x are
  combined in three roundings of their magnitudes.
* the weight's gradient: (rows of a block + blocks / 16 + 16 + 8) u of sum |g xh| besides
  sum |g| err(xh).
"""

import numpy as np
import pytest

from _helpers import to_device
from oracle import fp8
from test_gpu_fp8 import HALF, U, dtype_of, f64, on_device, values

pytestmark = pytest.mark.gpu

S = 45 * U
EPS = 1e-5
# Half the least step of a type: below 2^-14 fp16's values lie 2^-24 apart, whatever
# the value, so a rounding there is off by up to 2^-25 (bf16 and fp32: 2^-134, 2^-150).
LEAST = {"fp32": 2.0 ** -150, "bf16": 2.0 ** -134, "fp16": 2.0 ** -25}


class Case:
    def __init__(self, n, d, kind, w_kind, rms, affine=True, seed=0):
        rng = np.random.default_rng(seed + 13 * n + d)
        self.n, self.d, self.kind, self.w_kind, self.rms = n, d, kind, w_kind, rms
        cast = lambda v, k: values_as(v, k)  # noqa: E731
        size = np.exp2(rng.integers(-6, 7, (n, 1)))
        self.x = cast((rng.standard_normal((n, d)) + 0.5) * size, kind)
        self.g = cast(rng.standard_normal((n, d)) * 0.01, kind)
        self.w = cast(1 + 0.3 * rng.standard_normal(d), w_kind) if affine else None
        self.b = cast(0.3 * rng.standard_normal(d), w_kind) if affine and not rms else None

    def tensors(self, torch, pad=0, shift=0):
        put = lambda v: None if v is None else to_device(v, torch).to(dtype_of(torch, self.w_kind))  # noqa: E731
        return (on_device(torch, self.x, self.kind, pad, shift), on_device(torch, self.g, self.kind, pad, shift), put(self.w),
                put(self.b))

    def reference(self):
        """(Norm, error of mean, relative error of rstd, error of xh, error of y before its rounding)"""
        x = self.x.astype(np.float64)
        r = fp8.layer_norm(x, self.w, self.b, EPS, self.rms)
        e_mean = np.zeros(self.n) if self.rms else S * np.abs(x).mean(1) + U * np.abs(r.mean)
        centred = x - r.mean[:, None]
        e_c = (0 if self.rms else 1) * (U * np.abs(centred) + e_mean[:, None])
        square = (centred ** 2).sum(1)
        e_square = (2 * np.abs(centred) * e_c + e_c ** 2).sum(1) + (S + 2 * U) * square
        e_rstd = 0.5 * e_square / self.d * r.rstd ** 2 * 1.01 + 8 * U
        e_xh = e_c * r.rstd[:, None] * 1.01 + np.abs(r.xh) * (e_rstd[:, None] + 2 * U)
        w = np.ones(self.d) if self.w is None else np.abs(self.w.astype(np.float64))
        e_y = e_xh * w + 2 * U * np.abs(r.xh) * w + U * np.abs(r.y)
        return r, e_mean, e_rstd, e_xh, e_y


def values_as(v, kind):
    v = np.asarray(v, np.float32)
    if kind == "fp16":
        return v.astype(np.float16).astype(np.float32)
    if kind == "bf16":
        from lm_head_exact_gb300 import synthetic
        return synthetic.bf16_bits_to_f32(synthetic.bf16_bits(v))
    return v


def near(got, want, tol, what):
    got = f64(got)
    assert got.shape == want.shape
    over = np.abs(got - want) / np.maximum(tol, 1e-300)
    assert np.all(np.abs(got - want) <= tol), f"{what}: {over.max():.3g} times the tolerance at {np.unravel_index(over.argmax(), over.shape)}"


KINDS = [("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16"), ("fp32", "fp32")]
SHAPES = [(1, 1), (3, 2), (5, 8), (2, 31), (9, 64), (33, 257), (7, 264), (513, 1000), (40, 1024), (600, 1025), (3, 2056), (6, 4096),
          (530, 4096), (2, 8192), (3, 8200), (2, 9001), (520, 12304), (2, 32768), (2, 32761)]


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("kind,w_kind", KINDS)
@pytest.mark.parametrize("n,d", SHAPES)
def test_layer_norm_and_gradients(fs, torch_cuda, n, d, kind, w_kind, rms):
    torch = torch_cuda
    c = Case(n, d, kind, w_kind, rms)
    for pad, shift in ((0, 0), (3, 1)) if n * d < 100000 else ((0, 0),):
        x, g, w, b = c.tensors(torch, pad, shift)
        y, mean, rstd = fs.layer_norm(x, w, b, eps=EPS, rms=rms)
        r, e_mean, e_rstd, e_xh, e_y = c.reference()
        what = f"{n} x {d} {kind} {w_kind} rms={rms} pad={pad}"
        near(rstd, r.rstd, e_rstd * r.rstd, what + " rstd")
        if rms:
            assert mean is None
        else:
            near(mean, r.mean, e_mean, what + " mean")
        near(y, r.y, e_y + HALF[kind] * np.abs(r.y) + LEAST[kind], what + " y")
        check_gradients(c, r, e_rstd, e_xh, fs.layer_norm_backward(g, x, w, mean, rstd), what)


def check_gradients(c, r, e_rstd, e_xh, got, what):
    gx, gw, gb = got
    g = c.g.astype(np.float64)
    w = np.ones(c.d) if c.w is None else c.w.astype(np.float64)
    a = np.abs(g * w)
    want = fp8.layer_norm_gradients(g, r, c.w, c.rms)
    xh = np.abs(r.xh)
    m_a = np.abs((g * w).mean(1)) * (not c.rms)
    m_ax = np.abs((g * w * r.xh).mean(1))
    e_ma = (S + 2 * U) * a.mean(1) * (not c.rms)
    e_max = (S + 3 * U) * (a * xh).mean(1) + (a * e_xh).mean(1)
    terms = a + m_a[:, None] + xh * m_ax[:, None]
    e = U * a + e_ma[:, None] + e_xh * m_ax[:, None] + xh * e_max[:, None] + 4 * U * terms
    tol = r.rstd[:, None] * (e * 1.01 + terms * (e_rstd[:, None] + U)) + HALF[c.kind] * np.abs(want[0]) + LEAST[c.kind]
    near(gx, want[0], tol, what + " grad_x")
    steps = (c.n / 1 + 304 / 16 + 24) * U
    near(gw, want[1], steps * (np.abs(g) * xh).sum(0) + (np.abs(g) * e_xh).sum(0) * 1.01 + HALF[c.w_kind] * np.abs(want[1]) + LEAST[c.w_kind],
         what + " grad_weight")
    near(gb, want[2], steps * np.abs(g).sum(0) + HALF[c.w_kind] * np.abs(want[2]) + LEAST[c.w_kind], what + " grad_bias")


def test_without_weight_and_bias(fs, torch_cuda):
    torch = torch_cuda
    for rms in (False, True):
        c = Case(20, 300, "bf16", "fp32", rms, affine=False)
        x, g, _, _ = c.tensors(torch)
        y, mean, rstd = fs.layer_norm(x, eps=EPS, rms=rms)
        r, _, e_rstd, e_xh, e_y = c.reference()
        near(y, r.y, e_y + HALF["bf16"] * np.abs(r.y), "y")
        check_gradients(c, r, e_rstd, e_xh, fs.layer_norm_backward(g, x, None, mean, rstd), "no weight")
        gx, gw, gb = fs.layer_norm_backward(g, x, None, mean, rstd, need_weight=False, need_bias=False)
        assert gw is None and gb is None and bool((gx == fs.layer_norm_backward(g, x, None, mean, rstd)[0]).all())
        gx, gw, gb = fs.layer_norm_backward(g, x, None, mean, rstd, need_x=False, weight_dtype=torch.bfloat16)
        assert gx is None and gw.dtype == torch.bfloat16


def test_many_rows(fs, torch_cuda):
    """Blocks that go through many rows each, of every width class."""
    torch = torch_cuda
    for n, d, kind in ((20000, 64, "bf16"), (9001, 520, "fp16"), (5000, 2048, "bf16"), (3001, 1001, "fp32")):
        c = Case(n, d, kind, "fp32", False)
        x, g, w, b = c.tensors(torch)
        y, mean, rstd = fs.layer_norm(x, w, b, eps=EPS)
        r, _, e_rstd, e_xh, e_y = c.reference()
        near(y, r.y, e_y + HALF[kind] * np.abs(r.y) + LEAST[kind], f"{n} x {d} y")
        check_gradients(c, r, e_rstd, e_xh, fs.layer_norm_backward(g, x, w, mean, rstd), f"{n} x {d}")


def test_large_mean(fs, torch_cuda):
    """Rows far from zero: the squares are taken about the mean."""
    torch = torch_cuda
    rng = np.random.default_rng(0)
    x = (1000 + rng.standard_normal((4, 512))).astype(np.float32)
    y, _, rstd = fs.layer_norm(to_device(x, torch), eps=0.0)
    r = fp8.layer_norm(x, eps=0.0)
    # a centred value is within S * 1000 + u of its own; relative to a spread of 1 that is 3e-3
    assert np.abs(f64(y) - r.y).max() < 1.01 * S * 1000 * 1.5 + 1e-4


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("n,d", [(1, 1), (3, 130), (16, 4096), (600, 264), (515, 1001), (5, 8192), (2, 9000), (3, 32761), (520, 4097)])
def test_quantised_norm(fs, torch_cuda, n, d, kind, rms):
    """The quantiser's values of the norm's fp32 result.  That result is within
    e_y of its exact value, so each 8-bit value is that of some number in
    that range: its distance to the exact y is half a step of e4m3 (2^-4, or 2^-10 scales
    near zero) and e_y; and the scale is amax / 448 within e_y."""
    torch = torch_cuda
    c = Case(n, d, kind, "fp32", rms)
    for pad, shift in ((0, 0), (5, 3)):
        x, _, w, b = c.tensors(torch, pad, shift)
        q, scale = fs.layer_norm_fp8(x, w, b, eps=EPS, rms=rms)
        r, _, _, _, e_y = c.reference()
        s, v = f64(scale), f64(q.float())
        blocks = -(-d // 128)
        wide = np.zeros((n, blocks * 128))
        wide[:, :d] = np.abs(r.y)
        e_wide = np.zeros((n, blocks * 128))
        e_wide[:, :d] = e_y
        amax, e_amax = wide.reshape(n, blocks, 128).max(2), e_wide.reshape(n, blocks, 128).max(2)
        assert s.shape == (n, blocks)
        assert np.all(np.abs(s - np.maximum(amax / 448, 2.0 ** -100)) <= e_amax / 448 + U * s)
        each = np.repeat(s, 128, 1)[:, :d]
        assert np.all(np.abs(v) <= 448)
        assert np.all(np.abs(v * each - r.y) <= np.maximum(2.0 ** -4 * (np.abs(r.y) + e_y), 2.0 ** -10 * each) * (1 + 4 * U) + 2 * e_y)
        if kind == "fp32" and d % 4 == 0 and shift == 0:
            # the same kernel's fp32 result, quantised by the quantiser, bit for bit (rows off
            # a 16-byte boundary are summed in another order where y is written, which
            # moves mean and rstd within their tolerances)
            y, _, _ = fs.layer_norm(x, w, b, eps=EPS, rms=rms)
            q2, s2 = fs.quantize_fp8(y)
            assert bool((s2 == scale).all()) and bool((q2.view(torch.uint8) == q.view(torch.uint8)).all())


def test_norm_ends(fs, torch_cuda):
    """Rows of one value, of NaN and of infinity stay in their rows."""
    torch = torch_cuda
    x = torch.randn((6, 256), device="cuda")
    clean, _, _ = fs.layer_norm(x)
    x[1] = 3.0
    x[2, 7] = float("nan")
    x[3, 9] = float("inf")
    y, mean, rstd = fs.layer_norm(x)
    assert bool((y[1] == 0).all()) and abs(rstd[1].item() - 1e5 ** 0.5) < 1e-2
    assert bool(y[2].isnan().all()) and bool(y[3].isnan().all())
    assert bool((y[[0, 4, 5]] == clean[[0, 4, 5]]).all())
    q, scale = fs.layer_norm_fp8(x)
    assert bool(q[2].float().isnan().all()) and bool((q[1].float() == 0).all())
    gx, gw, gb = fs.layer_norm_backward(torch.ones_like(x), x, None, mean, rstd)
    assert bool(gw.isnan().all()) and bool((gb == 6).all()) and bool(gx[[0, 1, 4, 5]].isfinite().all())


def test_in_place(fs, torch_cuda):
    torch = torch_cuda
    for d in (64, 1001, 4096):
        x, g = torch.randn((50, d), device="cuda").bfloat16(), torch.randn((50, d), device="cuda").bfloat16()
        y, mean, rstd = fs.layer_norm(x)
        gx, gw, gb = fs.layer_norm_backward(g, x, None, mean, rstd)
        same = g.clone()
        gx2, gw2, _ = fs.layer_norm_backward(same, x, None, mean, rstd, out=same)
        assert gx2 is same and bool((gx2 == gx).all()) and bool((gw2 == gw).all())
        own = x.clone()
        y2, _, _ = fs.layer_norm(own, out=own)
        assert y2 is own and bool((own == y).all())


def test_nothing(fs, torch_cuda):
    torch = torch_cuda
    x = torch.empty((0, 40), device="cuda")
    y, mean, rstd = fs.layer_norm(x)
    assert y.shape == (0, 40) and rstd.shape == (0,)
    gx, gw, gb = fs.layer_norm_backward(x, x, None, mean, rstd)
    assert gx.shape == (0, 40) and bool((gw == 0).all()) and bool((gb == 0).all())
