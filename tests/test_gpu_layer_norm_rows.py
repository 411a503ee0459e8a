"""Layer norm over many rows, where a block goes through several: column sums
that are exact in fp32 whatever their order, results in place of inputs and
beside them, and short rows off 16-byte boundaries.

The exact cases: g, x and mean are whole numbers and rstd is 1, so that every
term g (x - mean) is one, and sums of their magnitudes stay below 2^24: fp32
holds each partial sum, and the result is equal to the sum in 64 bits.  A lost
or doubled row shows whatever the number of rows."""

import numpy as np
import pytest

from test_gpu_fp8 import HALF, dtype_of, f64
from test_gpu_layer_norm import EPS, LEAST, Case, check_gradients, near

pytestmark = pytest.mark.gpu


def _whole(torch, rng, n, d, kind, high, pad=0, shift=0):
    """Whole numbers in [-high, high] in a matrix whose rows lie `pad` further
    apart than they are long, `shift` elements into its memory."""
    v = rng.integers(-high, high + 1, (n, d)).astype(np.float32)
    flat = torch.full((n * (d + pad) + shift,), float("nan"), dtype=dtype_of(torch, kind), device="cuda")
    view = flat[shift:].view(n, d + pad)[:, :d]
    view.copy_(torch.from_numpy(v))
    return v.astype(np.float64), view


# (n, d, type, distance between g's memory and x's, in elements: where it is no multiple of 16 bytes, element by element)
SUMS = [(20000, 64, "bf16", 0), (20000, 65, "bf16", 0), (9001, 301, "fp16", 0), (6000, 33, "fp32", 0), (30001, 256, "bf16", 0),
        (9001, 520, "fp16", 0), (5000, 1000, "bf16", 0), (4999, 1001, "fp32", 0), (5000, 2048, "bf16", 0), (5003, 4096, "fp16", 0),
        (2000, 4096, "fp32", 0), (1999, 4097, "bf16", 0), (700, 7000, "fp32", 0), (913, 8192, "bf16", 0), (700, 9000, "fp16", 0),
        (620, 12304, "bf16", 0), (613, 12305, "bf16", 0), (5000, 65, "bf16", 1), (3000, 1001, "fp16", 3), (700, 9001, "fp32", 1)]


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("need_x", [True, False])
@pytest.mark.parametrize("n,d,kind,off", SUMS)
def test_column_sums_are_exact(fs, torch_cuda, n, d, kind, off, need_x, rms):
    torch = torch_cuda
    rng = np.random.default_rng(n + d)
    g, gt = _whole(torch, rng, n, d, kind, 2, shift=off)
    x, xt = _whole(torch, rng, n, d, kind, 5)
    mean = np.zeros(n) if rms else rng.integers(-3, 4, n).astype(np.float64)
    assert 2 * 8 * n < 2 ** 24
    mt = None if rms else torch.from_numpy(mean.astype(np.float32)).cuda()
    gx, gw, gb = fs.layer_norm_backward(gt, xt, None, mt, torch.ones(n, device="cuda"), need_x=need_x)
    assert (gx is not None) == need_x
    np.testing.assert_array_equal(f64(gw), (g * (x - mean[:, None])).sum(0))
    np.testing.assert_array_equal(f64(gb), g.sum(0))
    assert fs.device_error() == 0


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("n,d,kind", [(20000, 65, "bf16"), (9001, 301, "fp16"), (6000, 33, "fp32"), (5001, 497, "bf16"), (4870, 7, "fp32")])
def test_many_short_rows_off_boundaries(fs, torch_cuda, n, d, kind, rms):
    """Tolerances: those of test_gpu_layer_norm (of the sums: above)."""
    torch = torch_cuda
    c = Case(n, d, kind, "fp32", rms)
    x, g, w, b = c.tensors(torch)
    y, mean, rstd = fs.layer_norm(x, w, b, eps=EPS, rms=rms)
    r, e_mean, e_rstd, e_xh, e_y = c.reference()
    near(rstd, r.rstd, e_rstd * r.rstd, "rstd")
    near(y, r.y, e_y + HALF[kind] * np.abs(r.y) + LEAST[kind], "y")
    check_gradients(c, r, e_rstd, e_xh, fs.layer_norm_backward(g, x, w, mean, rstd), f"{n} x {d}")


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("d", [64, 65, 520, 1001, 2048, 4096, 4097, 9000])
def test_many_rows_in_place(fs, torch_cuda, d, kind):
    """y over x, grad_x over grad, grad_x over x: the bits of separate outputs,
    where blocks ask for rows ahead of those that they write."""
    torch = torch_cuda
    n = 5000 if d < 600 else 2000
    dtype = dtype_of(torch, kind)
    gen = torch.Generator(device="cuda").manual_seed(d)
    x, g = (torch.randn(n, d, generator=gen, device="cuda").to(dtype) for _ in range(2))
    w = torch.rand(d, generator=gen, device="cuda") + 0.5
    y, mean, rstd = fs.layer_norm(x, w)
    own = x.clone()
    y2, mean2, rstd2 = fs.layer_norm(own, w, out=own)
    assert y2 is own and torch.equal(own, y) and torch.equal(mean2, mean) and torch.equal(rstd2, rstd)
    want = fs.layer_norm_backward(g, x, w, mean, rstd)
    own = g.clone()
    got = fs.layer_norm_backward(own, x, w, mean, rstd, out=own)
    assert got[0] is own and all(torch.equal(a, b) for a, b in zip(got, want))
    own = x.clone()
    got = fs.layer_norm_backward(g, own, w, mean, rstd, out=own)
    assert got[0] is own and all(torch.equal(a, b) for a, b in zip(got, want))
    alone = fs.layer_norm_backward(g, x, w, mean, rstd, need_x=False)
    assert alone[0] is None and torch.equal(alone[1], want[1]) and torch.equal(alone[2], want[2])
    assert fs.device_error() == 0


@pytest.mark.parametrize("d,gap", [(64, 0), (65, 0), (1001, 7), (2048, 0), (4096, 8), (4097, 1)])
def test_results_beside_their_inputs(fs, torch_cuda, d, gap):
    """Columns of one matrix: x left, y or grad_x right of it, bits and
    neighbours as of matrices apart that lie alike."""
    torch = torch_cuda
    n = 700
    gen = torch.Generator(device="cuda").manual_seed(d + gap)
    made = lambda: torch.randn(n, 2 * d + gap, generator=gen, device="cuda").bfloat16()  # noqa: E731
    both, g, apart = made(), made()[:, :d], made()
    left, right = both[:, :d], both[:, d + gap:]
    x = both.clone()[:, :d]
    y, mean, rstd = fs.layer_norm(x, out=apart[:, d + gap:])
    want = fs.layer_norm_backward(g, x, None, mean, rstd, out=torch.empty_like(both)[:, d + gap:])
    between = both[:, d:d + gap].clone()
    y2, mean2, rstd2 = fs.layer_norm(left, out=right)
    assert torch.equal(right, y) and torch.equal(left, x) and torch.equal(mean2, mean) and torch.equal(rstd2, rstd)
    got = fs.layer_norm_backward(g, left, None, mean, rstd, out=right)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.equal(left, x) and torch.equal(both[:, d:d + gap], between) and fs.device_error() == 0
