"""The 8-bit path's oracle against independent implementations: PyTorch's own
conversions to 8 bits, its fp64 layer norm and autograd, and finite differences."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import fp8  # noqa: E402

TYPES = {fp8.E4M3: torch.float8_e4m3fn, fp8.E5M2: torch.float8_e5m2}


@pytest.mark.parametrize("fmt", [fp8.E4M3, fp8.E5M2])
def test_rounding_is_that_of_the_type(fmt):
    every = torch.arange(256, dtype=torch.uint8).view(TYPES[fmt]).double()
    every = every[torch.isfinite(every)]
    np.testing.assert_array_equal(fp8.round_fp8(every.numpy(), fmt), every.numpy())
    edges = torch.sort(every.unique()).values
    mid = (edges[1:] + edges[:-1]) / 2                       # ties
    rng = np.random.default_rng(0)
    v = torch.cat((mid, mid * (1 + 2e-7), mid * (1 - 2e-7),
                   torch.from_numpy(rng.standard_normal(20000) * np.exp2(rng.uniform(-20, 8, 20000))))).float()
    v = v[v.abs() <= fp8.LARGEST[fmt]]
    np.testing.assert_array_equal(fp8.round_fp8(v.double().numpy(), fmt), v.to(TYPES[fmt]).double().numpy())


@pytest.mark.parametrize("fmt", [fp8.E4M3, fp8.E5M2])
@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("shape", [(1, 1), (3, 127), (130, 129), (257, 300)])
def test_quantised_in_elementary_steps(fmt, block, shape):
    """The same formula, block by block, in PyTorch's fp32."""
    rng = np.random.default_rng(shape[1])
    x = (rng.standard_normal(shape) * np.exp2(rng.integers(-30, 30, (shape[0], 1)))).astype(np.float32)
    x[0, 0] = 0.0
    got = fp8.quantise(x, block, fmt)
    t = torch.from_numpy(x)
    for i in range(0, shape[0], block):
        for j in range(0, shape[1], 128):
            b = t[i:i + block, j:j + 128]
            scale = torch.clamp(b.abs().max() / torch.tensor(fp8.LARGEST[fmt]), min=2.0 ** -100)
            assert float(scale) == got.scale[i // block, j // 128]
            want = (b * (1.0 / scale)).to(TYPES[fmt]).double().numpy()
            np.testing.assert_array_equal(got.q[i:i + block, j:j + 128], want)
            # within half a step of the value: 2^-4 or 2^-3 of it, or half the least step
            half = 2.0 ** (-4 if fmt == fp8.E4M3 else -3)
            least = 2.0 ** (-10 if fmt == fp8.E4M3 else -17) * float(scale)
            err = np.abs(got.value[i:i + block, j:j + 128] - b.double().numpy())
            assert np.all(err <= np.maximum(half * np.abs(b.double().numpy()), least) * (1 + 2.0 ** -20))


def test_quantised_ends():
    x = np.zeros((4, 130), np.float32)
    x[1, 5], x[2, 5], x[3, :2] = np.nan, np.inf, (1e-38, -3e38)
    x[1, 6] = 2.0
    got = fp8.quantise(x)
    assert np.all(got.scale[0] == 2.0 ** -100) and np.all(got.q[0] == 0)
    assert np.isnan(got.q[1, 5]) and got.q[1, 6] == 448 and got.scale[1, 0] == np.float64(np.float32(2 / 448))
    assert got.scale[2, 0] == np.inf and np.all(np.isnan(got.value[2, :128])) and np.all(got.value[2, 128:] == 0)
    assert got.q[3, 0] == 0 and got.q[3, 1] == -448


@pytest.mark.parametrize("rms", [False, True])
def test_layer_norm_against_autograd(rms):
    rng = np.random.default_rng(3)
    n, d = 5, 37
    x, w, b, g = (torch.from_numpy(rng.standard_normal(s)) for s in ((n, d), (d,), (d,), (n, d)))
    x = (x * 3 + 1).requires_grad_()
    w.requires_grad_()
    b.requires_grad_()
    if rms:
        y = torch.nn.functional.rms_norm(x, (d,), w, 1e-5) + b
    else:
        y = torch.nn.functional.layer_norm(x, (d,), w, b, 1e-5)
    y.backward(g)
    got = fp8.layer_norm(x.detach(), w.detach(), b.detach(), 1e-5, rms)
    np.testing.assert_allclose(got.y, y.detach().numpy(), rtol=1e-12, atol=1e-12)
    for have, want in zip(fp8.layer_norm_gradients(g, got, w.detach(), rms), (x, w, b)):
        np.testing.assert_allclose(have, want.grad.numpy(), rtol=1e-11, atol=1e-12)


@pytest.mark.parametrize("rms", [False, True])
def test_layer_norm_gradient_against_differences(rms):
    rng = np.random.default_rng(4)
    x, w, g = rng.standard_normal((2, 9)), rng.standard_normal(9), rng.standard_normal((2, 9))
    loss = lambda v: float((fp8.layer_norm(v, w, None, 1e-5, rms).y * g).sum())  # noqa: E731
    gx = fp8.layer_norm_gradients(g, fp8.layer_norm(x, w, None, 1e-5, rms), w, rms)[0]
    for i in range(2):
        for j in range(9):
            step = np.zeros_like(x)
            step[i, j] = 1e-5
            assert abs((loss(x + step) - loss(x - step)) / 2e-5 - gx[i, j]) < 1e-8 * (1 + abs(gx[i, j])) * 100


def test_product_is_the_definition():
    rng = np.random.default_rng(5)
    a, b = fp8.quantise(rng.standard_normal((3, 260))), fp8.quantise(rng.standard_normal((130, 260)), 128, fp8.E5M2)
    out, size = fp8.product(a, b)
    want = sum(a.scale[2, k // 128] * a.q[2, k] * b.q[129, k] * b.scale[1, k // 128] for k in range(260))
    assert abs(out[2, 129] - want) < 1e-12 * size[2, 129]
