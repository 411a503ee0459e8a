"""Products of 8-bit matrices whose every partial sum fp32 holds, and greedy
samples over such logits.

Elements are -1, 0 or 1 and scales 1/2 or 1, so products are multiples of 1/4 of
magnitudes up to 1.  Up to 2^22 of them sum to less than 2^24 quarters: each
partial sum, in any order, is a number of fp32, and results are equal to those in
64 bits.  A lost, doubled or wrongly scaled block shows whatever the depth."""

import numpy as np
import pytest

from test_gpu_fp8 import f64

pytestmark = pytest.mark.gpu


def _operand(torch, rng, rows, k, block, e5m2=False):
    """(values in 64 bits, q, scale); NaNs lie behind q's rows."""
    q = rng.integers(-1, 2, (rows, k)).astype(np.int8)
    blocks = -(-k // 128)
    scale = np.exp2(-rng.integers(0, 2, (-(-rows // block), blocks))).astype(np.float32)
    memory = torch.full((rows, (k + 15) // 16 * 16 + 16), 0x7f, dtype=torch.uint8, device="cuda")
    qt = memory.view(torch.float8_e5m2 if e5m2 else torch.float8_e4m3fn)[:, :k]
    qt.copy_(torch.from_numpy(q).float().to(qt.dtype).cuda())
    value = q.astype(np.float32) * np.repeat(np.repeat(scale, block, 0)[:rows], 128, 1)[:, :k]
    return value.astype(np.float64), qt, torch.from_numpy(scale).cuda()


SUMS = [(1, 700, 5000), (7, 10, 300000), (8, 33, 1000003), (64, 7, 1000003), (33, 130, 80000), (64, 1000, 16400), (20, 300, 200001),
        (65, 200, 100000), (129, 257, 30001), (257, 192, 40000), (300, 1001, 1000), (1, 33000, 4200), (9, 8200, 4100), (16, 6145, 4112),
        (40, 4100, 4200), (1500, 2049, 300)]


@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("m,n,k", SUMS)
def test_sums_are_exact(fs, torch_cuda, m, n, k, block):
    torch = torch_cuda
    assert k <= 2 ** 22
    rng = np.random.default_rng(m + n + k)
    a, aq, asc = _operand(torch, rng, m, k, 1)
    b, bq, bsc = _operand(torch, rng, n, k, block, e5m2=k % 2 == 1)
    got = fs.fp8_matmul(aq, asc, bq, bsc, out_dtype=torch.float32)
    np.testing.assert_array_equal(f64(got), a @ b.T)
    assert fs.device_error() == 0


@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("B,d,V", [(1, 512, 3001), (16, 1000, 3001), (40, 513, 5000), (64, 4096, 20000), (100, 384, 777), (140, 300, 5000),
                                   (300, 2048, 2500)])
def test_greedy_samples_are_the_largest_product(fs, torch_cuda, B, d, V, block):
    """Bit for bit, and of equal ones the smallest id: whole quarters tie often."""
    torch = torch_cuda
    rng = np.random.default_rng(B + d + V)
    h, hq, hs = _operand(torch, rng, B, d, 1)
    W, Wq, Ws = _operand(torch, rng, V, d, block)
    logits = h @ W.T
    ids, mx = fs.sample_fp8(hq, hs, Wq, Ws, torch.zeros(B, device="cuda"), 0, 0)
    np.testing.assert_array_equal(f64(mx), logits.max(1))
    np.testing.assert_array_equal(ids.cpu().numpy(), logits.argmax(1))
    got = fs.fp8_matmul(hq, hs, Wq, Ws, out_dtype=torch.float32)
    np.testing.assert_array_equal(f64(got), logits)
    assert fs.device_error() == 0


@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("dtype", ["float8_e4m3fn", "float8_e5m2"])
@pytest.mark.parametrize("cols", [1, 17, 128, 1000])
def test_what_a_single_row_is_quantised_into(fs, torch_cuda, cols, dtype, transpose, block):
    torch = torch_cuda
    x = torch.randn(cols, 1, device="cuda") if transpose else torch.randn(1, cols, device="cuda")
    q, scale = fs.quantize_fp8(x, block_rows=block, dtype=getattr(torch, dtype), transpose=transpose)
    assert q.shape == (1, cols) and q.dtype == getattr(torch, dtype) and q.is_contiguous()
    assert scale.shape == (1, -(-cols // 128)) and scale.dtype == torch.float32
