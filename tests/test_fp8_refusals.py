"""What the 8-bit path and the norm refuse, on the host before any kernel
runs, and what passes between them in a policy step, on the CPU."""

import ctypes

import pytest

Z = ctypes.c_void_p(0)


def _last(lib):
    return lib.fs_last_error().decode()


@pytest.fixture(scope="module")
def lib(built_library):
    from lm_head_exact_gb300 import binding
    return binding.library()


def test_quantise_refuses(lib):
    def call(kind=1, rows=4, cols=8, stride=8, transpose=0, block=1, q_kind=3, q_stride=16, s_row=1, s_col=4):
        return lib.fs_quantize_fp8(Z, kind, rows, cols, stride, transpose, block, q_kind, Z, q_stride, Z, s_row, s_col, Z)

    assert call(rows=-1) == 1 and call(cols=-1) == 1
    assert call(rows=1 << 31) == 2 and call(cols=1 << 31) == 2
    for kind in (-1, 3, 4, 5):
        assert call(kind=kind) == 1 and "type" in _last(lib)
    assert call(q_kind=1) == 1 and "8-bit" in _last(lib) and call(q_kind=5) == 1
    assert call(transpose=2) == 1
    for block in (0, 2, 64, 256):
        assert call(block=block) == 1 and "1 or 128" in _last(lib)
    assert call(stride=7) == 1 and "row stride" in _last(lib) and call(stride=-8) == 1
    assert call(q_stride=24) == 2 and "multiple of 16" in _last(lib)
    assert call(q_stride=0) == 1
    assert call(s_row=-1) == 1 and "scales" in _last(lib)
    assert call() == 1 and "q is NULL" in _last(lib)
    assert call(rows=0) == 0 and call(cols=0, q_stride=0, stride=0) == 0


def test_product_refuses(lib):
    def call(a_kind=3, b_kind=3, m=4, n=5, k=40, a_stride=48, b_stride=48, block=128, out_kind=1, out_stride=5):
        return lib.fs_fp8_matmul(Z, a_kind, a_stride, Z, 1, 4, Z, b_kind, b_stride, Z, 1, 1, block, m, n, k, Z, out_kind,
                                 out_stride, Z)

    assert call(m=-1) == 1 and call(n=-1) == 1 and call(k=-1) == 1
    assert call(m=1 << 31) == 2 and call(n=1 << 31) == 2 and call(k=(1 << 24) + 1) == 2
    assert call(a_kind=1) == 1 and call(m=0, b_kind=0) == 1 and call(out_kind=3) == 1
    assert call(a_stride=40) == 2 and call(m=0, b_stride=50) == 2 and call(a_stride=32) == 1
    assert call(m=0, block=7) == 1 and "1 or 128" in _last(lib)
    assert call(out_stride=4) == 1
    assert call() == 1 and "a is NULL" in _last(lib)
    assert call(m=0) == 1 and "b is NULL" in _last(lib)                      # (what there is is checked)
    assert call(m=0, n=0) == 0


def test_sampler_refuses(lib):
    def call(B=4, d=40, V=100, h_stride=48, W_stride=48, block=128):
        return lib.fs_sample_fp8(Z, h_stride, Z, 1, 4, Z, W_stride, Z, 1, 1, block, B, d, V, Z, Z, 0, 0, 0, Z, Z, Z)

    assert call(B=-1) == 1 and "B >= 0" in _last(lib)
    assert call(d=0) == 1 and call(V=-1) == 1
    assert call(V=1 << 31) == 2 and call(B=1 << 31) == 2 and call(d=(1 << 24) + 1) == 2
    assert call(h_stride=40) == 2
    assert call() == 1 and "h is NULL" in _last(lib)
    assert call(B=0) == 0


def test_norm_refuses(lib):
    def call(kind=1, n=4, d=8, stride=8, w_kind=0, rms=0, eps=1e-5, y=Z, q=Z):
        return lib.fs_layer_norm(Z, kind, n, d, stride, Z, Z, w_kind, rms, eps, y, 8, Z, Z, q, 3, 16, Z, 1, 4, Z)

    def back(kind=1, n=4, d=8, g_stride=8, stride=8, w_kind=0, rms=0):
        return lib.fs_layer_norm_backward(Z, g_stride, Z, kind, n, d, stride, Z, w_kind, rms, Z, Z, Z, 8, Z, Z, Z, 0, Z)

    for f in (call, back):
        assert f(n=-1) == 1 and f(d=0) == 1 and "d > 0" in _last(lib)
        assert f(d=32769, stride=32769) == 2 and f(n=1 << 31) == 2
        assert f(kind=3) == 1 and f(w_kind=2) == 1 and "weights are fp32 or" in _last(lib)
        assert f(rms=2) == 1 and f(stride=7) == 1
    for eps in (-1.0, float("nan"), float("inf")):
        assert call(eps=eps) == 1 and "eps" in _last(lib)
    assert call() == 1 and "one of y and q" in _last(lib)
    assert call(y=ctypes.c_void_p(4096), q=ctypes.c_void_p(8192)) == 1 and "one of y and q" in _last(lib)
    assert call(n=0) == 0
    assert back(g_stride=7) == 1
    assert back() == 1 and "g is NULL" in _last(lib)
    assert back(n=0) == 0
    size = lib.fs_layer_norm_backward_workspace_bytes
    assert size(0, 8) == 0 and size(4, 0) == 0 and size(4, 8) >= 4 * 2 * 8 * 4
    assert size(1 << 30, 32768) < 100 << 20                                    # does not grow with the rows


def test_binding_refuses(built_library):
    torch = pytest.importorskip("torch")
    from lm_head_exact_gb300 import binding as fs
    x, q, s = torch.zeros(4, 40), torch.zeros(4, 40).to(torch.float8_e4m3fn), torch.zeros(4, 1)
    t = torch.ones(4)
    for call in (lambda: fs.quantize_fp8(x), lambda: fs.fp8_matmul(q, s, q, s), lambda: fs.sample_fp8(q, s, q, s, t, 0, 0),
                 lambda: fs.layer_norm(x), lambda: fs.layer_norm_fp8(x), lambda: fs.layer_norm_backward(x, x, None, t, t)):
        with pytest.raises(fs.FlashSampleError, match="CUDA tensor"):
            call()


def test_binding_checks_shapes_and_types(built_library):
    torch = pytest.importorskip("torch")
    from lm_head_exact_gb300 import binding as fs

    class OnDevice(torch.Tensor):                     # says it is on the device, for the binding's checks
        is_cuda = True

    def D(t):
        return torch.Tensor._make_subclass(OnDevice, t)

    x, e4 = torch.zeros(4, 300), torch.float8_e4m3fn
    q, s = D(x.to(e4)), D(torch.zeros(4, 3))
    W, ws = D(torch.zeros(200, 300).to(e4)), D(torch.zeros(2, 3))
    with pytest.raises(fs.FlashSampleError, match="block_rows must be"):
        fs.quantize_fp8(D(x), block_rows=64)
    with pytest.raises(fs.FlashSampleError, match="float8_e4m3fn or"):
        fs.quantize_fp8(D(x), dtype=torch.float32)
    for a, asc, b, bsc, what in ((q, s, D(torch.zeros(200, 299).to(e4)), ws, r"\[m, k\]"),
                                 (q, D(torch.zeros(1, 3)), W, ws, "a row for each"),
                                 (q, s, W, D(torch.zeros(200, 2)), "b_scale must be"),
                                 (q, s, W, D(torch.zeros(2, 3, dtype=torch.float64)), "float32"),
                                 (D(x), s, W, ws, "must not be"), (D(x[0].to(e4)), s, W, ws, "matrix"),
                                 (D(x.to(e4).t().contiguous().t()), s, W, ws, "contiguous rows")):
        with pytest.raises(fs.FlashSampleError, match=what):
            fs.fp8_matmul(a, asc, b, bsc)
    e5 = D(x.to(torch.float8_e5m2))
    with pytest.raises(fs.FlashSampleError, match="must not be"):
        fs.sample_fp8(e5, s, W, ws, D(torch.ones(4)), 0, 0)
    h = D(x.bfloat16())
    with pytest.raises(fs.FlashSampleError, match="weight must be"):
        fs.layer_norm(h, D(torch.ones(300, dtype=torch.float16)))
    with pytest.raises(fs.FlashSampleError, match="one type"):
        fs.layer_norm(h, D(torch.ones(300)), D(torch.ones(300).bfloat16()))
    with pytest.raises(fs.FlashSampleError, match="shape"):
        fs.layer_norm(h, D(torch.ones(299)))
    with pytest.raises(fs.FlashSampleError, match="weight_dtype"):
        fs.layer_norm_backward(h, h, None, None, D(torch.ones(4)), weight_dtype=torch.float16)


def test_a_policy_step_through_the_final_norm(monkeypatch):
    """The head sees normed states; what comes back is the gradient ahead of the
    norm, and the norm's own."""
    torch = pytest.importorskip("torch")
    from lm_head_exact_gb300 import policy_step as ps
    from test_policy_step import Plain

    class WithNorm(Plain):
        def layer_norm(self, x, weight, bias, eps, rms):
            self.calls.append(("layer_norm", rms))
            y = torch.nn.functional.layer_norm(x, x.shape[1:], weight, bias, eps)
            return y, x.mean(1), (x.var(1, unbiased=False) + eps).rsqrt()

        def layer_norm_backward(self, grad, x, weight, mean, rstd, need_bias=True, out=None):
            assert out is grad
            xh, a = (x - mean[:, None]) * rstd[:, None], grad * weight
            gw, gb = (grad * xh).sum(0), grad.sum(0) if need_bias else None
            out.copy_(rstd[:, None] * (a - a.mean(1, keepdim=True) - xh * (a * xh).mean(1, keepdim=True)))
            return out, gw, gb

    g = torch.Generator().manual_seed(0)
    h, W = torch.randn(12, 16, generator=g) * 3 + 1, torch.randn(30, 16, generator=g)
    plain = WithNorm(torch.randint(0, 30, (12,), generator=g))
    monkeypatch.setattr(ps, "fs", plain)
    starts, temp = torch.tensor([0, 4, 12]), torch.full((12,), 0.8)
    norm = ps.FinalNorm(torch.randn(16, generator=g), torch.randn(16, generator=g))
    r = ps.roll_out(h, W, temp, starts, lambda ids: torch.tensor([1.0, 2.0]), 1, 2, norm=norm)
    assert r.h is h and plain.calls[0] == ("layer_norm", False)
    moved = (W * 1.1)
    out = ps.policy_step(r, moved, norm=norm)
    hh, w, b = h.clone().requires_grad_(), norm.weight.clone().requires_grad_(), norm.bias.clone().requires_grad_()
    y = torch.nn.functional.layer_norm(hh, (16,), w, b, norm.eps)
    logp = torch.log_softmax(y @ moved.T / 0.8, 1).gather(1, r.ids[:, None])[:, 0]
    A = r.advantages.repeat_interleave(starts.diff())
    (-(A * (logp - r.old_logp).exp()).mean()).backward()
    for got, want in ((out.grad_h, hh.grad), (out.grad_norm_weight, w.grad), (out.grad_norm_bias, b.grad)):
        torch.testing.assert_close(got, want, rtol=1e-4, atol=1e-6)
    clipped = ps.policy_step(r, moved, norm=norm, max_norm=1e-3)
    assert len(plain.calls[-1][1]) == 4
    total = torch.cat([t.flatten() for t in (clipped.grad_h, clipped.grad_W, clipped.grad_norm_weight, clipped.grad_norm_bias)])
    assert abs(float(total.norm()) - 1e-3) < 1e-5
