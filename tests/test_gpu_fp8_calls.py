"""Calls of the 8-bit path and of the norm on given streams, from several host
threads, within captured graphs and after failures; and the operators together,
as a layer, a training step and a decode loop use them."""

import numpy as np
import pytest

from _helpers import compare, to_device
from lm_head_exact_gb300 import synthetic
from oracle import fp8, sampler
from test_gpu_fp8 import f64
from test_gpu_training_calls import _in_a_thread, _on_another_stream, _run_threads, _streams_left_as_new  # noqa: F401

pytestmark = pytest.mark.gpu

KINDS = ["quantise", "quantise weight", "product", "thin product", "sample", "norm", "norm fp8", "norm gradient"]


class Calls:
    """One call of each kind on inputs of its own: ``Calls(...)(kind)`` gives
    the tensors it returns."""

    def __init__(self, fs, torch, seed=0, n=200, d=272, V=1504):
        g = torch.Generator(device="cuda").manual_seed(21 + seed)
        rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.fs, self.torch, self.V = fs, torch, V
        self.x, self.grad = rand(n, d).bfloat16(), rand(n, d).bfloat16()
        self.weight, self.bias = rand(d), rand(d)
        self.W = rand(V, d).bfloat16()
        self.x8, self.W8 = fs.quantize_fp8(self.x), fs.quantize_fp8(self.W, block_rows=128)
        self.thin8 = fs.quantize_fp8(self.x[:9])
        self.temp = torch.ones(9, device="cuda")
        self.stats = fs.layer_norm(self.x, self.weight, self.bias)[1:]
        torch.cuda.synchronize()

    def __call__(self, kind, stream=None, out=None):
        fs, s = self.fs, dict(stream=stream)
        if out is not None:
            s["out"] = out
        got = {"quantise": lambda: fs.quantize_fp8(self.x, **s),
               "quantise weight": lambda: fs.quantize_fp8(self.W, block_rows=128, transpose=True, **s),
               "product": lambda: [fs.fp8_matmul(*self.x8, *self.W8, **s)],
               "thin product": lambda: [fs.fp8_matmul(*self.thin8, *self.W8, **s)],
               "sample": lambda: fs.sample_fp8(*self.thin8, *self.W8, self.temp, 5, 6, **s),
               "norm": lambda: fs.layer_norm(self.x, self.weight, self.bias, **s),
               "norm fp8": lambda: fs.layer_norm_fp8(self.x, self.weight, self.bias, rms=True, **s),
               "norm gradient": lambda: fs.layer_norm_backward(self.grad, self.x, self.weight, *self.stats, **s)}[kind]()
        return list(got)


def same(torch, a, b):
    """Equal bits (8-bit types have no comparison of their own)."""
    return all(torch.equal(x.view(torch.uint8) if x.element_size() == 1 else x, y.view(torch.uint8) if y.element_size() == 1
                           else y) for x, y in zip(a, b))


@pytest.mark.parametrize("kind", KINDS)
def test_results_on_a_given_stream(fs, torch_cuda, kind):
    """The results' memory is not still in use on the current stream, and the
    results are the same.  (Tensors of their types and sizes have been dropped.)"""
    torch = torch_cuda
    calls = Calls(fs, torch)
    want = calls(kind)
    as_bytes = lambda ts: [torch.as_strided(t, (t.untyped_storage().nbytes() // t.element_size(),), (1,), 0).view(torch.uint8)  # noqa: E731
                           for t in ts]
    shapes = [((t.numel(),), torch.uint8) for t in as_bytes(want)]
    _on_another_stream(torch, shapes, lambda s: as_bytes(calls(kind, s)), as_bytes(want))
    fs.device_error()


@pytest.mark.parametrize("kind", KINDS)
def test_first_call_of_a_host_thread(fs, torch_cuda, kind):
    torch = torch_cuda
    calls = Calls(fs, torch, seed=1)
    want = calls(kind)
    torch.cuda.synchronize()
    got = _in_a_thread(lambda: calls(kind))
    torch.cuda.synchronize()
    assert same(torch, want, got) and fs.device_error() == 0


@pytest.mark.parametrize("kind", ["sample", "product", "norm gradient"])
def test_threads_that_share_a_stream(fs, torch_cuda, kind):
    """A sampler's keys and a gradient's partial sums are their call's own."""
    torch = torch_cuda
    calls = [Calls(fs, torch, seed=k, n=200 + 300 * k, V=1500 + 700 * k) for k in range(2)]
    alone = [c(kind) for c in calls]
    torch.cuda.synchronize()
    jobs = [(lambda c: lambda: c(kind))(c) for c in calls]
    for want, got in zip(alone, _run_threads(torch, jobs, 200)):
        for r in got:
            assert same(torch, want, r)
    assert fs.device_error() == 0


@pytest.mark.parametrize("kind", KINDS)
def test_two_streams_at_once(fs, torch_cuda, kind):
    torch = torch_cuda
    calls = [Calls(fs, torch, seed=k, n=600, V=4000) for k in range(2)]
    alone = [c(kind) for c in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(30):
        for c, s, r in zip(calls, streams, got):
            with torch.cuda.stream(s):
                r.append(c(kind))
    torch.cuda.synchronize()
    for want, rs in zip(alone, got):
        assert all(same(torch, want, r) for r in rs)
    assert fs.device_error() == 0


@pytest.mark.parametrize("kind", KINDS)
def test_captured_and_replayed(fs, torch_cuda, kind):
    """Two graphs of one stream, replayed in turn with new inputs in place of
    the captured ones."""
    torch = torch_cuda
    calls = [Calls(fs, torch, seed=k) for k in range(2)]
    other = Calls(fs, torch, seed=2)
    stream = torch.cuda.Stream()
    fs.workspace_reserve(64, 1504, stream=stream)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for c in calls:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            outs.append(c(kind))
        graphs.append(graph)
    want = [c(kind) for c in calls]
    last = other(kind)
    with torch.cuda.stream(stream):
        for _ in range(3):
            for graph in graphs:
                graph.replay()
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert same(torch, w, o)
    for name in ("x", "grad", "weight", "bias", "W"):
        getattr(calls[0], name).copy_(getattr(other, name))
    for name in ("x8", "W8", "thin8", "stats"):
        for a, b in zip(getattr(calls[0], name), getattr(other, name)):
            a.copy_(b)
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        graphs[0].replay()
        graphs[1].replay()
    torch.cuda.synchronize()
    assert same(torch, last, outs[0]) and same(torch, want[1], outs[1])
    assert fs.device_error() == 0


@pytest.mark.parametrize("kind", KINDS)
def test_a_launch_that_fails(fs, torch_cuda, kind):
    """An error, and the next call is whole."""
    torch = torch_cuda
    calls = Calls(fs, torch)
    want = calls(kind)
    fs.debug_set_fault(fs.FS_FAULT_LAUNCH)
    try:
        with pytest.raises(fs.FlashSampleError) as e:
            calls(kind)
    finally:
        fs.debug_set_fault(fs.FS_FAULT_NONE)
    assert e.value.status == "FS_ERR_CUDA"
    assert same(torch, want, calls(kind))


def test_a_workspace_that_cannot_grow(fs, torch_cuda):
    torch = torch_cuda
    calls = Calls(fs, torch)
    want = calls("sample")
    torch.cuda.synchronize()
    fs.check(fs.library().fs_workspace_release())
    fs.debug_set_fault(fs.FS_FAULT_ALLOC)
    try:
        with pytest.raises(fs.FlashSampleError) as e:
            calls("sample")
    finally:
        fs.debug_set_fault(fs.FS_FAULT_NONE)
    assert e.value.status == "FS_ERR_WORKSPACE"
    assert same(torch, want, calls("sample"))


def test_refuses_memory_in_two_roles(fs, torch_cuda):
    torch = torch_cuda
    calls = Calls(fs, torch)
    x, (q, s), (W, ws) = calls.x, calls.x8, calls.W8
    memory = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    x2 = memory[:400 * 256].view(torch.bfloat16).view(200, 256)
    with pytest.raises(fs.FlashSampleError, match="overlaps"):
        fs.quantize_fp8(x2, out=(memory[256:256 + 200 * 256].view(torch.float8_e4m3fn).view(200, 256), torch.empty(200, 2, device="cuda")))
    a = memory[:200 * 256].view(torch.float8_e4m3fn).view(200, 256)
    with pytest.raises(fs.FlashSampleError, match="overlaps"):
        fs.fp8_matmul(a, torch.ones(200, 2, device="cuda"), a, torch.ones(200, 2, device="cuda"),
                      out=memory[512:512 + 200 * 400].view(torch.bfloat16).view(200, 200))
    with pytest.raises(fs.FlashSampleError, match="align"):
        fs.fp8_matmul(memory[8:8 + 200 * 256].view(torch.float8_e4m3fn).view(200, 256), torch.ones(200, 2, device="cuda"), a,
                      torch.ones(200, 2, device="cuda"))
    with pytest.raises(fs.FlashSampleError, match="multiple of 16"):
        fs.fp8_matmul(memory[:200 * 264].view(torch.float8_e4m3fn).view(200, 264)[:, :256], torch.ones(200, 2, device="cuda"),
                      a, torch.ones(200, 2, device="cuda"))
    with pytest.raises(fs.FlashSampleError, match="overlap"):
        fs.layer_norm(x2, out=memory[512:512 + 400 * 256].view(torch.bfloat16).view(200, 256))
    with pytest.raises(fs.FlashSampleError, match="out must be"):
        fs.fp8_matmul(q, s, W, ws, out=torch.empty(200, calls.V, device="cuda"), out_dtype=torch.bfloat16)
    with pytest.raises(fs.FlashSampleError):
        fs.fp8_matmul(q, s, W, ws, out=torch.empty(200, calls.V - 1, device="cuda"))
    with pytest.raises(fs.FlashSampleError):
        fs.fp8_matmul(q.cpu(), s, W, ws)
    assert x.shape == (200, 272)


# ---------------------------------------------------------------- together
def _bounds(x, q, fmt_half=2.0 ** -4):
    """How far a quantised matrix may lie from x, per element: half a step of
    e4m3, and below its least normal 2^-6 half of 2^-9, times the scale; the
    product with 1/scale is rounded twice (2 x 2^-24, counted as 2^-20)."""
    rows, cols = x.shape
    scale = f64(q[1])
    s = np.repeat(scale, 128, 1)[:, :cols]
    if scale.shape[0] != rows:
        s = np.repeat(s, 128, 0)[:rows]
    return np.abs(x) * (fmt_half + 2.0 ** -20) + s * 2.0 ** -10


@pytest.mark.parametrize("n,d,ffn", [(1, 256, 512), (16, 264, 300), (300, 512, 1000)])
def test_a_layer_in_8_bits(fs, torch_cuda, n, d, ffn):
    """Norm, up, activation, down, residual, norm, head: the activations stay
    within the bound that the quantisers' half steps give against 64 bits, and
    the samples are those of the head's own inputs."""
    torch = torch_cuda
    g = torch.Generator(device="cuda").manual_seed(31)
    x = torch.randn(n, d, generator=g, device="cuda").bfloat16()
    up, down, W = ((torch.randn(*s, generator=g, device="cuda") * s[1] ** -0.5).bfloat16() for s in ((ffn, d), (d, ffn), (2000, d)))
    weight = torch.rand(d, generator=g, device="cuda") + 0.5
    up8, down8, W8 = (fs.quantize_fp8(m, block_rows=128) for m in (up, down, W))
    x8 = fs.layer_norm_fp8(x, weight, eps=1e-6, rms=True)
    a = fs.fp8_matmul(*x8, *up8)
    a8 = fs.quantize_fp8(a)
    y = x + fs.fp8_matmul(*a8, *down8)
    h8 = fs.layer_norm_fp8(y, weight, eps=1e-6, rms=True)
    temp = torch.full((n,), 0.8, device="cuda")
    ids, mx = fs.sample_fp8(*h8, *W8, temp, 3, 4)

    normed = lambda v: f64(v) / np.sqrt((f64(v) ** 2).mean(1, keepdims=True) + 1e-6) * f64(weight)  # noqa: E731
    half, U = 2.0 ** -8, 2.0 ** -24

    def near(got, left, left8, right, right8, plus=0.0):
        """got against left right^T (+ plus): quantised factors, 128 + blocks
        roundings of the sum, one to bf16 (two with the addition)."""
        el, er = _bounds(left, left8), _bounds(f64(right), right8)
        L, R = np.abs(left), np.abs(f64(right))
        # (the norm's own rounding to fp32: 2^-18 covers its sums)
        tol = (L * (1 + 2.0 ** -18) + el) @ (R + er).T - L @ R.T + ((2 * 128 + 2 + left.shape[1] / 128 + 1) * U) * (L @ R.T) * 1.2
        out = left @ f64(right).T
        tol = (tol + np.abs(out) * half) * (1 + half) + np.abs(plus + out) * half
        assert np.all(np.abs(f64(got) - (plus + out)) <= tol)
        assert np.linalg.norm(f64(got) - (plus + out)) < 0.2 * np.linalg.norm(out)

    near(a, normed(x), x8, up, up8)
    near(y, f64(a), a8, down, down8, f64(x))
    deq = lambda q8: fp8.Quantised(None, f64(q8[1]), f64(q8[0]) * np.repeat(np.repeat(  # noqa: E731
        f64(q8[1]), 128, 1)[:, :q8[0].shape[1]], 1 if q8[1].shape[0] == q8[0].shape[0] else 128, 0)[:q8[0].shape[0]])
    logits = deq(h8).value @ deq(W8).value.T
    compare(ids.cpu().numpy(), mx.cpu().numpy(), sampler.sample_from_logits(logits, np.full(n, 0.8, np.float32), 3, 4,
                                                                           np.arange(n), np.arange(2000)), what="layer")
    assert fs.device_error() == 0


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("w_dtype", ["bfloat16", "float32"])
def test_policy_step_through_the_final_norm(fs, torch_cuda, rms, w_dtype):
    """Loss and gradients ahead of the norm, and the norm's own, against
    autograd in 64 bits with the normed states' rounding to bf16 taken over."""
    torch = torch_cuda
    from lm_head_exact_gb300 import policy_step as ps
    g = torch.Generator(device="cuda").manual_seed(33)
    n, d, V, S = 120, 128, 1500, 8
    h = (torch.randn(n, d, generator=g, device="cuda") * 3 + 0.5).bfloat16()
    W = (torch.randn(V, d, generator=g, device="cuda") * 0.1).bfloat16()
    w_type = getattr(torch, w_dtype)
    norm = ps.FinalNorm((torch.rand(d, generator=g, device="cuda") + 0.5).to(w_type),
                        None if rms else torch.randn(d, generator=g, device="cuda").to(w_type), rms=rms)
    starts = torch.arange(0, n + 1, n // S, device="cuda")
    r = ps.roll_out(h, W, torch.full((n,), 0.9, device="cuda"), starts, lambda ids: (ids.view(S, -1) % 7).float().mean(1),
                    1234, 3, norm=norm)
    moved = ps.FinalNorm((norm.weight.float() * 1.03).to(w_type), norm.bias, norm.eps, rms)
    out = ps.policy_step(r, W, ref_logp=r.old_logp, kl_coef=0.1, norm=moved)

    h64, w64 = h.double().requires_grad_(), moved.weight.double().requires_grad_()
    b64 = None if rms else moved.bias.double().requires_grad_()
    mu = 0.0 if rms else h64.mean(1, keepdim=True)
    xh = (h64 - mu) / (((h64 - mu) ** 2).mean(1, keepdim=True) + norm.eps).sqrt()
    y = xh * w64 if rms else xh * w64 + b64
    y_used = fs.layer_norm(h, moved.weight, moved.bias, rms=rms)[0].double()
    y = y + (y_used - y).detach()                             # the values that the kernels saw
    y.retain_grad()
    logp = torch.log_softmax(y @ W.double().T / 0.9, 1).gather(1, r.ids[:, None])[:, 0]
    ratio = (logp - r.old_logp.double()).exp()
    A = r.advantages.double().repeat_interleave(n // S)
    q = r.old_logp.double() - logp
    loss = (-torch.minimum(ratio * A, ratio.clamp(0.8, 1.28) * A) + 0.1 * (q.exp() - 1 - q)).mean()
    loss.backward()
    assert abs(float(out.stats[0]) - float(loss.detach())) < 1e-4
    # grad_y: ds and the result each rounded to bf16 (2^-8), 2^-12 for the scores' error in ds; grad_h is one more
    # rounding of a projection of rstd w grad_y, whose errors are measured by what is projected
    e = 2 * 2.0 ** -8 + 2.0 ** -12
    rstd = 1 / (((h64 - mu) ** 2).mean(1, keepdim=True) + norm.eps).sqrt()
    size = float((rstd * w64 * y.grad).detach().norm())
    assert float((out.grad_h.double() - h64.grad).norm()) < e * size + 2.0 ** -8 * float(h64.grad.norm())
    own = 2.0 ** -8 if w_dtype == "bfloat16" else 2.0 ** -20
    terms = (y.grad * xh).abs().sum(0).detach()
    assert float((out.grad_norm_weight.double() - w64.grad).norm()) < e * float(terms.norm()) + own * float(w64.grad.norm())
    if rms:
        assert out.grad_norm_bias is None
    else:
        assert float((out.grad_norm_bias.double() - b64.grad).norm()) < e * float(y.grad.abs().sum(0).norm()) + own * float(b64.grad.norm())
    assert out.grad_norm_weight.dtype == w_type
    assert fs.device_error() == 0


SMALL = dict(d=256, q=256, kv=64, ffn=512)


@pytest.mark.parametrize("B", [1, 8, 70])
def test_decode_loop_in_8_bits(fs, torch_cuda, B):
    """Ids in range, the same on every run; the last step's are those of the
    body's own result."""
    torch = torch_cuda
    from lm_head_exact_gb300 import decode_loop
    W = to_device(synthetic.normal_blocks_bf16(1, 4096, 256, 0.02), torch)
    loop = decode_loop.DecodeLoop(W, layers=2, layer=SMALL, fp8=True)
    ids0 = torch.arange(B, device="cuda", dtype=torch.int64) * 57
    temp = torch.ones(B, device="cuda")
    _, a = loop.run(ids0, temp, steps=3, warmup=3)
    t, b = loop.run(ids0, temp, steps=3, warmup=3)
    assert torch.equal(a, b) and bool(((a >= 0) & (a < 4096)).all()) and t.step_us > 0
    ids = ids0
    for step in range(9):
        ids, _ = fs.sample_fp8(*loop.body(W[ids]), *loop.W8, temp, 1234, step)
    assert torch.equal(a, ids)
    with pytest.raises(ValueError, match="no 8-bit form"):
        loop.run(ids0, temp, steps=1, fused=False, warmup=0)
    assert fs.device_error() == 0


def test_decode_loop_compared(fs, torch_cuda):
    torch = torch_cuda
    from lm_head_exact_gb300 import decode_loop
    W = to_device(synthetic.normal_blocks_bf16(1, 4096, 256, 0.02), torch)
    for r in decode_loop.measure_fp8(W, batches=(1, 16), layers=2, steps=4, warmup=3, layer=SMALL):
        assert r["fp8_step_us"] > 0 and r["bf16_head_us"] > 0 and np.isfinite(r["step_time_reduction"])
