"""The training operators on the GPU against their fp64 forms.

Tolerances (u = 2^-24 the half step of fp32, 2^-8 that of bf16):

* a logit is a sum of d exact products held in fp32, rounded or cut once for
  each: |x err| <= (d + 2) 2u inv_t sum |h W| + 2u |x| (bias, scaling);
* lse moves by at most the largest x error; its sum of V exponentials, each
  within 2^-21, adds (V / 8 + 32) u (terms are added within groups before the
  groups are joined) and the logarithm 4u |lse|;
* ds = c (1[own] - p): p carries the relative error of exp(x - lse), and the
  result is rounded to bf16: 2^-8 |ds|;
* grad_h and grad_W sum products of ds over V or n terms held in fp32 and are
  rounded once to bf16: the errors of ds times the other factor, 2u per term,
  2^-8 of the result.
"""

import math

import numpy as np
import pytest

from _helpers import to_device
from lm_head_exact_gb300 import synthetic
from oracle import training as tr

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF_BF16, HALF_FP16 = 2.0 ** -8, 2.0 ** -11


def _bf16(x):
    bits = synthetic.bf16_bits(np.asarray(x, np.float32))
    return bits, synthetic.bf16_bits_to_f32(bits)


class Head:
    def __init__(self, n, d, V, bias="none", seed=0, scale=1.5):
        rng = np.random.default_rng(seed + 1000 * n + 7 * V + d)
        self.hb, self.h = _bf16(rng.standard_normal((n, d)))
        self.Wb, self.W = _bf16(rng.standard_normal((V, d)) * scale / math.sqrt(d))
        self.ids = rng.integers(0, V, n)
        self.ids[rng.random(n) < 0.1] = -1
        self.temp = rng.uniform(0.5, 1.5, n).astype(np.float32)
        self.g = (rng.standard_normal(n) / n).astype(np.float32)
        self.g[rng.random(n) < 0.1] = 0.0
        self.bias = None
        if bias == "shared":
            self.bias = np.where(rng.random(V) < 0.2, -np.inf, rng.standard_normal(V)).astype(np.float32)
        elif bias == "rows":
            self.bias = rng.standard_normal((n, V)).astype(np.float32)

    def device(self, torch, pad=0):
        bias = self.bias
        if bias is not None and bias.ndim == 2 and pad:
            wide = np.zeros((bias.shape[0], bias.shape[1] + pad), np.float32)
            wide[:, :bias.shape[1]] = bias
            bias = to_device(wide, torch)[:, :bias.shape[1]]
        elif bias is not None:
            bias = to_device(bias, torch)
        return (to_device(self.hb, torch), to_device(self.Wb, torch), torch.from_numpy(self.ids).cuda(),
                to_device(self.temp, torch), bias, to_device(self.g, torch))

    def reference(self):
        s = tr.scores(self.h, self.W, self.ids, self.temp, self.bias)
        return s, tr.score_gradients(self.h, self.W, self.ids, s, self.g)

    def tolerances(self, s, grads):
        ds, live, gh, gW = grads
        d, V, n = self.h.shape[1], self.W.shape[0], len(self.ids)
        h = np.where(live[:, None], self.h, 0.0).astype(np.float64)
        size = np.abs(self.h.astype(np.float64)) @ np.abs(self.W.astype(np.float64)).T
        if self.bias is not None:
            size = size + np.where(np.isfinite(self.bias), np.abs(self.bias), 0.0)
        tx = (d + 4) * 2 * U * size * s.inv_t[:, None]
        tx_max = tx.max(1)
        lse = np.where(np.isfinite(s.lse), np.abs(s.lse), 0.0)
        t_lse = tx_max + (V / 8 + 32) * U + 4 * U * lse
        t_logp = 2 * tx_max + t_lse + 4 * U * lse
        p = np.where(live[:, None], np.exp(s.x - s.lse[:, None]), 0.0)
        c = np.abs(self.g.astype(np.float64) * s.inv_t)[:, None] * live[:, None]
        t_ds = c * p * (tx + t_lse[:, None] + 2.0 ** -20 + 8 * U * lse[:, None]) + np.abs(ds) * (HALF_BF16 + 4 * U) + 1e-38
        t_ds = np.where(live[:, None], t_ds, 0.0)
        aW, ah = np.abs(self.W.astype(np.float64)), np.abs(h)
        t_gh = t_ds @ aW + (V + 32) * 2 * U * (np.abs(ds) @ aW) + HALF_BF16 * np.abs(gh)
        t_gW = t_ds.T @ ah + (n + 32) * 2 * U * (np.abs(ds).T @ ah) + HALF_BF16 * np.abs(gW)
        return t_logp, t_lse, t_gh * 1.01 + 1e-37, t_gW * 1.01 + 1e-37


def _near(got, want, tol, what):
    got = np.asarray(got, np.float64)
    np.testing.assert_array_equal(np.isnan(got), np.isnan(want), err_msg=what)
    np.testing.assert_array_equal(got == -np.inf, want == -np.inf, err_msg=what)
    fin = np.isfinite(want)
    with np.errstate(all="ignore"):
        over = np.where(fin, np.abs(got - want) / tol, 0.0)
    assert np.all(over <= 1), f"{what}: {over.max():.3g} times the tolerance at {np.unravel_index(over.argmax(), over.shape)}"


def _f(t):
    return t.detach().float().cpu().numpy()


SHAPES = [(1, 8, 1), (1, 64, 1000), (2, 40, 63), (31, 72, 257), (64, 128, 64), (65, 136, 65), (128, 64, 513),
          (129, 200, 1001), (255, 64, 130), (257, 520, 700), (300, 256, 4097), (16, 1024, 3000)]


@pytest.mark.parametrize("kept", [True, False])
@pytest.mark.parametrize("bias", ["none", "shared", "rows"])
@pytest.mark.parametrize("n,d,V", SHAPES)
def test_scores_and_gradients(fs, torch_cuda, n, d, V, bias, kept):
    torch = torch_cuda
    hp = Head(n, d, V, bias)
    h, W, ids, temp, b, g = hp.device(torch, pad=3)
    keep = fs.logprob_buffer(n, V) if kept else None
    logp, lse = fs.token_logprobs(h, W, ids, temp, bias=b, kept=keep)
    gh, gW = fs.token_logprobs_backward(h, W, ids, temp, logp, lse, g, bias=b, kept=keep)
    s, grads = hp.reference()
    tols = hp.tolerances(s, grads)
    what = f"n={n} d={d} V={V} bias={bias} kept={kept}"
    _near(_f(logp), s.logp, tols[0], what + " logp")
    _near(_f(lse), s.lse, tols[1], what + " lse")
    _near(_f(gh), grads[2], tols[2], what + " grad_h")
    _near(_f(gW), grads[3], tols[3], what + " grad_W")
    assert fs.device_error() == 0


@pytest.mark.parametrize("n,d,V", [(40, 4104, 300), (300, 2056, 515), (1031, 72, 2000), (513, 520, 1030)])
def test_long_sums_and_several_column_tiles(fs, torch_cuda, n, d, V):
    """Widths whose logits are formed in several pieces; more tokens than one
    and than four tiles hold."""
    test_scores_and_gradients(fs, torch_cuda, n, d, V, "shared", True)
    test_scores_and_gradients(fs, torch_cuda, n, d, V, "rows", False)


def test_vocabulary_in_pieces(fs, torch_cuda):
    """So many tokens that ds is formed for a part of the vocabulary at a time
    (4 GiB): both pieces' grad_W, and grad_h over both."""
    torch = torch_cuda
    n, d, V = 70000, 8, 33000
    gen = torch.Generator(device="cuda").manual_seed(3)
    h = torch.randn(n, d, generator=gen, device="cuda").bfloat16()
    W = torch.randn(V, d, generator=gen, device="cuda").bfloat16()
    ids = torch.randint(0, V, (n,), generator=gen, device="cuda")
    temp, g = torch.ones(n, device="cuda"), torch.randn(n, generator=gen, device="cuda")
    logp, lse = fs.token_logprobs(h, W, ids, temp)
    gh, gW = fs.token_logprobs_backward(h, W, ids, temp, logp, lse, g)
    keep = fs.logprob_buffer(n, V)
    logp2, lse2 = fs.token_logprobs(h, W, ids, temp, kept=keep)
    gh2, gW2 = fs.token_logprobs_backward(h, W, ids, temp, logp2, lse2, g, kept=keep)
    assert torch.equal(logp, logp2) and torch.equal(lse, lse2)
    W64 = W.double()
    want_W = torch.zeros(V, d, dtype=torch.float64, device="cuda")
    size_W = torch.zeros_like(want_W)
    for i in range(0, n, 5000):
        at = slice(i, i + 5000)
        h64 = h[at].double()
        x = h64 @ W64.T
        z = x.logsumexp(1)
        assert float((lse[at].double() - z).abs().max()) < 1e-4
        ds = -(x - z[:, None]).exp()
        ds[torch.arange(ds.shape[0], device="cuda"), ids[at]] += 1
        ds *= g[at].double()[:, None]
        want = ds @ W64
        # ds and the result rounded to bf16, fp32 sums of V terms
        tol = (2.0 ** -8 + 2.0 ** -12) * (ds.abs() @ W64.abs()) + 2.0 ** -8 * want.abs()
        for got in (gh, gh2):
            assert bool(((got[at].double() - want).abs() <= tol).all())
        want_W += ds.T @ h64
        size_W += ds.abs().T @ h64.abs()
    tol = (2.0 ** -8 + 2.0 ** -10) * size_W + 2.0 ** -8 * want_W.abs()
    for got in (gW, gW2):
        assert bool(((got.double() - want_W).abs() <= tol).all())


@pytest.mark.parametrize("n", [100, 300])
def test_a_head_larger_than_l2(fs, torch_cuda, n):
    """139 MB of W and of grad_W, logits formed in several pieces."""
    torch = torch_cuda
    d, V = 4096, 17001
    gen = torch.Generator(device="cuda").manual_seed(n)
    h = torch.randn(n, d, generator=gen, device="cuda").bfloat16()
    W = (torch.randn(V, d, generator=gen, device="cuda") * 1.5 / 64).bfloat16()
    ids = torch.randint(0, V, (n,), generator=gen, device="cuda")
    ids[3:9] = ids[3]                                      # several tokens with one row of grad_W
    temp, g = torch.ones(n, device="cuda"), torch.randn(n, generator=gen, device="cuda") / n
    logp, lse = fs.token_logprobs(h, W, ids, temp)
    gh, gW = fs.token_logprobs_backward(h, W, ids, temp, logp, lse, g)
    h64, W64 = h.double(), W.double()
    x = h64 @ W64.T
    z = x.logsumexp(1)
    rows = torch.arange(n, device="cuda")
    # d / 16 additions, each cut by at most 2u of what they sum up to
    tol = d / 16 * 2 * U * float((h64.abs() @ W64.abs().T).max())
    assert float((lse.double() - z).abs().max()) < tol and float((logp.double() - (x[rows, ids] - z)).abs().max()) < 2 * tol
    ds = -(x - z[:, None]).exp()
    ds[rows, ids] += 1
    ds *= g.double()[:, None]
    own = torch.zeros_like(ds)
    own[rows, ids] = ds[rows, ids]
    # every entry of ds but the token's own is rounded to bf16; 2^-10 for the scores' error; results rounded once
    for got, want, size, own_size in ((gh, ds @ W64, (ds - own).abs() @ W64.abs(), own.abs() @ W64.abs()),
                                      (gW, ds.T @ h64, (ds - own).abs().T @ h64.abs(), own.abs().T @ h64.abs())):
        tol = (2.0 ** -8 + 2.0 ** -10) * size + 2.0 ** -10 * own_size + 2.0 ** -8 * want.abs()
        assert bool(((got.double() - want).abs() <= tol).all())


@pytest.mark.parametrize("kept", [True, False])
@pytest.mark.parametrize("n", [9, 150])
def test_rows_that_take_no_part(fs, torch_cuda, n, kept):
    """Ids outside the vocabulary, invalid temperatures, rows whose mask leaves
    nothing, a token that is masked, rows of NaN: no other row notices."""
    torch = torch_cuda
    d, V = 64, 300
    hp = Head(n, d, V, "rows", seed=5)
    hp.ids[:8] = -1, V, 2 ** 40, -2 ** 40, 3, 4, 5, 6
    hp.temp[:9] = 1, 1, 1, 1, np.nan, -1, 1, 1, 0
    hp.bias[6] = -np.inf
    hp.bias[7, 6] = -np.inf
    hp.g[:9] = 1.0
    hp.ids[8] = 17
    clean = hp.h.copy()
    hp.hb[:6] = 0x7FC0                                     # NaN in rows that take no part
    bias = hp.bias.copy()
    h, W, ids, temp, b, g = hp.device(torch)
    keep = fs.logprob_buffer(n, V) if kept else None
    logp, lse = fs.token_logprobs(h, W, ids, temp, bias=b, kept=keep)
    gh, gW = fs.token_logprobs_backward(h, W, ids, temp, logp, lse, g, bias=b, kept=keep)
    hp.h, hp.bias = clean, bias
    s, grads = hp.reference()
    assert list(grads[1][:9]) == [False] * 8 + [True]
    tols = hp.tolerances(s, grads)
    got = _f(lse)
    assert np.isnan(got[:4]).all() and (got[4:7] == -np.inf).all() and np.isfinite(got[7:]).all()
    got = _f(logp)
    assert (got[:6] == 0).all() and (got[6:8] == -np.inf).all()
    _near(got[8:], s.logp[8:], tols[0][8:], "logp")
    _near(_f(gh), grads[2], tols[2], "grad_h")
    _near(_f(gW), grads[3], tols[3], "grad_W")
    assert (_f(gh)[:8] == 0).all()


@pytest.mark.parametrize("n", [3, 140])
def test_nan_and_infinite_logits_stay_in_their_row(fs, torch_cuda, n):
    torch = torch_cuda
    hp = Head(n, 64, 500, "rows", seed=6)
    hp.ids[:] = np.arange(n) % 500
    hp.bias[0, 7] = np.nan
    hp.bias[1, 8] = np.inf
    h, W, ids, temp, b, g = hp.device(torch)
    logp, lse = (_f(t) for t in fs.token_logprobs(h, W, ids, temp, bias=b))
    assert np.isnan(lse[:2]).all() and np.isnan(logp[:2]).all()
    assert np.isfinite(lse[2:]).all() and np.isfinite(logp[2:]).all()


def test_lowest_value_masks_and_large_logits(fs, torch_cuda):
    """A mask of fp32's lowest value, and logits far outside exp's range."""
    torch = torch_cuda
    hp = Head(70, 64, 1000, "rows", seed=8, scale=300.0)
    hp.bias[:, ::3] = np.finfo(np.float32).min
    hp.bias[3] = np.finfo(np.float32).min                   # nothing but the mask: every entry is equal
    hp.temp[3] = 1.0
    hp.ids[:] = 3 * (np.arange(70) % 300) + 1
    h, W, ids, temp, b, g = hp.device(torch)
    logp, lse = fs.token_logprobs(h, W, ids, temp, bias=b)
    s, grads = hp.reference()
    rows = np.arange(70) != 3
    tols = hp.tolerances(s, grads)
    size = np.abs(hp.h.astype(np.float64)) @ np.abs(hp.W.astype(np.float64)).T + 10
    tx = ((64 + 4) * 2 * U * size * s.inv_t[:, None]).max(1)   # of the entries that are not masked
    _near(_f(lse)[rows], s.lse[rows], (tx + 1000 * U + 8 * U * np.abs(s.lse))[rows], "lse")
    _near(_f(logp)[rows], s.logp[rows], (4 * tx + 1000 * U + 16 * U * np.abs(s.lse))[rows], "logp")
    assert _f(lse)[3] == np.finfo(np.float32).min
    del tols


@pytest.mark.parametrize("n,V", [(0, 40), (5, 0), (0, 0)])
def test_empty(fs, torch_cuda, n, V):
    torch = torch_cuda
    h, W = torch.ones(n, 16, device="cuda").bfloat16(), torch.ones(V, 16, device="cuda").bfloat16()
    ids, temp = torch.zeros(n, dtype=torch.int64, device="cuda"), torch.ones(n, device="cuda")
    logp, lse = fs.token_logprobs(h, W, ids, temp)
    assert (_f(lse) == -np.inf).all() and (_f(logp) == 0).all()
    gh, gW = fs.token_logprobs_backward(h, W, ids, temp, logp, lse, torch.ones(n, device="cuda"))
    assert gh.shape == (n, 16) and gW.shape == (V, 16) and not _f(gh).any() and not _f(gW).any()


def test_scores_of_the_samplers_own_tokens(fs, torch_cuda):
    """Sampled ids with the sampler's temperatures and bias: frequencies and
    scores describe one distribution (greedy rows score under softmax of the
    logits)."""
    torch = torch_cuda
    V, rows = 24, 4096
    hp = Head(1, 64, V, "shared", seed=9)
    h = to_device(hp.hb, torch).expand(rows, -1).contiguous()
    W, bias = to_device(hp.Wb, torch), to_device(hp.bias, torch)
    temp = torch.full((rows,), 0.8, device="cuda")
    ids, _ = fs.sample(h, W, temp, 1234, 0, bias=bias)
    logp, _ = fs.token_logprobs(h, W, ids, temp, bias=bias)
    got = np.bincount(ids.cpu().numpy(), minlength=V) / rows
    every, _ = fs.token_logprobs(h[:V], W, torch.arange(V, device="cuda"), temp[:V], bias=bias)
    p = np.exp(_f(every).astype(np.float64))
    assert abs(p.sum() - 1) < 1e-5
    assert np.all(np.abs(got - p) <= 5 * np.sqrt(p * (1 - p) / rows) + 1e-12)     # five standard deviations
    np.testing.assert_array_equal(_f(logp), _f(every)[ids.cpu().numpy()])


def test_one_gradient_alone_and_given_outputs(fs, torch_cuda):
    torch = torch_cuda
    hp = Head(77, 128, 600)
    h, W, ids, temp, b, g = hp.device(torch)
    logp, lse = fs.token_logprobs(h, W, ids, temp)
    gh, gW = fs.token_logprobs_backward(h, W, ids, temp, logp, lse, g)
    a, none = fs.token_logprobs_backward(h, W, ids, temp, logp, lse, g, need_W=False)
    assert none is None and torch.equal(a, gh)
    none, c = fs.token_logprobs_backward(h, W, ids, temp, logp, lse, g, need_h=False)
    assert none is None and torch.equal(c, gW)
    oh, oW = torch.empty_like(h), torch.empty_like(W)
    r = fs.token_logprobs_backward(h, W, ids, temp, logp, lse, g, out=(oh, oW))
    assert r[0] is oh and r[1] is oW and torch.equal(oh, gh) and torch.equal(oW, gW)
    with pytest.raises(fs.FlashSampleError, match="overlap"):
        fs.token_logprobs_backward(h, W, ids, temp, logp, lse, g, out=(h, oW))
    with pytest.raises(fs.FlashSampleError, match="logprob_buffer"):
        fs.token_logprobs(h, W, ids, temp, kept=torch.empty(5, device="cuda"))
    with pytest.raises(fs.FlashSampleError, match="contiguous"):
        fs.token_logprobs(h[:, ::2], W[:, ::2], ids, temp)
    with pytest.raises(fs.FlashSampleError, match="aligned"):
        fs.token_logprobs(torch.empty(77 * 128 + 1, device="cuda").bfloat16()[1:].view(77, 128), W, ids, temp)


def test_outputs_stay_inside_their_buffers(fs, torch_cuda):
    """Guard bands around every output, odd sizes."""
    torch = torch_cuda
    n, d, V = 131, 72, 777
    hp = Head(n, d, V, "rows", seed=3)
    h, W, ids, temp, b, g = hp.device(torch)

    def guarded(count, dtype):
        buf = torch.full((count + 256,), 7.0, dtype=dtype, device="cuda")
        return buf, buf[128:128 + count]

    bufs = [guarded(n, torch.float32), guarded(n, torch.float32), guarded(n * d, torch.bfloat16),
            guarded(V * d, torch.bfloat16), guarded(fs.logprob_buffer(n, V).numel(), torch.float32)]
    out = fs.token_logprobs(h, W, ids, temp, bias=b, kept=bufs[4][1], out=(bufs[0][1], bufs[1][1]))
    for kept in (bufs[4][1], None):
        fs.token_logprobs_backward(h, W, ids, temp, *out, g, bias=b, kept=kept,
                                   out=(bufs[2][1].view(n, d), bufs[3][1].view(V, d)))
    for buf, _ in bufs:
        assert (buf[:128] == 7).all() and (buf[-128:] == 7).all()


def test_scores_are_the_same_each_time_on_another_stream_and_in_a_graph(fs, torch_cuda):
    torch = torch_cuda
    hp = Head(200, 256, 5000, "shared")
    h, W, ids, temp, b, g = hp.device(torch)

    def step(stream=None):
        keep = fs.logprob_buffer(200, 5000)
        logp, lse = fs.token_logprobs(h, W, ids, temp, bias=b, kept=keep, stream=stream)
        return (logp, lse) + fs.token_logprobs_backward(h, W, ids, temp, logp, lse, g, bias=b, kept=keep, stream=stream)

    first = step()
    for a, c in zip(first, step()):
        assert torch.equal(a, c)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(other):
        again = step()
    torch.cuda.current_stream().wait_stream(other)
    for a, c in zip(first, again):
        assert torch.equal(a, c)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=other):
        captured = step()
    old = [t.clone() for t in first]
    h.copy_(torch.flip(h, [0]))
    graph.replay()
    torch.cuda.synchronize()
    assert not torch.equal(captured[0], old[0])
    h.copy_(torch.flip(h, [0]))
    graph.replay()
    torch.cuda.synchronize()
    for a, c in zip(old, captured):
        assert torch.equal(a, c)


def test_directional_derivative(fs, torch_cuda):
    """grad_h and grad_W against differences of the library's own loss."""
    torch = torch_cuda
    hp = Head(40, 128, 900, seed=4)
    h, W, ids, temp, _, g = hp.device(torch)
    g = g.sign() / 4
    logp, lse = fs.token_logprobs(h, W, ids, temp)
    gh, gW = fs.token_logprobs_backward(h, W, ids, temp, logp, lse, g)
    for x, grad in ((h, gh), (W, gW)):
        # along the gradient itself, in steps that the leaves' bf16 can hold
        step = (grad.double() / grad.double().norm() * 0.5)
        up, down = (x.double() + step).bfloat16(), (x.double() - step).bfloat16()
        move = up.double() - down.double()
        f = [float((g.double() * fs.token_logprobs(*((y, W) if x is h else (h, y)), ids, temp)[0].double()).sum())
             for y in (up, down)]
        want = float((grad.double() * move).sum())
        # cubic term of the difference: steps of norm 1/2 against curvature of order one
        assert abs((f[0] - f[1]) - want) <= 0.05 * abs(want) + 1e-3


# ---------------------------------------------------------------- policy loss
def _policy_inputs(lengths, seed, mask, ref, per_seq):
    rng = np.random.default_rng(seed)
    N = int(sum(lengths))
    old = -rng.exponential(1.5, N).astype(np.float32)
    logp = (old + 0.25 * rng.standard_normal(N)).astype(np.float32)
    r = (logp + 0.4 * rng.standard_normal(N)).astype(np.float32) if ref else None
    if ref and N > 4:
        r[:3] = logp[:3] + np.float32([1e-3, -1e-4, 3.0])
    adv = rng.standard_normal(len(lengths) if per_seq else N).astype(np.float32)
    m = rng.random(N) < 0.7 if mask else None
    return logp, old, adv, m, r


def _check_policy(stats, grad, want, logp, old, adv, ref, kl, mask=None):
    N = len(logp)
    if mask is not None:                                   # masked tokens: their gradient is zero, exactly
        logp, old, adv = (np.where(mask, a, np.float32(0)) for a in (logp, old, adv))
        ref = None if ref is None else np.where(mask, ref, np.float32(0))
    w = np.where(np.isfinite(want.weight), want.weight, 0.0)
    d = np.abs(logp.astype(np.float64) - old)
    rA = np.where(np.isfinite(d), np.exp(logp.astype(np.float64) - old) * np.abs(adv), 0.0)
    em = np.zeros(N) if ref is None else np.abs(np.expm1(ref.astype(np.float64) - logp))
    q = np.zeros(N) if ref is None else np.abs(ref.astype(np.float64) - logp)
    # exp within 2 ulp of an argument rounded by half a step of d or q; the
    # products, the weight's division and its product: 8 half steps
    rel = 12 * U
    t_term = w * (rA * (rel + 2 * U * d) + 8 * U * rA)
    t_kl = w * ((em + q) * rel + q * (1 + em) * 2 * U + U * em) * (0 if ref is None else 1)
    t_grad = t_term + abs(kl) * w * (em * rel + (1 + em) * q * 2 * U) + 8 * U * np.abs(want.grad) + 1e-44
    on = np.isfinite(want.grad)
    _near(grad[on], want.grad[on], t_grad[on], "grad")
    take = w > 0
    size = np.where(want.grad != 0, 1, 1)
    t_policy = np.nansum(np.where(take, t_term + w * np.abs(adv) * 2 * U + 8 * U * w * rA, 0) * size) + U * abs(want.policy)
    t_klsum = np.nansum(np.where(take, t_kl, 0)) + U * abs(want.kl)
    for k, (got, x, t) in enumerate(zip(stats, (want.loss, want.policy, want.kl, want.clipped),
                                        (t_policy + abs(kl) * t_klsum + 2 * U * abs(want.loss), t_policy, t_klsum,
                                         8 * U * want.clipped))):
        assert abs(got - x) <= t + 1e-40, (k, got, x, t)


@pytest.mark.parametrize("mean", ["token", "sequence", "none"])
@pytest.mark.parametrize("mask,ref,per_seq", [(False, False, False), (True, True, True), (False, True, True),
                                              (True, False, False)])
@pytest.mark.parametrize("lengths", [[1], [5], [3, 0, 0, 900, 1, 1, 31, 0], [4096, 4095, 2], list(range(0, 300, 7)),
                                     [0, 0, 40000, 0]])
def test_policy_loss(fs, torch_cuda, lengths, mask, ref, per_seq, mean):
    torch = torch_cuda
    logp, old, adv, m, r = _policy_inputs(lengths, len(lengths), mask, ref, per_seq)
    kl = 0.07 if ref else 0.0
    starts = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int64, device="cuda")
    dev = lambda a: None if a is None else torch.from_numpy(a).cuda()  # noqa: E731
    if m is not None:
        logp[~m] = np.nan                                  # nobody wrote anything there
        old[~m] = np.inf
    args = (dev(logp), dev(old), dev(adv))
    kw = dict(seq_starts=starts, mask=dev(m), ref_logp=dev(r), clip_low=0.2, clip_high=0.3, kl_coef=kl, mean=mean,
              adv_per_seq=per_seq)
    stats, grad = fs.policy_loss(*args, **kw)
    full = np.repeat(adv, lengths) if per_seq else adv
    want = tr.policy(logp, old, full, lengths, m, r, 0.2, 0.3, kl, mean)
    _check_policy(_f(stats).astype(np.float64), _f(grad), want, logp, old, full, r, kl, m)
    again, grad2 = fs.policy_loss(*args, **kw)
    assert torch.equal(stats, again) and torch.equal(grad, grad2)
    # the same tokens from addresses that are not aligned for wide loads
    shift = lambda t: None if t is None else torch.cat((t[:1], t))[1:]  # noqa: E731
    _, grad3 = fs.policy_loss(shift(args[0]), shift(args[1]), args[2] if per_seq else shift(args[2]),
                              **dict(kw, mask=shift(kw["mask"]), ref_logp=shift(kw["ref_logp"])))
    assert torch.equal(grad, grad3)


@pytest.mark.parametrize("mean", ["token", "sequence"])
def test_policy_loss_padded(fs, torch_cuda, mean):
    torch = torch_cuda
    S, L = 13, 77
    logp, old, adv, m, r = _policy_inputs([L] * S, 4, True, True, True)
    m[3 * L:5 * L] = False
    dev = lambda a: torch.from_numpy(a).cuda().view(S, L)  # noqa: E731
    stats, grad = fs.policy_loss(dev(logp), dev(old), torch.from_numpy(adv).cuda(), mask=dev(m), ref_logp=dev(r),
                                 kl_coef=0.1, mean=mean)
    want = tr.policy(logp, old, np.repeat(adv, L), [L] * S, m, r, kl_coef=0.1, mean=mean)
    assert grad.shape == (S, L)
    _check_policy(_f(stats).astype(np.float64), _f(grad).ravel(), want, logp, old, np.repeat(adv, L), r, 0.1, m)


def test_policy_loss_borders(fs, torch_cuda):
    """Log ratios on a border and one step either side are decided as in fp64."""
    torch = torch_cuda
    hi, lo = math.log1p(0.2), math.log1p(-0.2)
    old = np.zeros(4000, np.float32)
    old[1::2] = -3.7
    step = np.arange(-1000, 1000, dtype=np.float64) * 2.0 ** -23
    logp = np.concatenate([old[:2000] + hi + step, old[2000:] + lo + step]).astype(np.float32)
    adv = np.where(np.arange(4000) < 2000, 1.0, -1.0).astype(np.float32)
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    stats, grad = fs.policy_loss(dev(logp), dev(old), dev(adv), mean="none")
    want = tr.policy(logp, old, adv, [4000], mean="none")
    np.testing.assert_array_equal(_f(grad) == 0, want.is_clipped)
    assert float(stats[3]) == want.is_clipped.sum()


def test_policy_loss_where_nothing_is_left(fs, torch_cuda):
    torch = torch_cuda
    logp = torch.full((2, 9), math.nan, device="cuda")
    for mean in ("token", "sequence", "none"):
        stats, grad = fs.policy_loss(logp, logp, torch.ones(2, device="cuda"), mask=torch.zeros(2, 9, dtype=torch.bool, device="cuda"),
                                     ref_logp=logp, kl_coef=0.1, mean=mean)
        assert not _f(stats).any() and not _f(grad).any()
    # and the next call on the stream counts afresh
    x = torch.zeros(2, 9, device="cuda")
    stats, grad = fs.policy_loss(x, x, torch.ones(2, device="cuda"), mask=torch.ones(2, 9, dtype=torch.bool, device="cuda"))
    np.testing.assert_allclose(_f(grad), -1 / 18, rtol=4 * U)
    empty = torch.zeros(0, device="cuda")
    stats, grad = fs.policy_loss(empty, empty, torch.zeros(0, device="cuda"), seq_starts=torch.zeros(1, dtype=torch.int64, device="cuda"),
                                 adv_per_seq=True)
    assert not _f(stats).any() and grad.numel() == 0


def test_policy_loss_refuses(fs, torch_cuda):
    torch = torch_cuda
    x = torch.zeros(6, device="cuda")
    starts = torch.arange(7, device="cuda")
    with pytest.raises(fs.FlashSampleError, match="adv_per_seq"):
        fs.policy_loss(x, x, x, seq_starts=starts)
    with pytest.raises(fs.FlashSampleError, match="mean"):
        fs.policy_loss(x, x, x, mean="tokens")
    with pytest.raises(fs.FlashSampleError, match="mask must be"):
        fs.policy_loss(x, x, x, mask=x)
    with pytest.raises(fs.FlashSampleError, match="ref_logp"):
        fs.policy_loss(x, x, x, kl_coef=0.1)
    with pytest.raises(fs.FlashSampleError, match="shape"):
        fs.policy_loss(x, x[:5].clone(), x)
    with pytest.raises(fs.FlashSampleError, match="contiguous"):
        fs.policy_loss(x.expand(3, 6).t(), x.expand(3, 6).t(), x)


# ---------------------------------------------------------------- gradient norm
def _half(torch, dtype):
    return {torch.float32: U, torch.bfloat16: HALF_BF16, torch.float16: HALF_FP16}[dtype]


def _grads(torch, sizes, dtypes, seed=0, scale=0.1):
    gen = torch.Generator().manual_seed(seed)
    return [(torch.randn(s, generator=gen) * scale).to(dt).cuda() for s, dt in zip(sizes, dtypes)]


@pytest.mark.parametrize("sizes", [[1], [0, 5, 0], [16384, 16383, 16385, 7], [100000, 3, 1 << 20], [13] * 49, [31] * 700])
@pytest.mark.parametrize("max_norm", [0.5, 1e9, 0.0, math.inf])
def test_clip_grad_norm(fs, torch_cuda, sizes, max_norm):
    torch = torch_cuda
    kinds = [torch.float32, torch.bfloat16, torch.float16]
    grads = _grads(torch, sizes, [kinds[i % 3] for i in range(len(sizes))], seed=len(sizes))
    host = [g.double().cpu().numpy() for g in grads]
    want = tr.grad_norm(host)
    t_norm = 40 * U                          # squares of 64 in fp32 each 64 half steps of their sum at most, halved by the root
    outs = [torch.empty_like(g) for g in grads]
    norm = fs.clip_grad_norm(grads, max_norm, out=outs)
    assert norm.shape == () and abs(float(norm) - want) <= t_norm * want
    for g, x in zip(grads, host):
        np.testing.assert_array_equal(g.double().cpu().numpy(), x)
    f = tr.clip_factor(want, max_norm)
    for g, o, x in zip(grads, outs, host):
        tol = np.abs(x * f) * (_half(torch, g.dtype) * 1.01 + t_norm + 3 * U) + (2.0 ** -24 if g.dtype == torch.float16 else 1e-38)
        _near(o.double().cpu().numpy(), x * f, tol, f"{g.dtype} out")
        if f == 1.0:
            assert torch.equal(o, g)
    same = fs.clip_grad_norm(grads, max_norm)
    assert torch.equal(same, norm)
    for g, o in zip(grads, outs):
        assert torch.equal(g, o)


def test_clip_grad_norm_of_the_largest(fs, torch_cuda):
    torch = torch_cuda
    grads = _grads(torch, [1000, 17, 40000], [torch.bfloat16, torch.float32, torch.float16], seed=3)
    want = max(float(g.float().abs().max()) for g in grads)
    assert float(fs.clip_grad_norm(grads, math.inf, norm_type=math.inf)) == want


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("norm_type", [2.0, math.inf])
def test_clip_grad_norm_that_is_not_finite_scales_nothing(fs, torch_cuda, bad, norm_type):
    torch = torch_cuda
    grads = _grads(torch, [5000, 33], [torch.bfloat16, torch.float32])
    grads[0][4097] = bad
    old = [g.clone() for g in grads]
    norm = float(fs.clip_grad_norm(grads, 1.0, norm_type=norm_type))
    assert math.isnan(norm) if math.isnan(bad) else norm == math.inf
    for g, o in zip(grads, old):
        assert torch.equal(g.view(torch.int16 if g.dtype == torch.bfloat16 else torch.int32),
                           o.view(torch.int16 if g.dtype == torch.bfloat16 else torch.int32))
    clean = _grads(torch, [5000], [torch.float32])
    assert math.isfinite(float(fs.clip_grad_norm(clean, 1.0, norm_type=norm_type)))


def test_clip_grad_norm_of_views_and_none(fs, torch_cuda):
    """Odd offsets into a flat buffer; the neighbours stay as they are."""
    torch = torch_cuda
    for dtype in (torch.float32, torch.bfloat16):
        flat = _grads(torch, [40000], [dtype], scale=1.0)[0]
        old = flat.clone()
        views = [flat[1:17000], flat[17003:17004], flat[20001:39999]]
        want = tr.grad_norm([v.double().cpu().numpy() for v in views])
        assert abs(float(fs.clip_grad_norm(views, 1.0)) - want) <= 40 * U * want
        hit = torch.zeros(40000, dtype=torch.bool, device="cuda")
        for a, b in ((1, 17000), (17003, 17004), (20001, 39999)):
            hit[a:b] = True
        assert torch.equal(flat[~hit], old[~hit])
        _near(flat[hit].double().cpu().numpy(), old[hit].double().cpu().numpy() / want,
              np.abs(old[hit].double().cpu().numpy() / want) * (_half(torch, dtype) * 1.01 + 50 * U) + 1e-6 * 1e-3, "views")
    assert float(fs.clip_grad_norm([], 1.0)) == 0.0
    with pytest.raises(fs.FlashSampleError, match="overlaps"):
        fs.clip_grad_norm([flat[:100]], 1.0, out=[flat[50:150]])
    with pytest.raises(fs.FlashSampleError, match="type and shape"):
        fs.clip_grad_norm([flat[:100]], 1.0, out=[flat[:99]])
    with pytest.raises(fs.FlashSampleError, match="contiguous"):
        fs.clip_grad_norm([flat[::2]], 1.0)


def test_policy_and_clip_in_a_graph(fs, torch_cuda):
    """Both can be captured once their stream's workspace is reserved, and
    replays take the tensors' new contents."""
    torch = torch_cuda
    logp, old, adv, m, r = _policy_inputs([50, 70], 1, True, True, True)
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    a = [dev(x) for x in (logp, old, adv, m, r)]
    starts = torch.tensor([0, 50, 120], device="cuda")
    g = _grads(torch, [3000], [torch.float32])[0]
    src = g.clone()
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    fs.check(fs.library().fs_workspace_release())          # another test may have used this stream
    with pytest.raises(fs.FlashSampleError) as e:
        with torch.cuda.graph(torch.cuda.CUDAGraph(), stream=stream):
            fs.clip_grad_norm([g], 1.0)
    assert e.value.status == "FS_ERR_WORKSPACE"
    torch.cuda.synchronize()
    fs.workspace_reserve(1, 1, stream=stream)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        stats, grad = fs.policy_loss(a[0], a[1], a[2], seq_starts=starts, mask=a[3], ref_logp=a[4], kl_coef=0.1, mean="sequence")
        norm = fs.clip_grad_norm([g], 1.0)
    for k in (1.0, 2.0):
        a[2].copy_(dev(adv) * k)
        g.copy_(src * k)
        graph.replay()
        torch.cuda.synchronize()
        s2, g2 = fs.policy_loss(a[0], a[1], a[2], seq_starts=starts, mask=a[3], ref_logp=a[4], kl_coef=0.1, mean="sequence")
        assert torch.equal(stats, s2) and torch.equal(grad, g2)
        assert abs(float(norm) - k * float(src.double().norm())) <= 40 * U * float(norm) and float(g.norm()) <= 1.0001


def test_injected_failures_are_reported_and_passed(fs, torch_cuda):
    """A failing launch or allocation comes back as the call's error, and the
    next call works."""
    torch = torch_cuda
    hp = Head(20, 64, 200)
    h, W, ids, temp, _, g = hp.device(torch)
    logp, lse = fs.token_logprobs(h, W, ids, temp)
    calls = [lambda s=None: fs.token_logprobs(h, W, ids, temp, stream=s),
             lambda s=None: fs.token_logprobs_backward(h, W, ids, temp, logp, lse, g, stream=s),
             lambda s=None: fs.policy_loss(logp, logp, g, stream=s), lambda s=None: fs.clip_grad_norm([g.clone()], 1.0, stream=s)]
    torch.cuda.synchronize()
    for call in calls:
        fs.debug_set_fault(fs.FS_FAULT_LAUNCH)
        try:
            with pytest.raises(fs.FlashSampleError) as e:
                call()
        finally:
            fs.debug_set_fault(fs.FS_FAULT_NONE)
        assert e.value.status == "FS_ERR_CUDA" and "injected" in str(e.value)
        call()
    for call in (calls[0], calls[2], calls[3]):              # those that need the library's block on a new stream
        fs.check(fs.library().fs_workspace_release())
        stream = torch.cuda.Stream()
        fs.debug_set_fault(fs.FS_FAULT_ALLOC)
        try:
            with pytest.raises(fs.FlashSampleError) as e:
                call(stream)
        finally:
            fs.debug_set_fault(fs.FS_FAULT_NONE)
        assert e.value.status == "FS_ERR_WORKSPACE"
        call(stream)
    torch.cuda.synchronize()
    assert fs.device_error() == 0
