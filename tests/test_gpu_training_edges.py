"""The training operators where their values are extreme, against fp64.

u = 2^-24 is the half step of fp32, 2^-8 that of bf16.  Logits are put in
through the bias alone (h or W is zero), so they are exact, and what is left
is the error of the operators themselves.
"""

import math

import numpy as np
import pytest

from lm_head_exact_gb300 import synthetic
from oracle import training as tr

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF_BF16 = 2.0 ** -8


def _bf16(torch, x):
    bits = synthetic.bf16_bits(np.asarray(x, np.float32))
    return torch.from_numpy(bits.view(np.int16)).cuda().view(torch.bfloat16), synthetic.bf16_bits_to_f32(bits)


def _host(t):
    return t.detach().double().cpu().numpy()


class NearCertain:
    """n rows whose own token has probability 1 - delta at logits around level;
    the rest is spread over 1 to 40 other tokens."""

    V = 1000

    def __init__(self, n, seed=0):
        rng = np.random.default_rng(seed)
        self.bias = np.full((n, self.V), -np.inf, np.float32)
        self.ids = np.arange(n) % 500
        self.delta = np.array([1e-3, 1e-4, 1e-5])[np.arange(n) % 3]
        for t in range(n):
            level = np.float32([20.0, 200.0, -150.0, 3000.0][t // 3 % 4] + rng.random())
            others = rng.choice(np.arange(500, self.V), rng.integers(1, 41), replace=False)
            w = rng.uniform(0.5, 1.5, len(others))
            self.bias[t, self.ids[t]] = level
            self.bias[t, others] = level + np.log(w / w.sum() * self.delta[t])
        self.temp = np.array([1.0, 0.5], np.float32)[rng.integers(0, 2, n)]
        self.bias *= self.temp[:, None]                    # exact: powers of two
        self.g = rng.uniform(0.5, 2.0, n).astype(np.float32) * rng.choice([-1, 1], n).astype(np.float32)

    def device(self, torch):
        return tuple(torch.from_numpy(a).cuda() for a in (self.ids, self.temp, self.bias, self.g))


# 1 - p = sum of the others' exp over s.  An exponential is within 2^-22, its argument (at most 16, after
# the scaling to base 2) within half a step twice: 2^-19 of the sum.  The largest term, 1, is in at most
# 22 additions (5 within a warp's rows, 1 with the tile before, 16 in the merge), each off by u.
REL, ABS = 2.0 ** -19, 24 * U


@pytest.mark.parametrize("n", [12, 300])
def test_scores_of_near_certain_tokens(fs, torch_cuda, n):
    torch = torch_cuda
    c = NearCertain(n)
    ids, temp, bias, _ = c.device(torch)
    h, W = torch.zeros(n, 8, device="cuda").bfloat16(), torch.ones(c.V, 8, device="cuda").bfloat16()
    logp, lse = fs.token_logprobs(h, W, ids, temp, bias=bias)
    s = tr.scores(np.zeros((n, 8)), np.ones((c.V, 8)), c.ids, c.temp, c.bias)
    assert np.all(np.abs(s.logp + c.delta) < 0.01 * c.delta)
    assert np.all(np.abs(_host(logp) - s.logp) <= REL * np.abs(s.logp) + ABS)
    assert np.all(np.abs(_host(lse) - s.lse) <= 2 * U * np.abs(s.lse) + ABS)
    assert np.all(_host(logp) <= 0)


@pytest.mark.parametrize("kept", [True, False])
@pytest.mark.parametrize("n", [12, 300])
def test_gradients_of_near_certain_tokens(fs, torch_cuda, n, kept):
    """Their own entries of ds to what (1 - p) is known to; the others to the
    half step of bf16 in which the products take them."""
    torch = torch_cuda
    c = NearCertain(n, seed=1)
    ids, temp, bias, g = c.device(torch)
    rng = np.random.default_rng(2)
    for zero in ("h", "W"):
        h, h64 = _bf16(torch, np.zeros((n, 16)) if zero == "h" else rng.standard_normal((n, 16)))
        W, W64 = _bf16(torch, np.zeros((c.V, 16)) if zero == "W" else rng.standard_normal((c.V, 16)))
        keep = fs.logprob_buffer(n, c.V) if kept else None
        logp, lse = fs.token_logprobs(h, W, ids, temp, bias=bias, kept=keep)
        gh, gW = fs.token_logprobs_backward(h, W, ids, temp, logp, lse, g, bias=bias, kept=keep)
        s = tr.scores(h64, W64, c.ids, c.temp, c.bias)
        ds, live, want_h, want_W = tr.score_gradients(h64, W64, c.ids, s, c.g)
        assert live.all()
        coef = np.abs(c.g * s.inv_t)
        rows = np.arange(n)
        # the own entry: 1 - p as above, its remainder added in fp32
        t_ds = np.abs(ds) * (HALF_BF16 + REL + 2 * U * np.abs(s.lse)[:, None])
        t_ds[rows, c.ids] = np.abs(ds[rows, c.ids]) * (REL + 8 * U) + coef * ABS
        for got, want, tol in ((gh, want_h, t_ds @ np.abs(W64) + 64 * U * (np.abs(ds) @ np.abs(W64))),
                               (gW, want_W, t_ds.T @ np.abs(h64) + 64 * U * (np.abs(ds).T @ np.abs(h64)))):
            tol = 1.01 * tol + HALF_BF16 * np.abs(want) + 1e-37
            over = np.abs(_host(got) - want) / tol
            assert over.max() <= 1, (zero, over.max(), np.unravel_index(over.argmax(), over.shape))


@pytest.mark.parametrize("kept", [True, False])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("n", [3, 300])
def test_a_masked_token_in_a_row_that_is_not_finite(fs, torch_cuda, n, bad, kept):
    """logp is NaN like lse, not -inf, and the row's gradient is NaN, not
    zero; the other rows' scores and grad_h are as without it."""
    torch = torch_cuda
    gen = torch.Generator(device="cuda").manual_seed(n)
    h, W = (torch.randn(m, 64, generator=gen, device="cuda").bfloat16() for m in (n, 500))
    ids, temp, g = torch.arange(n, device="cuda"), torch.ones(n, device="cuda"), torch.ones(n, device="cuda")
    results = []
    for x in (0.0, bad):
        bias = torch.zeros(n, 500, device="cuda")
        bias[1, 1] = -math.inf if x else 0.0               # the token of row 1
        bias[1, 400] = x
        keep = fs.logprob_buffer(n, 500) if kept else None
        logp, lse = fs.token_logprobs(h, W, ids, temp, bias=bias, kept=keep)
        gh, _ = fs.token_logprobs_backward(h, W, ids, temp, logp, lse, g, bias=bias, kept=keep)
        results.append((logp, lse, gh))
    rest = torch.arange(n, device="cuda") != 1
    for clean, got in zip(*results):
        assert bool(got[1].isnan().all())
        assert torch.equal(clean[rest], got[rest])


def _clip_case(torch, name):
    """Gradients by name: finite, but beyond where fp32 holds their squares."""
    rng = np.random.default_rng(3)
    x = rng.standard_normal(40000)
    return {
        "large": [torch.tensor(x * 1e25).float(), torch.tensor(x[:77] * 1e20).bfloat16()],
        "one_large": [torch.tensor(np.where(np.arange(40000) == 20001, 1e30, x)).float()],
        "norm_past_fp32": [torch.full((20000,), 3e38), torch.full((501,), -3e38).bfloat16()],
        "small": [torch.tensor(x * 1e-21).float(), torch.tensor(x[:300] * 1e-22).bfloat16()],
        "small_and_zero": [torch.zeros(50000), torch.tensor(x[:20000] * 1e-20).float()],
        "odd": [torch.tensor(x[:16391] * 1e22).float()],
    }[name]


@pytest.mark.parametrize("name", ["large", "one_large", "norm_past_fp32", "small", "small_and_zero", "odd"])
def test_clip_grad_norm_of_finite_extremes(fs, torch_cuda, name):
    """Finite gradients have the norm that fp64 gives them and are scaled by
    it, in place and not."""
    torch = torch_cuda
    grads = [g.cuda() for g in _clip_case(torch, name)]
    host = [_host(g) for g in grads]
    want = tr.grad_norm(host)
    t_norm = 40 * U                          # squares of 64 in fp32, 64 half steps of their sum, halved by the root
    for max_norm in (1.0, 0.25 * want):
        outs = [torch.empty_like(g) for g in grads]
        norm = float(fs.clip_grad_norm(grads, max_norm, out=outs))
        if want < 3.4e38:
            assert abs(norm - want) <= t_norm * want
        else:
            assert norm == math.inf
        f = tr.clip_factor(want, max_norm)
        for g, o, x in zip(grads, outs, host):
            half = {torch.float32: U, torch.bfloat16: HALF_BF16}[g.dtype]
            # (2^-149: a step of fp32 below its normal range; the first of two factors may leave one, times the other)
            assert np.all(np.abs(_host(o) - x * f) <= np.abs(x * f) * (half * 1.01 + t_norm + 4 * U) + 2.0 ** -149)
        same = [g.clone() for g in grads]
        fs.clip_grad_norm(same, max_norm)
        for a, b in zip(same, outs):
            assert torch.equal(a, b)


@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_clip_grad_norm_of_an_infinity_among_large_values(fs, torch_cuda, bad):
    torch = torch_cuda
    g = torch.full((40000,), 1e30, device="cuda")
    g[333] = bad
    old = g.clone()
    norm = float(fs.clip_grad_norm([g], 1.0))
    assert math.isnan(norm) if math.isnan(bad) else norm == math.inf
    assert torch.equal(g.view(torch.int32), old.view(torch.int32))


def test_policy_loss_of_a_sequence_of_more_than_2_to_the_31_tokens(fs, torch_cuda):
    """One sequence of 2^32 + 5 tokens, weighted by its own length."""
    torch = torch_cuda
    N = (1 << 32) + 5
    x = torch.zeros(N, device="cuda")
    starts = torch.tensor([0, N], device="cuda")
    stats, grad = fs.policy_loss(x, x, torch.ones(1, device="cuda"), seq_starts=starts, mean="sequence", adv_per_seq=True)
    # every term is the weight, 1 / N: two conversions, a product and a division, half a step each
    for at in (slice(0, 1000), slice((1 << 31) - 500, (1 << 31) + 500), slice(N - 1000, N)):
        assert float((grad[at].double() * N + 1).abs().max()) <= 4 * U
    assert abs(float(stats[1]) + 1) <= 20 * U               # (16 rounds of fp32 sums on top)


@pytest.mark.parametrize("mean", ["token", "none"])
def test_policy_loss_of_ratios_past_fp32(fs, torch_cuda, mean):
    """exp(logp - old) above fp32's range: no advantage, no term; a small
    negative one, a finite term."""
    torch = torch_cuda
    logp = np.float32([-0.5, -0.25, -1.0, -0.5, -2.0, -0.125, -0.75])
    old = np.float32([-100.5, -300.0, -91.0, -89.0, -2.5, -120.0, -95.75])
    adv = np.float32([0.0, 0.0, -1e-6, 0.0, 0.5, 1.0, -1e-4])
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    stats, grad = fs.policy_loss(dev(logp), dev(old), dev(adv), mean=mean)
    want = tr.policy(logp, old, adv, [7], mean=mean)
    # exp of half the difference within 2 steps, twice; the products and the weight: 16 half steps
    assert np.all(np.abs(_host(grad) - want.grad) <= 16 * U * np.abs(want.grad))
    for got, x in zip(_host(stats), (want.loss, want.policy, 0.0, want.clipped)):
        assert abs(got - x) <= 20 * U * abs(x)
    inf = torch.full((1,), -math.inf, device="cuda")       # 0 times an infinite ratio is none of these
    assert math.isnan(float(fs.policy_loss(torch.zeros(1, device="cuda"), inf, torch.zeros(1, device="cuda"))[0][0]))


def test_policy_loss_that_only_measures_the_kl(fs, torch_cuda):
    """kl_coef 0: an estimate past fp32's range is reported, and neither loss
    nor gradient holds a NaN from 0 times infinity."""
    torch = torch_cuda
    logp = np.float32([-100.0, -0.5, -1.0])
    old = np.float32([-99.5, -0.5, -1.25])
    adv = np.float32([-0.5, 1.0, -1.0])
    ref = np.float32([-0.5, -0.75, -1.0])
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    stats, grad = fs.policy_loss(dev(logp), dev(old), dev(adv), ref_logp=dev(ref))
    want = tr.policy(logp, old, adv, [3], ref=ref)
    assert np.all(np.abs(_host(grad) - want.grad) <= 16 * U * np.abs(want.grad))
    got = _host(stats)
    assert abs(got[0] - want.policy) <= 20 * U and abs(got[1] - want.policy) <= 20 * U and got[2] == math.inf
    plain, grad2 = fs.policy_loss(dev(logp), dev(old), dev(adv))
    assert torch.equal(grad, grad2) and torch.equal(plain[:2], stats[:2])


def _peaked_tolerances(hp, s, grads):
    """As Head.tolerances, with an own entry whose remainder is added in fp32
    and which is known to what 1 - p is."""
    ds, live, gh, gW = grads
    n, V, d = len(hp.ids), hp.W.shape[0], hp.h.shape[1]
    rows = np.nonzero(live)[0]
    h64 = np.where(live[:, None], np.abs(hp.h.astype(np.float64)), 0.0)
    W64 = np.abs(hp.W.astype(np.float64))
    size = np.abs(hp.h.astype(np.float64)) @ W64.T
    tx = (d + 4) * 2 * U * size * s.inv_t[:, None]
    t_lse = tx.max(1) + (V / 8 + 32) * U + 4 * U * np.abs(s.lse)
    p = np.where(live[:, None], np.exp(s.x - s.lse[:, None]), 0.0)
    c = np.abs(hp.g.astype(np.float64) * s.inv_t)[:, None] * live[:, None]
    t_ds = c * p * (tx + t_lse[:, None] + 2.0 ** -20 + 8 * U * np.abs(s.lse)[:, None]) + np.abs(ds) * (HALF_BF16 + 4 * U)
    t_ds[rows, hp.ids[rows]] = (c * (tx + t_lse[:, None]))[rows, hp.ids[rows]] + 8 * U * np.abs(ds[rows, hp.ids[rows]])
    tol = [t_ds @ W64 + (V + 32) * 2 * U * (np.abs(ds) @ W64) + HALF_BF16 * np.abs(gh),
           t_ds.T @ h64 + (n + 32) * 2 * U * (np.abs(ds).T @ h64) + HALF_BF16 * np.abs(gW)]
    return [1.01 * t + 1e-37 for t in tol]


@pytest.mark.parametrize("kept", [True, False])
@pytest.mark.parametrize("n,d,V", [(20, 64, 3000), (100, 256, 1000), (300, 72, 1700)])
def test_gradients_of_peaked_rows(fs, torch_cuda, n, d, V, kept):
    """Most of a row's probability on one to three tokens, its own among them
    for half the rows."""
    torch = torch_cuda
    from test_gpu_training import Head
    hp = Head(n, d, V, "none", seed=21, scale=12.0)
    top = np.argmax(hp.h.astype(np.float64) @ hp.W.astype(np.float64).T, 1)
    hp.ids = np.where((np.arange(n) % 2 == 0) & (hp.ids >= 0), top, hp.ids)
    h, W, ids, temp, _, g = hp.device(torch)
    keep = fs.logprob_buffer(n, V) if kept else None
    logp, lse = fs.token_logprobs(h, W, ids, temp, kept=keep)
    got = fs.token_logprobs_backward(h, W, ids, temp, logp, lse, g, kept=keep)
    s, grads = hp.reference()
    for x, want, tol, what in zip(got, grads[2:], _peaked_tolerances(hp, s, grads), ("grad_h", "grad_W")):
        over = np.abs(_host(x) - want) / tol
        assert over.max() <= 1, (what, over.max(), np.unravel_index(over.argmax(), over.shape))


# Rounding a result to bf16 is off by 2^-8 / m / sqrt(3) (m the mantissa in [1, 2), spread evenly over its
# logarithm) in the mean square: 0.00166 of it.  In flat rows the own entry is nearly all of ds; rounding
# it too would make that 0.0023.  The bound lies between, 20% above the first.
FLAT_ERROR = 0.0020


def _error(got, want):
    return float(np.linalg.norm(got - want) / np.linalg.norm(want))


@pytest.mark.parametrize("kept", [True, False])
@pytest.mark.parametrize("n,d,V", [(100, 256, 1000), (300, 520, 1700)])
def test_own_entries_are_not_rounded_to_bf16(fs, torch_cuda, n, d, V, kept):
    torch = torch_cuda
    from test_gpu_training import Head
    hp = Head(n, d, V, "none", seed=21)
    h, W, ids, temp, _, g = hp.device(torch)
    keep = fs.logprob_buffer(n, V) if kept else None
    logp, lse = fs.token_logprobs(h, W, ids, temp, kept=keep)
    got = fs.token_logprobs_backward(h, W, ids, temp, logp, lse, g, kept=keep)
    _, (ds, live, want_h, want_W) = hp.reference()
    assert _error(_host(got[0]), want_h) < FLAT_ERROR and _error(_host(got[1]), want_W) < FLAT_ERROR
    # with every entry of ds rounded, the reference itself is further off
    round_bf16 = lambda a: synthetic.bf16_bits_to_f32(synthetic.bf16_bits(a.astype(np.float32))).astype(np.float64)  # noqa: E731
    ds = round_bf16(ds)
    h64 = np.where(live[:, None], hp.h.astype(np.float64), 0.0)
    assert _error(round_bf16(ds @ hp.W), want_h) > FLAT_ERROR and _error(round_bf16(ds.T @ h64), want_W) > FLAT_ERROR


def test_own_entries_when_the_vocabulary_comes_in_pieces(fs, torch_cuda):
    """So many tokens that ds is formed for a part of the vocabulary at a time:
    the remainder belongs to the piece that holds the token."""
    torch = torch_cuda
    n, d, V = 70000, 64, 33000
    gen = torch.Generator(device="cuda").manual_seed(22)
    h = torch.randn(n, d, generator=gen, device="cuda").bfloat16()
    W = (torch.randn(V, d, generator=gen, device="cuda") / 8).bfloat16()
    ids = torch.randint(0, V, (n,), generator=gen, device="cuda")
    temp, g = torch.ones(n, device="cuda"), torch.randn(n, generator=gen, device="cuda")
    logp, lse = fs.token_logprobs(h, W, ids, temp)
    got = [fs.token_logprobs_backward(h, W, ids, temp, logp, lse, g)]
    keep = fs.logprob_buffer(n, V)
    logp, lse = fs.token_logprobs(h, W, ids, temp, kept=keep)
    got.append(fs.token_logprobs_backward(h, W, ids, temp, logp, lse, g, kept=keep))
    del keep
    W64 = W.double()
    want_h, want_W = torch.empty(n, d, dtype=torch.float64, device="cuda"), torch.zeros_like(W64)
    for i in range(0, n, 5000):
        at = slice(i, i + 5000)
        h64 = h[at].double()
        ds = -(h64 @ W64.T).softmax(1)
        ds[torch.arange(ds.shape[0], device="cuda"), ids[at]] += 1
        ds *= g[at].double()[:, None]
        want_h[at] = ds @ W64
        want_W += ds.T @ h64
    for gh, gW in got:
        for x, want in ((gh, want_h), (gW, want_W)):
            for half in (slice(0, len(x) // 2), slice(len(x) // 2, None)):     # (both pieces of grad_W)
                assert float((x[half].double() - want[half]).norm() / want[half].norm()) < FLAT_ERROR
