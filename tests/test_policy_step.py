"""What a policy step passes between the operators, with plain forms of them
on the CPU."""

import pytest

torch = pytest.importorskip("torch")

from lm_head_exact_gb300 import policy_step as ps  # noqa: E402


class Plain:
    """The calls that a policy step makes, in elementary operations; they are
    recorded by name."""

    def __init__(self, sampled):
        self.sampled = sampled
        self.calls = []

    def sample(self, h, W, temp, seed, step, bias=None):
        self.calls.append(("sample", bias))
        return self.sampled, None

    def logprob_buffer(self, n, V, device=None):
        return torch.empty(n, V)

    def _x(self, h, W, temp, bias):
        x = h.float() @ W.float().T
        return (x if bias is None else x + bias) / temp[:, None]

    def token_logprobs(self, h, W, ids, temp, bias=None, kept=None):
        self.calls.append(("token_logprobs", bias))
        lp = self._x(h, W, temp, bias).log_softmax(1)
        scored = (ids >= 0) & (ids < W.shape[0]) & (temp >= 0)
        own = lp.gather(1, ids.clamp(0, W.shape[0] - 1)[:, None])[:, 0]
        return torch.where(scored, own, 0.0), self._x(h, W, temp, bias).logsumexp(1)

    def policy_loss(self, logp, old, adv, seq_starts, mask, ref_logp, clip_low, clip_high, kl_coef, mean, adv_per_seq):
        assert mask is None or mask.dtype == torch.bool
        self.calls.append(("policy_loss", mask))
        A = adv.repeat_interleave(seq_starts.diff())
        on = torch.ones_like(logp, dtype=torch.bool) if mask is None else mask
        g = torch.where(on, -A * (logp - old).exp() / on.sum(), 0.0)
        return torch.stack((g.sum(), g.sum(), 0 * g.sum(), 0 * g.sum())), g

    def token_logprobs_backward(self, h, W, ids, temp, logp, lse, g, bias=None, kept=None):
        self.calls.append(("token_logprobs_backward", bias))
        ds = -self._x(h, W, temp, bias).softmax(1)
        scored = (ids >= 0) & (ids < W.shape[0]) & (temp >= 0)
        ds[torch.arange(len(ids)), ids.clamp(0, W.shape[0] - 1)] += 1
        ds *= torch.where(scored, g / temp, 0.0)[:, None]
        return ds @ W.float(), ds.T @ h.float()

    def clip_grad_norm(self, grads, max_norm):
        norm = torch.cat([g.flatten() for g in grads]).norm()
        self.calls.append(("clip_grad_norm", [g.data_ptr() for g in grads]))
        for g in grads:
            g *= min(1.0, max_norm / (float(norm) + 1e-6))
        return norm


@pytest.fixture
def world(monkeypatch):
    g = torch.Generator().manual_seed(0)
    h, W = torch.randn(12, 16, generator=g), torch.randn(30, 16, generator=g)
    plain = Plain(torch.randint(0, 30, (12,), generator=g))
    monkeypatch.setattr(ps, "fs", plain)
    temp = torch.full((12,), 0.7)
    starts = torch.tensor([0, 4, 5, 12])

    def reward(ids):
        return torch.stack([(ids[a:b] % 3).float().mean() for a, b in zip(starts[:-1], starts[1:])])

    return plain, h, W, temp, starts, reward


def test_a_step_does_not_clip_before_the_body_is_known(world):
    """grad_h is the gradient of activations: without a bound for both
    together, both come as they are."""
    plain, h, W, temp, starts, reward = world
    r = ps.roll_out(h, W, temp, starts, reward, 1, 2)
    out = ps.policy_step(r, W * 1.1)
    assert out.grad_norm is None and not any(name == "clip_grad_norm" for name, _ in plain.calls)
    both = ps.policy_step(r, W * 1.1, max_norm=1e-3)
    norm = torch.cat([out.grad_h.flatten(), out.grad_W.flatten()]).norm()
    assert torch.allclose(both.grad_norm, norm)
    assert torch.allclose(both.grad_W, out.grad_W * 1e-3 / (norm + 1e-6))


def test_the_toy_clips_the_head_alone(world, monkeypatch):
    plain = world[0]
    made = []
    real = ps.policy_step
    monkeypatch.setattr(ps, "policy_step", lambda *a, **k: made.append(real(*a, **k)) or made[-1])
    plain.sampled = torch.arange(8) % 5
    ps.train_toy(steps=1, V=12, d=16, sequences=4, length=2, device="cpu")
    assert len(made) == 2
    assert [c[1] for c in plain.calls if c[0] == "clip_grad_norm"] == [[m.grad_W.data_ptr()] for m in made]


def test_one_sequence_alone_has_no_advantage(world):
    plain, h, W, temp, _, _ = world
    r = ps.roll_out(h, W, temp, torch.tensor([0, 12]), lambda ids: ids.float().mean()[None], 1, 2)
    assert torch.equal(r.advantages, torch.zeros(1))


def test_the_samplers_bias_reaches_every_score(world):
    """Tokens drawn under a bias are scored, and differentiated, under it: the
    ratio of an unchanged policy is 1."""
    plain, h, W, temp, starts, reward = world
    bias = torch.where(torch.arange(30) % 4 == 0, -float("inf"), 0.0)
    plain.sampled = plain.sampled // 4 * 4 + 1
    plain.sampled.clamp_(max=29)
    r = ps.roll_out(h, W, temp, starts, reward, 1, 2, bias=bias)
    out = ps.policy_step(r, W)
    torch.testing.assert_close(out.logp, r.old_logp)
    torch.testing.assert_close(r.old_logp, plain.token_logprobs(h, W, r.ids, temp, bias)[0])
    assert not out.grad_W[::4].any()                       # forbidden tokens learn nothing
    names = [name for name, b in plain.calls if b is bias]
    assert names.count("sample") == 1 and names.count("token_logprobs") == 3 and "token_logprobs_backward" in names


@pytest.mark.parametrize("masked", [False, True])
def test_rows_without_a_token_take_no_part(world, masked):
    """Neither the loss nor its means see the sampler's -1 or rows whose
    temperature is invalid."""
    plain, h, W, temp, starts, reward = world
    temp = temp.clone()
    plain.sampled[3] = -1
    temp[7] = -1.0
    temp[8] = float("nan")
    r = ps.roll_out(h, W, temp, starts, reward, 1, 2)
    if masked:
        r.mask = torch.arange(12) != 5
    out = ps.policy_step(r, W)
    took = [m for name, m in plain.calls if name == "policy_loss"][0]
    assert [i for i in range(12) if not took[i]] == ([3, 5, 7, 8] if masked else [3, 7, 8])
    A = r.advantages.repeat_interleave(starts.diff())
    assert torch.allclose(out.stats[0], -A[took].mean(), atol=1e-6)
