"""The fp64 forms of the training operators against what they are defined by:
probabilities that sum to one, and derivatives taken as differences."""

import numpy as np
import pytest

from oracle import training as tr


def _head(n=5, V=11, d=6, seed=0):
    rng = np.random.default_rng(seed)
    ids = rng.integers(0, V, n)
    return rng.standard_normal((n, d)), rng.standard_normal((V, d)), ids, rng.uniform(0.4, 1.6, n)


def test_scores_are_normalized():
    h, W, ids, temp = _head()
    s = tr.scores(h, W, ids, temp)
    np.testing.assert_allclose(np.exp(s.x - s.lse[:, None]).sum(1), 1.0, rtol=1e-12)
    every = [tr.scores(h, W, np.full(5, v), temp).logp for v in range(11)]
    np.testing.assert_allclose(np.exp(every).sum(0), 1.0, rtol=1e-12)


def test_scores_of_rows_that_take_no_part():
    h, W, ids, temp = _head(n=6)
    ids[:3] = -1, 11, 4
    temp[2:5] = np.nan, -1.0, 0.0
    s = tr.scores(h, W, ids, temp)
    assert list(s.scored) == [False, False, False, False, True, True]
    assert (s.logp[:4] == 0).all() and np.isfinite(s.lse[:2]).all() and (s.lse[2:4] == -np.inf).all()
    np.testing.assert_allclose(s.x[4], h[4] @ W.T)
    bias = np.zeros((6, 11))
    bias[0] = -np.inf
    bias[5, ids[5]] = -np.inf
    s = tr.scores(h, W, np.where(np.arange(6) == 0, 3, ids), temp, bias)
    assert s.lse[0] == -np.inf and s.logp[0] == -np.inf and s.logp[5] == -np.inf and np.isfinite(s.lse[5])


def test_score_gradients_are_the_differences():
    h, W, ids, temp = _head()
    ids[1] = -1
    g = np.array([0.7, 1.3, -0.4, 0.0, 1.1])
    bias = np.random.default_rng(1).standard_normal((5, 11))
    s = tr.scores(h, W, ids, temp, bias)
    _, live, gh, gW = tr.score_gradients(h, W, ids, s, g)
    assert list(live) == [True, False, True, False, True]

    def loss(h, W):
        return float((g * tr.scores(h, W, ids, temp, bias).logp).sum())

    eps = 1e-6
    for a, grad in ((h, gh), (W, gW)):
        for at in np.ndindex(a.shape):
            old = a[at]
            a[at] = old + eps
            up = loss(h, W)
            a[at] = old - eps
            down = loss(h, W)
            a[at] = old
            assert abs((up - down) / (2 * eps) - grad[at]) < 1e-8


@pytest.mark.parametrize("mean", ["token", "sequence", "none"])
def test_policy_gradient_is_the_difference(mean):
    rng = np.random.default_rng(3)
    lengths = [4, 0, 7, 1, 9]
    N = sum(lengths)
    logp = -rng.uniform(0.1, 3, N)
    old, ref = logp + 0.3 * rng.standard_normal(N), logp + 0.3 * rng.standard_normal(N)
    adv = rng.standard_normal(N)
    mask = rng.random(N) < 0.8
    mask[11] = False                                   # the sequence of one token is left empty
    args = dict(lengths=lengths, mask=mask, ref=ref, clip_low=0.2, clip_high=0.3, kl_coef=0.1, mean=mean)
    p = tr.policy(logp, old, adv, **args)
    assert p.is_clipped.any() and not p.is_clipped.all()
    eps = 1e-6
    for i in range(N):
        x = logp.copy()
        x[i] += eps
        up = tr.policy(x, old, adv, **args).loss
        x[i] -= 2 * eps
        assert abs((up - tr.policy(x, old, adv, **args).loss) / (2 * eps) - p.grad[i]) < 1e-8
    total = {"token": 1.0, "sequence": 1.0, "none": mask.sum()}[mean]
    np.testing.assert_allclose(p.weight[mask].sum(), total)


def test_policy_clips_by_the_smaller_term():
    old = np.zeros(8)
    logp = np.log([1.5, 1.5, 0.5, 0.5, 1.0, 1.2, 0.8, 3.0])
    adv = np.array([1.0, -1.0, 1.0, -1.0, 1.0, 0.0, 0.0, 2.0])
    p = tr.policy(logp, old, adv, [8])
    r = np.exp(logp)
    np.testing.assert_allclose(p.policy, -np.minimum(r * adv, np.clip(r, 0.8, 1.2) * adv).mean())
    assert list(p.is_clipped) == [True, False, False, True, False, False, False, True]


def test_norm_and_factor():
    a = [np.array([3.0]), np.zeros(0), np.array([[4.0]])]
    assert tr.grad_norm(a) == 5.0 and tr.grad_norm(a, float("inf")) == 4.0 and tr.grad_norm([]) == 0.0
    assert tr.clip_factor(5.0, 10.0) == 1.0 and abs(tr.clip_factor(5.0, 1.0) - 0.2) < 1e-6
    assert tr.clip_factor(np.inf, 1.0) == 1.0 and tr.clip_factor(5.0, 0.0) == 0.0


@pytest.mark.parametrize("bad", [np.nan, np.inf])
def test_scores_of_a_masked_token_in_a_row_that_is_not_finite(bad):
    """A row without a log-sum has no log-probability of any token, of one at
    -inf neither, and such a row's gradient does not vanish unseen."""
    h, W, ids, temp = _head()
    bias = np.zeros((5, 11))
    bias[2, ids[2]] = -np.inf
    bias[2, (ids[2] + 1) % 11] = bad
    with np.errstate(all="ignore"):
        s = tr.scores(h, W, ids, temp, bias)
        ds, live, _, _ = tr.score_gradients(h, W, ids, s, np.ones(5))
    assert np.isnan(s.lse[2]) and np.isnan(s.logp[2]) and live[2] and np.isnan(ds[2]).all()
    assert np.isfinite(s.logp[[0, 1, 3, 4]]).all()
