"""Plain fp64 forms of the training operators: token log-probabilities through
the LM head with gradients, the clipped policy loss, the global gradient norm.
Test infrastructure only; written from the formulas in include/flashsample.h.
"""

from dataclasses import dataclass

import numpy as np


@dataclass
class Scores:
    x: np.ndarray        # scaled logits [n, V]
    lse: np.ndarray      # [n]
    logp: np.ndarray     # [n]
    scored: np.ndarray   # bool [n]
    inv_t: np.ndarray    # [n], 0 where the temperature is invalid


def scores(h, W, ids, temp, bias=None):
    """x = (h W^T + bias) / T; log-sum-exp; log-probability of ids (fp64)."""
    h, W, temp = (np.asarray(a, np.float64) for a in (h, W, temp))
    ids = np.asarray(ids)
    V = W.shape[0]
    x = h @ W.T
    if bias is not None:
        x = x + np.asarray(bias, np.float64)
    with np.errstate(all="ignore"):
        valid = temp >= 0
        inv_t = np.where(temp > 0, 1 / temp, np.where(temp == 0, 1.0, 0.0))
        x = x * inv_t[:, None]
        scored = valid & (ids >= 0) & (ids < V)
        if V == 0:
            lse = np.full(len(temp), -np.inf)
        else:
            top = x.max(1)
            shift = np.where(np.isfinite(top), top, 0.0)
            lse = shift + np.log(np.exp(x - shift[:, None]).sum(1))
            lse = np.where(np.isnan(x).any(1) | (x == np.inf).any(1), np.nan, lse)
        lse = np.where(valid, lse, -np.inf)
        own = x[np.arange(len(ids)), np.where(scored, ids, 0)] if V else np.zeros(len(ids))
        logp = np.where(scored, np.where((own == -np.inf) & ~np.isnan(lse), -np.inf, own - lse), 0.0)
    return Scores(x, lse, logp, scored, inv_t)


def score_gradients(h, W, ids, s, g):
    """(ds [n, V], live [n], grad_h [n, d], grad_W [V, d]) of scores() for
    dL/dlogp = g; rows that carry no gradient take no part."""
    h, W, g = (np.asarray(a, np.float64) for a in (h, W, g))
    ids = np.asarray(ids)
    live = s.scored & (g != 0) & (s.lse != -np.inf) & (s.logp != -np.inf)
    ds = np.zeros(s.x.shape)
    for t in np.nonzero(live)[0]:
        ds[t] = -np.exp(s.x[t] - s.lse[t])
        ds[t, ids[t]] += 1.0
        ds[t] *= g[t] * s.inv_t[t]
    return ds, live, ds @ W, ds.T @ np.where(live[:, None], h, 0.0)


@dataclass
class Policy:
    loss: float
    policy: float
    kl: float
    clipped: float
    grad: np.ndarray
    weight: np.ndarray
    is_clipped: np.ndarray


def policy(logp, old, adv, lengths, mask=None, ref=None, clip_low=0.2, clip_high=0.2, kl_coef=0.0, mean="token"):
    """The loss over packed tokens of sequences with these lengths; adv is
    given per token."""
    logp, old, adv = (np.asarray(a, np.float64) for a in (logp, old, adv))
    N = len(logp)
    on = np.ones(N, bool) if mask is None else np.asarray(mask, bool)
    seq = np.repeat(np.arange(len(lengths)), lengths)
    if mean == "token":
        weight = np.full(N, 1.0 / max(1, on.sum()))
    elif mean == "none":
        weight = np.ones(N)
    else:
        count = np.bincount(seq[on], minlength=len(lengths))
        with np.errstate(divide="ignore"):
            weight = 1.0 / (count[seq] * max(1, (count > 0).sum()))
    loss = kl = clipped = 0.0
    grad, is_clipped = np.zeros(N), np.zeros(N, bool)
    for i in np.nonzero(on)[0]:
        delta, A = logp[i] - old[i], adv[i]
        r = np.exp(delta)
        is_clipped[i] = (A > 0 and delta > np.log1p(clip_high)) or (A < 0 and delta < np.log1p(-clip_low))
        bound = 1 + clip_high if A > 0 else 1 - clip_low
        loss -= weight[i] * (bound * A if is_clipped[i] else r * A)
        clipped += weight[i] * is_clipped[i]
        grad[i] = 0.0 if is_clipped[i] else -r * A
        if ref is not None:
            q = float(ref[i]) - logp[i]
            kl += weight[i] * (np.expm1(q) - q)
            grad[i] -= kl_coef * np.expm1(q)
        grad[i] *= weight[i]
    return Policy(loss + kl_coef * kl, loss, kl, clipped, grad, weight, is_clipped)


def grad_norm(arrays, norm_type=2.0):
    flat = [np.asarray(a, np.float64).ravel() for a in arrays if a.size]
    if not flat:
        return 0.0
    if norm_type == 2.0:
        return float(np.sqrt(sum(np.sum(a * a) for a in flat)))
    return float(max(np.max(np.abs(a)) for a in flat))


def clip_factor(norm, max_norm):
    if not np.isfinite(norm):
        return 1.0
    return min(1.0, max_norm / (norm + 1e-6))
