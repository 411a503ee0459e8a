"""A policy step through the final norm whose batch has rows without a token:
their hidden states may hold anything."""

import pytest

torch = pytest.importorskip("torch")

from lm_head_exact_gb300 import policy_step as ps  # noqa: E402
from test_policy_step import Plain  # noqa: E402


class WithNorm(Plain):
    """The norm in elementary operations, by its formulas; scores whose rows
    without a gradient may hold anything, as the library's do."""

    def layer_norm(self, x, weight, bias, eps, rms):
        mean = torch.zeros(len(x)) if rms else x.mean(1)
        rstd = ((x - mean[:, None]) ** 2).mean(1).add(eps).rsqrt()
        y = (x - mean[:, None]) * rstd[:, None]
        y = y if weight is None else y * weight
        return y if bias is None else y + bias, None if rms else mean, rstd

    def layer_norm_backward(self, grad, x, weight, mean, rstd, need_weight=True, need_bias=True, out=None):
        assert out is grad
        self.calls.append(("layer_norm_backward", need_weight))
        xh = (x if mean is None else x - mean[:, None]) * rstd[:, None]
        a = grad if weight is None else grad * weight
        gw, gb = (grad * xh).sum(0) if need_weight else None, grad.sum(0) if need_bias else None
        m_a = 0.0 if mean is None else a.mean(1, keepdim=True)
        out.copy_(rstd[:, None] * (a - m_a - xh * (a * xh).mean(1, keepdim=True)))
        return out, gw, gb

    def token_logprobs_backward(self, h, W, ids, temp, logp, lse, g, bias=None, kept=None):
        live = (ids >= 0) & (ids < W.shape[0]) & (temp >= 0) & (g != 0)
        grad_h, grad_W = super().token_logprobs_backward(torch.where(live[:, None], h, 0.0), W, ids, temp, logp, lse, g, bias)
        return torch.where(live[:, None], grad_h, 0.0), grad_W


def _step(monkeypatch, h, norm, mask=None, holes=(), **how):
    g = torch.Generator().manual_seed(1)
    W, ids = torch.randn(30, h.shape[1], generator=g), torch.randint(0, 30, (len(h),), generator=g)
    ids[list(holes)] = -1
    plain = WithNorm(ids)
    monkeypatch.setattr(ps, "fs", plain)
    r = ps.Rollout(h=h, ids=ids, temp=torch.full((len(h),), 0.8), seq_starts=torch.tensor([0, 4, len(h)]),
                   old_logp=torch.full((len(h),), -3.0), advantages=torch.tensor([1.0, -0.5]), mask=mask)
    return ps.policy_step(r, W, norm=norm, **how), plain


@pytest.mark.parametrize("eps", [1e-5, 0.0])
@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("fill", [float("nan"), float("inf"), 0.0, 7.0])
def test_rows_without_a_token_reach_no_gradient_of_the_norm(monkeypatch, fill, rms, eps):
    g = torch.Generator().manual_seed(0)
    h = torch.randn(12, 16, generator=g) * 3 + 1
    norm = ps.FinalNorm(torch.rand(16, generator=g) + 0.5, None if rms else torch.randn(16, generator=g), eps, rms)
    mask = torch.ones(12, dtype=torch.bool)
    mask[[5, 9]] = False
    want, _ = _step(monkeypatch, h, norm, mask, holes=(2, 11))
    h = h.clone()
    h[[2, 5, 9, 11]] = fill
    got, _ = _step(monkeypatch, h, norm, mask, holes=(2, 11))
    for name in ("grad_h", "grad_W", "grad_norm_weight", "grad_norm_bias"):
        a, b = getattr(want, name), getattr(got, name)
        assert (a is None) == (b is None) == (rms and name == "grad_norm_bias")
        if a is not None:
            assert bool(b.isfinite().all()) and torch.equal(a, b)
    assert bool((got.grad_h[[2, 5, 9, 11]] == 0).all())


def test_a_norm_without_weight_has_no_gradient_of_one(monkeypatch):
    h = torch.randn(12, 16, generator=torch.Generator().manual_seed(0))
    got, plain = _step(monkeypatch, h, ps.FinalNorm(None), max_norm=1e-3)
    assert got.grad_norm_weight is None and got.grad_norm_bias is None
    assert ("layer_norm_backward", False) in plain.calls
    assert len(plain.calls[-1][1]) == 2                        # what is clipped: grad_h and grad_W
    total = torch.cat((got.grad_h.flatten(), got.grad_W.flatten()))
    assert abs(float(total.norm()) - 1e-3) < 1e-5
