"""The training operators as they are used together: one policy step against
PyTorch's autograd on the same numbers, and a head that learns."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu


def _rollout(torch, ps, n=120, d=128, V=1500, S=8):
    g = torch.Generator(device="cuda").manual_seed(5)
    h = torch.randn(n, d, generator=g, device="cuda").bfloat16()
    W = (torch.randn(V, d, generator=g, device="cuda") * 0.1).bfloat16()
    temp = torch.full((n,), 0.9, device="cuda")
    starts = torch.arange(0, n + 1, n // S, device="cuda")
    r = ps.roll_out(h, W, temp, starts, lambda ids: (ids.view(S, -1) % 7).float().mean(1), 1234, 3)
    return r, W


@pytest.mark.parametrize("keep", [True, False])
def test_policy_step_matches_autograd(fs, torch_cuda, keep):
    torch = torch_cuda
    from lm_head_exact_gb300 import policy_step as ps
    r, W = _rollout(torch, ps)
    moved = (W.float() * 1.05).bfloat16()                     # the policy has moved since the rollout
    out = ps.policy_step(r, moved, ref_logp=r.old_logp, kl_coef=0.1, max_norm=1e9, keep_logits=keep)
    h64, W64 = r.h.double().requires_grad_(), moved.double().requires_grad_()
    logp = torch.log_softmax(h64 @ W64.T / r.temp.double()[:, None], 1).gather(1, r.ids[:, None]).squeeze(1)
    ratio = (logp - r.old_logp.double()).exp()
    A = r.advantages.double().repeat_interleave(120 // 8)
    q = r.old_logp.double() - logp
    loss = (-torch.minimum(ratio * A, ratio.clamp(0.8, 1.28) * A) + 0.1 * (q.exp() - 1 - q)).mean()
    loss.backward()
    # scores: fp32 sums of 128 products; gradients: ds and the result each rounded to bf16 (2^-8), and ds
    # besides moved by the scores' error (2^-12 covers both scores' 1e-4)
    assert abs(float(out.stats[0]) - float(loss.detach())) < 1e-4
    for got, want in ((out.grad_h, h64.grad), (out.grad_W, W64.grad)):
        err = (got.double() - want).norm() / want.norm()
        assert float(err) < 2 * 2.0 ** -8 + 2.0 ** -12
    want = float(torch.cat([out.grad_h.flatten(), out.grad_W.flatten()]).double().norm())
    assert abs(float(out.grad_norm) - want) < 1e-5 * want
    clipped = ps.policy_step(r, moved, ref_logp=r.old_logp, kl_coef=0.1, max_norm=0.25 * want, keep_logits=keep)
    total = float(torch.cat([clipped.grad_h.flatten(), clipped.grad_W.flatten()]).double().norm())
    assert abs(total / (0.25 * want) - 1) < 2.0 ** -8


def test_a_head_learns(fs, torch_cuda):
    from lm_head_exact_gb300 import policy_step as ps
    rewards = ps.train_toy(steps=20)
    assert np.isfinite(rewards).all()
    assert np.mean(rewards[-3:]) > np.mean(rewards[:2]) + 0.1


def test_policy_step_under_the_samplers_bias(fs, torch_cuda):
    """An unchanged policy has ratio 1 everywhere: the loss is minus the mean
    advantage, and forbidden tokens have no gradient."""
    torch = torch_cuda
    from lm_head_exact_gb300 import policy_step as ps
    g = torch.Generator(device="cuda").manual_seed(6)
    h = torch.randn(64, 128, generator=g, device="cuda").bfloat16()
    W = torch.randn(900, 128, generator=g, device="cuda").bfloat16()
    bias = torch.where(torch.arange(900, device="cuda") % 3 == 0, -float("inf"), 0.0)
    starts = torch.arange(0, 65, 8, device="cuda")
    r = ps.roll_out(h, W, torch.ones(64, device="cuda"), starts, lambda ids: (ids.view(8, 8) % 5).float().mean(1), 7, 8,
                    bias=bias)
    assert bool((r.ids % 3 != 0).all())
    out = ps.policy_step(r, W)
    assert torch.equal(out.logp, r.old_logp) or float((out.logp - r.old_logp).abs().max()) < 1e-5
    assert abs(float(out.stats[0]) + float(r.advantages.mean())) < 1e-4
    assert not bool(out.grad_W[::3].any()) and bool(out.grad_W[1::3].any())


def test_policy_step_with_rows_that_have_no_token(fs, torch_cuda):
    """Rows that the sampler left out: the step is that of the other rows."""
    torch = torch_cuda
    from lm_head_exact_gb300 import policy_step as ps
    g = torch.Generator(device="cuda").manual_seed(9)
    h = torch.randn(40, 64, generator=g, device="cuda").bfloat16()
    W = torch.randn(300, 64, generator=g, device="cuda").bfloat16()
    temp = torch.ones(40, device="cuda")
    temp[5:9] = -1.0
    starts = torch.tensor([0, 10, 40], device="cuda")
    r = ps.roll_out(h, W, temp, starts, lambda ids: torch.stack([ids[:10].float().mean(), ids[10:].float().mean()]), 1, 2)
    assert bool((r.ids[5:9] == -1).all())
    out = ps.policy_step(r, W)
    live = torch.cat([torch.arange(5), torch.arange(9, 40)]).cuda()
    alone = ps.policy_step(ps.Rollout(h[live], r.ids[live], temp[live], torch.tensor([0, 6, 36], device="cuda"),
                                      r.advantages, r.old_logp[live]), W)
    # the same 36 tokens, added in another order
    assert torch.allclose(out.stats, alone.stats, rtol=1e-5, atol=1e-6)
    assert torch.allclose(out.grad_h[live].float(), alone.grad_h.float(), rtol=2.0 ** -7, atol=1e-4)
    assert not bool(out.grad_h[5:9].any())
