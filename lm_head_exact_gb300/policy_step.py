"""One policy-gradient step on tokens that the sampler drew.

The sampler returns exact samples of softmax(logits / T); this is what a
post-training loop does with them next, all through the LM head and without
logits in a framework's graph:

1. the rollout's tokens are scored under the policy that drew them
   (``token_logprobs``: log-probabilities at the sampling temperatures);
2. the present policy scores them again, keeping its logits;
3. ``policy_loss`` gives the clipped loss with its KL term and dloss/dlogp;
4. ``token_logprobs_backward`` turns that into gradients of the hidden states
   and of the LM head.

grad_h goes on into the model's own backward pass
(``hidden.backward(grad_h)`` in PyTorch), and ``clip_grad_norm`` follows it,
over the gradients of all parameters: grad_W and the body's, not grad_h, which
is the gradient of activations.  Here, where the body is a fixed set of hidden
states, the head is all there is to update and to clip.

With a ``FinalNorm``, the hidden states are those ahead of the model's last norm:
they are normed for sampling and scoring, grad_h is the gradient ahead of the
norm, and the norm's own gradients come with it (parameters, to clip with
grad_W).

Usage: ``python -m lm_head_exact_gb300.policy_step [steps]`` on a GPU.
"""

from dataclasses import dataclass

from . import binding as fs


@dataclass
class FinalNorm:
    """The model's last norm, between its hidden states and the head."""
    weight: object          # [d] bf16 or fp32, or None: a norm without one
    bias: object = None     # [d] of weight's type
    eps: float = 1e-5
    rms: bool = False       # without the mean

    def __call__(self, h):
        """(normed, mean, rstd) of hidden states."""
        return fs.layer_norm(h, self.weight, self.bias, eps=self.eps, rms=self.rms)


@dataclass
class Rollout:
    """Tokens drawn from the policy: packed sequences and what they earned."""
    h: object               # bf16 [N, d] hidden states (ahead of the final norm, where there is one)
    ids: object             # int64 [N] sampled tokens
    temp: object            # fp32 [N] sampling temperatures
    seq_starts: object      # int64 [S + 1]
    advantages: object      # fp32 [S]
    old_logp: object        # fp32 [N] under the policy that drew them
    mask: object = None     # bool [N], False: not trained on
    bias: object = None     # fp32 [N, V] or [V], the sampler's, under which the tokens are scored too


def roll_out(h, W, temp, seq_starts, reward, seed, step, bias=None, norm=None):
    """Sample a token for every hidden state and score it under W (and the
    sampler's ``bias``, for instance -inf at forbidden tokens); ``reward``
    maps the ids to one value per sequence, which become advantages by
    subtracting their mean and dividing by their spread (one sequence alone
    has neither: advantage 0).  ``norm``: the FinalNorm ahead of the head."""
    normed = h if norm is None else norm(h)[0]
    ids, _ = fs.sample(normed, W, temp, seed, step, bias=bias)
    old_logp, _ = fs.token_logprobs(normed, W, ids, temp, bias=bias)
    r = reward(ids)
    spread = r.std() if r.numel() > 1 else 0.0
    advantages = ((r - r.mean()) / (spread + 1e-6)).contiguous()
    return Rollout(h, ids, temp, seq_starts, advantages, old_logp, bias=bias)


@dataclass
class StepResult:
    stats: object           # fp32 [4]: loss, policy term, KL term, share of clipped tokens
    grad_norm: object       # fp32 scalar, the norm that max_norm bounds (before scaling); None without max_norm
    grad_h: object          # bf16 [N, d]
    grad_W: object          # bf16 [V, d]
    logp: object            # fp32 [N]
    grad_norm_weight: object = None   # [d], the final norm's, where there is one and it has a weight
    grad_norm_bias: object = None     # [d], where it has a bias


def policy_step(rollout, W, ref_logp=None, clip_low=0.2, clip_high=0.28, kl_coef=0.0, mean="token", max_norm=None,
                keep_logits=True, norm=None):
    """Loss and gradients of one step on ``rollout`` under the head W.
    ``keep_logits`` spends 4 bytes per token and vocabulary row to form the
    logits once instead of twice.  Rows without a token (the sampler's -1, an
    invalid temperature) take no part, whatever the rollout's mask says, and
    their hidden states may hold anything.

    The gradients are not clipped here: the norm of the model's gradient is
    known after the body's backward pass only (clip_grad_norm over all
    parameters' gradients).  ``max_norm`` is for something else: it bounds the
    norm of grad_h and grad_W (and the final norm's gradients) taken as one
    vector, that is of the step's whole signal into head and body, and scales
    all by one factor.

    ``norm``: the present policy's FinalNorm; grad_h is then the gradient of the
    rollout's hidden states ahead of it."""
    r = rollout
    n, V = r.h.shape[0], W.shape[0]
    h, mu, rstd = (r.h, None, None) if norm is None else norm(r.h)
    kept = fs.logprob_buffer(n, V, device=r.h.device) if keep_logits else None
    logp, lse = fs.token_logprobs(h, W, r.ids, r.temp, bias=r.bias, kept=kept)
    # (unscored rows have logp 0 on both sides: a ratio of 1, and a part in the means)
    scored = (r.ids >= 0) & (r.ids < V) & (r.temp >= 0)
    mask = scored if r.mask is None else r.mask & scored
    stats, grad_logp = fs.policy_loss(logp, r.old_logp, r.advantages, seq_starts=r.seq_starts, mask=mask,
                                      ref_logp=ref_logp, clip_low=clip_low, clip_high=clip_high, kl_coef=kl_coef,
                                      mean=mean, adv_per_seq=True)
    grad_h, grad_W = fs.token_logprobs_backward(h, W, r.ids, r.temp, logp, lse, grad_logp, bias=r.bias, kept=kept)
    grad_weight = grad_bias = None
    if norm is not None:
        # (rows that take no part may hold anything, NaN included, which their gradient of 0 would not keep out)
        rest = ~mask
        x, rstd = r.h.masked_fill(rest[:, None], 0.0), rstd.masked_fill(rest, 0.0)
        mu = None if mu is None else mu.masked_fill(rest, 0.0)
        need = dict(need_bias=norm.bias is not None, **({} if norm.weight is not None else {"need_weight": False}))
        grad_h, grad_weight, grad_bias = fs.layer_norm_backward(grad_h, x, norm.weight, mu, rstd, out=grad_h, **need)
    grads = [g for g in (grad_h, grad_W, grad_weight, grad_bias) if g is not None]
    total = None if max_norm is None else fs.clip_grad_norm(grads, max_norm)
    return StepResult(stats, total, grad_h, grad_W, logp, grad_weight, grad_bias)


def train_toy(steps=20, V=48, d=64, sequences=256, length=4, lr=6.0, seed=1234, device="cuda"):
    """A head learns to emit even ids: the reward of a sequence is its share
    of them.  Returns the mean reward of every step."""
    import torch
    g = torch.Generator(device=device).manual_seed(seed)
    h = torch.randn(sequences * length, d, generator=g, device=device).bfloat16()
    master = torch.randn(V, d, generator=g, device=device) * 0.02
    temp = torch.ones(sequences * length, device=device)
    starts = torch.arange(0, sequences * length + 1, length, device=device)
    first = master.bfloat16()

    def reward(ids):
        return (ids.view(sequences, length) % 2 == 0).float().mean(1)

    rewards = []
    for step in range(steps):
        W = master.bfloat16()
        r = roll_out(h, W, temp, starts, reward, seed, step)
        rewards.append(reward(r.ids).mean())
        ref_logp, _ = fs.token_logprobs(h, first, r.ids, temp)
        for _ in range(2):                                   # two steps on the same tokens: the second may clip
            out = policy_step(r, master.bfloat16(), ref_logp=ref_logp, kl_coef=0.01)
            fs.clip_grad_norm([out.grad_W], 1.0)
            master -= lr * out.grad_W.float()
    return torch.stack(rewards).tolist()


if __name__ == "__main__":
    import sys
    for i, r in enumerate(train_toy(int(sys.argv[1]) if len(sys.argv) > 1 else 20)):
        print(f"step {i}: mean reward {r:.3f}")
