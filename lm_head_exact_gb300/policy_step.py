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

Usage: ``python -m lm_head_exact_gb300.policy_step [steps]`` on a GPU.
"""

from dataclasses import dataclass

from . import binding as fs


@dataclass
class Rollout:
    """Tokens drawn from the policy: packed sequences and what they earned."""
    h: object               # bf16 [N, d] hidden states
    ids: object             # int64 [N] sampled tokens
    temp: object            # fp32 [N] sampling temperatures
    seq_starts: object      # int64 [S + 1]
    advantages: object      # fp32 [S]
    old_logp: object        # fp32 [N] under the policy that drew them
    mask: object = None     # bool [N], False: not trained on
    bias: object = None     # fp32 [N, V] or [V], the sampler's, under which the tokens are scored too


def roll_out(h, W, temp, seq_starts, reward, seed, step, bias=None):
    """Sample a token for every hidden state and score it under W (and the
    sampler's ``bias``, for instance -inf at forbidden tokens); ``reward``
    maps the ids to one value per sequence, which become advantages by
    subtracting their mean and dividing by their spread (one sequence alone
    has neither: advantage 0)."""
    ids, _ = fs.sample(h, W, temp, seed, step, bias=bias)
    old_logp, _ = fs.token_logprobs(h, W, ids, temp, bias=bias)
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


def policy_step(rollout, W, ref_logp=None, clip_low=0.2, clip_high=0.28, kl_coef=0.0, mean="token", max_norm=None,
                keep_logits=True):
    """Loss and gradients of one step on ``rollout`` under the head W.
    ``keep_logits`` spends 4 bytes per token and vocabulary row to form the
    logits once instead of twice.  Rows without a token (the sampler's -1, an
    invalid temperature) take no part, whatever the rollout's mask says.

    The gradients are not clipped here: the norm of the model's gradient is
    known after the body's backward pass only (clip_grad_norm over all
    parameters' gradients).  ``max_norm`` is for something else: it bounds the
    norm of grad_h and grad_W taken as one vector, that is of the step's whole
    signal into head and body, and scales both by one factor."""
    r = rollout
    n, V = r.h.shape[0], W.shape[0]
    kept = fs.logprob_buffer(n, V, device=r.h.device) if keep_logits else None
    logp, lse = fs.token_logprobs(r.h, W, r.ids, r.temp, bias=r.bias, kept=kept)
    # (unscored rows have logp 0 on both sides: a ratio of 1, and a part in the means)
    scored = (r.ids >= 0) & (r.ids < V) & (r.temp >= 0)
    mask = scored if r.mask is None else r.mask & scored
    stats, grad_logp = fs.policy_loss(logp, r.old_logp, r.advantages, seq_starts=r.seq_starts, mask=mask,
                                      ref_logp=ref_logp, clip_low=clip_low, clip_high=clip_high, kl_coef=kl_coef,
                                      mean=mean, adv_per_seq=True)
    grad_h, grad_W = fs.token_logprobs_backward(r.h, W, r.ids, r.temp, logp, lse, grad_logp, bias=r.bias, kept=kept)
    norm = None if max_norm is None else fs.clip_grad_norm([grad_h, grad_W], max_norm)
    return StepResult(stats, norm, grad_h, grad_W, logp)


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
