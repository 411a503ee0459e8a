"""The training operators of the LM head, as cases to measure: scoring given tokens (log-probabilities through
the head), the same with its gradients, the clipped policy loss, and clipping by the global gradient norm.

``run`` computes an operator in elementary torch operations, or, with ``own`` set, through the library."""

import math
import random

import torch

own = False

DEV = "cuda"


def listed():
    return [
        # the smallest head of the repository's own tests: latency
        dict(name="score_small", op="score", T=16, d=256, V=4096, bias="none"),
        # one decode step's tokens scored by another model: bound by reading the head once
        dict(name="score_decode", op="score", T=16, d=4096, V=128256, bias="none"),
        # a ragged batch of prompts with some vocabulary entries forbidden
        dict(name="score_masked", op="score", T=517, d=4096, V=151936, bias="shared"),
        # a batch of tokens in a training step of a small model, odd sizes
        dict(name="grad_small", op="grad", T=257, d=520, V=32001, bias="none", keep=True),
        # one micro-batch through an 8B-class head, logits kept for the backward pass
        dict(name="grad_step", op="grad", T=2048, d=4096, V=128256, bias="none", keep=True),
        # a shorter ragged micro-batch, logits formed again in the backward pass to save memory, per-row bias
        dict(name="grad_lean", op="grad", T=773, d=4096, V=65537, bias="rows", keep=False),
        # a handful of short answers
        dict(name="policy_small", op="policy", S=8, L=100, padded=False, adv="seq", mask=False, ref=True, mean="token"),
        # answers padded to one length, with a mask, each answer weighted the same
        dict(name="policy_padded", op="policy", S=64, L=1024, padded=True, adv="seq", mask=True, ref=True, mean="sequence"),
        # a large rollout batch, packed, some tokens (tool output) masked, advantages by token
        dict(name="policy_large", op="policy", S=1024, L=4096, padded=False, adv="token", mask=True, ref=True, mean="token"),
        # a toy model: latency over a dozen small tensors
        dict(name="clip_small", op="clip", layers=2, d=100, kv=25, ffn=272, types="mixed"),
        # one decoder layer's gradients in bf16
        dict(name="clip_layer", op="clip", layers=1, d=4096, kv=1024, ffn=14336, types="bf16"),
        # several layers, 32-bit gradients of the norms beside 16-bit matrices
        dict(name="clip_layers", op="clip", layers=5, d=4096, kv=1024, ffn=14336, types="mixed"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("score", "grad", "policy", "clip"))
    if op in ("score", "grad"):
        while True:
            T, d, V = _log_int(rng, 1, 2048), 8 * _log_int(rng, 8, 512), _log_int(rng, 1000, 152000)
            if T * V <= 2048 * 128256 and d * V <= 4096 * 152000:
                break
        case = dict(op=op, T=T, d=d, V=V, bias=rng.choice(("none", "shared", "rows" if T <= 1024 else "shared")))
        return dict(case, keep=rng.random() < 0.6) if op == "grad" else case
    if op == "policy":
        return dict(op=op, S=_log_int(rng, 2, 1024), L=_log_int(rng, 8, 4096), padded=rng.random() < 0.4,
                    adv=rng.choice(("seq", "token")), mask=rng.random() < 0.6, ref=rng.random() < 0.7,
                    mean=rng.choice(("token", "sequence")))
    d = _log_int(rng, 64, 4096)
    return dict(op=op, layers=_log_int(rng, 1, 5), d=d, kv=max(1, d // rng.choice((1, 4, 8))),
                ffn=_log_int(rng, d, 3 * d), types=rng.choice(("mixed", "bf16", "fp32" if d < 2048 else "fp16")))


# ------------------------------------------------------------------ inputs
def _lengths(case):
    """Lengths of the sequences: from none to twice the mean, fixed by the case."""
    rng = random.Random(case["S"] * 1000003 + case["L"])
    if case["padded"]:
        return [case["L"]] * case["S"]
    return [rng.randint(0, 2 * case["L"]) for _ in range(case["S"] - 1)] + [case["L"]]


def _shapes(case):
    """The parameters of `layers` decoder layers, as (elements, whether a vector)."""
    d, kv, ffn = case["d"], case["kv"], case["ffn"]
    layer = [(d * (d + 2 * kv), False), (d * d, False), (2 * ffn * d, False), (ffn * d, False), (d, True), (d, True)]
    return layer * case["layers"]


def _rand(gen, *shape):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32)


def _prepare_head(case, gen):
    T, d, V = case["T"], case["d"], case["V"]
    h = _rand(gen, T, d).bfloat16()
    W = torch.empty((V, d), dtype=torch.bfloat16, device=DEV)
    for i in range(0, V, 32768):
        W[i:i + 32768] = _rand(gen, min(32768, V - i), d) * (1.5 / math.sqrt(d))
    ids = torch.randint(0, V, (T,), generator=gen, device=DEV)
    if T > 8:
        ids[torch.rand(T, generator=gen, device=DEV) < 0.05] = -1         # padding
    temp = 0.6 + 0.6 * torch.rand(T, generator=gen, device=DEV)
    bias = None
    if case["bias"] == "shared":                                          # some entries forbidden
        bias = torch.where(torch.rand(V, generator=gen, device=DEV) < 0.1, -math.inf, 0.0)
    elif case["bias"] == "rows":                                          # a dense adjustment for each row
        bias = 0.5 * _rand(gen, T, V)
    if bias is not None:                                                  # what was sampled was not forbidden
        if bias.dim() == 1:
            bias[ids.clamp(min=0)] = 0.0
    s = dict(op=case["op"], h=h, W=W, ids=ids, temp=temp, bias=bias)
    if case["op"] == "grad":
        g = _rand(gen, T) / T
        g[torch.rand(T, generator=gen, device=DEV) < 0.1] = 0.0           # clipped tokens
        s.update(g=g, keep=case["keep"])
    return s


def _prepare_policy(case, gen):
    S = case["S"]
    lengths = _lengths(case)
    N = sum(lengths)
    shape = (S, case["L"]) if case["padded"] else (N,)
    starts = torch.tensor([0] + lengths, dtype=torch.int64).cumsum(0).to(DEV)
    old = -torch.log1p(_rand(gen, *shape).abs() * 4.0)
    logp = old + 0.15 * _rand(gen, *shape) + 0.02
    ref = logp + 0.1 * _rand(gen, *shape) if case["ref"] else None
    adv = _rand(gen, S) + 0.25 if case["adv"] == "seq" else _rand(gen, *shape) + 0.25
    mask = None
    if case["mask"]:
        mask = torch.rand(shape, generator=gen, device=DEV) < 0.8
        if case["padded"]:                                                # answers end before the padding
            ends = torch.randint(0, case["L"] + 1, (S, 1), generator=gen, device=DEV)
            mask &= torch.arange(case["L"], device=DEV)[None] < ends
            logp = torch.where(mask, logp, math.nan)                      # nobody wrote anything there
    return dict(op="policy", logp=logp, old=old, ref=ref, adv=adv, mask=mask, mean=case["mean"],
                starts=None if case["padded"] else starts, clip_low=0.2, clip_high=0.28, kl=0.05 if case["ref"] else 0.0)


def _prepare_clip(case, gen):
    matrix = torch.float32 if case["types"] == "fp32" else torch.float16 if case["types"] == "fp16" else torch.bfloat16
    vector = torch.float32 if case["types"] == "mixed" else matrix
    shapes = _shapes(case)
    flat, views, outs = {}, [], []
    for vec in (False, True):
        n = sum(k for k, v in shapes if v == vec)
        buf = torch.empty(n, dtype=vector if vec else matrix, device=DEV)
        for i in range(0, n, 1 << 27):
            buf[i:i + (1 << 27)] = _rand(gen, min(1 << 27, n - i)) * 1e-2
        flat[vec] = (buf, torch.empty_like(buf))
    at = {False: 0, True: 0}
    for k, vec in shapes:
        g, o = flat[vec]
        views.append(g[at[vec]:at[vec] + k])
        outs.append(o[at[vec]:at[vec] + k])
        at[vec] += k
    return dict(op="clip", grads=views, outs=outs, flat=flat, max_norm=1.0)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    return {"policy": _prepare_policy, "clip": _prepare_clip}.get(case["op"], _prepare_head)(case, gen)


# ------------------------------------------------------------------ plain forms
def _plain_logits(s):
    x = s["h"].float() @ s["W"].float().t()
    if s["bias"] is not None:
        x += s["bias"]
    x /= s["temp"][:, None]
    return x


def _plain_score(s, x):
    lse = x.amax(1)
    lse = lse + torch.log(torch.exp(x - lse[:, None]).sum(1))
    rows = torch.arange(x.shape[0], device=x.device)
    scored = s["ids"] >= 0
    return torch.where(scored, x[rows, s["ids"].clamp(min=0)] - lse, 0.0), lse


def _plain_grad(s):
    x = _plain_logits(s)
    logp, lse = _plain_score(s, x)
    scored = (s["ids"] >= 0) & (s["g"] != 0)
    c = torch.where(scored, s["g"] / s["temp"], 0.0)
    ds = x.sub_(lse[:, None]).exp_().mul_(-c[:, None])
    rows = torch.arange(x.shape[0], device=x.device)
    ds[rows, s["ids"].clamp(min=0)] += c
    grad_h = (ds @ s["W"].float()).bfloat16()
    grad_W = (ds.t() @ s["h"].float()).bfloat16()
    return logp, lse, grad_h, grad_W


def _by_token(s, v):
    """A value of each sequence as one of each token."""
    if s["starts"] is None:
        return v[:, None].expand(s["logp"].shape)
    return torch.repeat_interleave(v, s["starts"].diff(), output_size=s["logp"].numel())


def _by_sequence(s, v):
    """Sums over the tokens of each sequence."""
    if s["starts"] is None:
        return v.sum(1)
    c = torch.cat((v.new_zeros(1), v.cumsum(0)))[s["starts"]]
    return c.diff()


def _plain_policy(s):
    on = s["mask"] if s["mask"] is not None else torch.ones_like(s["logp"], dtype=torch.bool)
    adv = s["adv"] if s["adv"].shape == s["logp"].shape else _by_token(s, s["adv"])
    if s["mean"] == "token":
        w = on / on.sum().clamp(min=1)
    else:
        n = _by_sequence(s, on.to(torch.int64))
        w = on / (_by_token(s, n) * (n > 0).sum()).clamp(min=1)
    d = s["logp"].double() - s["old"].double()                           # next to the borders
    ratio = torch.exp(s["logp"] - s["old"])
    clipped = torch.where(adv > 0, d > math.log1p(s["clip_high"]), (adv < 0) & (d < math.log1p(-s["clip_low"])))
    surrogate = torch.where(clipped, torch.where(adv > 0, 1 + s["clip_high"], 1 - s["clip_low"]), ratio) * adv
    grad = torch.where(clipped, 0.0, -ratio * adv)
    w64 = torch.where(on, w, 0.0).double()
    take = lambda v: torch.where(on, v.double() * w64, 0.0).sum()  # noqa: E731  long sums
    policy, kl = take(-surrogate), torch.zeros((), dtype=torch.float64, device=w.device)
    if s["ref"] is not None:
        q = s["ref"].double() - s["logp"].double()                       # e^q - 1 - q of small q
        kl = take(torch.expm1(q) - q)
        grad = grad - s["kl"] * torch.expm1(q).float()
    share = take(clipped)
    return torch.stack((policy + s["kl"] * kl, policy, kl, share)).float(), torch.where(on, grad * w, 0.0)


def _plain_clip(s):
    buffers = [b for b, _ in s["flat"].values()]
    total = sum(b.float().square().sum(dtype=torch.float64) for b in buffers)
    norm = total.sqrt()
    coef = (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0).float()
    return [norm.float()] + [(b.float() * coef).to(b.dtype) for b in buffers]


def run(s):
    if own:
        return _run_own(s)
    if s["op"] == "score":
        return _plain_score(s, _plain_logits(s))
    return {"grad": _plain_grad, "policy": _plain_policy, "clip": _plain_clip}[s["op"]](s)


# ------------------------------------------------------------------ through the library
def _run_own(s):
    from lm_head_exact_gb300 import binding as fs
    if s["op"] == "score":
        return fs.token_logprobs(s["h"], s["W"], s["ids"], s["temp"], bias=s["bias"])
    if s["op"] == "grad":
        kept = fs.logprob_buffer(s["h"].shape[0], s["W"].shape[0], device=s["h"].device) if s["keep"] else None
        logp, lse = fs.token_logprobs(s["h"], s["W"], s["ids"], s["temp"], bias=s["bias"], kept=kept)
        grad_h, grad_W = fs.token_logprobs_backward(s["h"], s["W"], s["ids"], s["temp"], logp, lse, s["g"],
                                                    bias=s["bias"], kept=kept)
        return logp, lse, grad_h, grad_W
    if s["op"] == "policy":
        return fs.policy_loss(s["logp"], s["old"], s["adv"], seq_starts=s["starts"], mask=s["mask"], ref_logp=s["ref"],
                              clip_low=s["clip_low"], clip_high=s["clip_high"], kl_coef=s["kl"], mean=s["mean"])
    norm = fs.clip_grad_norm(s["grads"], s["max_norm"], out=s["outs"])
    return [norm] + [o for _, o in s["flat"].values()]


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op = case["op"]
    if op in ("score", "grad"):
        T, d, V = case["T"], case["d"], case["V"]
        bias = {"none": 0, "shared": 4 * V, "rows": 4 * T * V}[case["bias"]]
        bytes_ = 2 * V * d + 2 * T * d + bias + 20 * T
        if op == "score":
            return dict(bytes=bytes_, flops=2 * T * V * d)
        return dict(bytes=bytes_ + 2 * V * d + 2 * T * d + 4 * T, flops=6 * T * V * d)
    if op == "policy":
        N, S = sum(_lengths(case)), case["S"]
        token = 8 + 4 + (4 if case["ref"] else 0) + (4 if case["adv"] == "token" else 0) + (1 if case["mask"] else 0)
        return dict(bytes=N * token + S * (12 if case["adv"] == "seq" else 8), flops=20 * N)
    width = {"bf16": (2, 2), "fp16": (2, 2), "fp32": (4, 4), "mixed": (2, 4)}[case["types"]]
    elements = [sum(k for k, v in _shapes(case) if v == vec) for vec in (False, True)]
    return dict(bytes=sum(2 * w * n for w, n in zip(width, elements)), flops=3 * sum(elements))


# ------------------------------------------------------------------ by definition, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    f8 = torch.float64
    if case["op"] in ("score", "grad"):
        W = s["W"].to(f8)
        logp, lse, grad_h, grad_W = [], [], [], torch.zeros(W.shape if case["op"] == "grad" else (0,), dtype=f8, device=DEV)
        for i in range(0, case["T"], 512):
            at = slice(i, i + 512)
            h, ids, temp = s["h"][at].to(f8), s["ids"][at], s["temp"][at].to(f8)
            x = h.matmul(W.T)
            if s["bias"] is not None:
                x = x + (s["bias"][at] if s["bias"].dim() == 2 else s["bias"]).to(f8)
            x = x / temp.unsqueeze(1)
            z = x.logsumexp(1)
            real = ids.ge(0)
            picked = x.gather(1, ids.clamp(min=0).unsqueeze(1)).squeeze(1) - z
            logp.append(torch.where(real, picked, torch.zeros_like(picked)))
            lse.append(z)
            if case["op"] == "grad":
                delta = torch.zeros_like(x).scatter_(1, ids.clamp(min=0).unsqueeze(1), 1.0) - x.softmax(1)
                delta *= (s["g"][at].to(f8) * real / temp).unsqueeze(1)
                grad_h.append(delta.matmul(W))
                grad_W += delta.T.matmul(h)
        out = torch.cat(logp), torch.cat(lse)
        return out if case["op"] == "score" else out + (torch.cat(grad_h), grad_W)
    if case["op"] == "policy":
        lengths = torch.tensor(_lengths(case), device=DEV)
        seq = torch.arange(case["S"], device=DEV).repeat_interleave(lengths)
        flat = lambda v: v.reshape(-1).to(f8)  # noqa: E731
        on = torch.ones_like(seq, dtype=torch.bool) if s["mask"] is None else s["mask"].reshape(-1)
        used = on.nonzero().squeeze(1)
        seq_u = seq[used]
        lp, old = flat(s["logp"])[used], flat(s["old"])[used]
        A = flat(s["adv"])[seq_u] if case["adv"] == "seq" else flat(s["adv"])[used]
        count = torch.bincount(seq_u, minlength=case["S"]).to(f8)
        weight = 1.0 / count[seq_u] / (count > 0).sum() if case["mean"] == "sequence" else torch.full_like(lp, 1.0 / max(1, used.numel()))
        r = (lp - old).exp()
        bounded = r.clamp(1 - s["clip_low"], 1 + s["clip_high"])
        free = r * A <= bounded * A
        term = -torch.minimum(r * A, bounded * A)
        g = torch.where(free, -r * A, torch.zeros_like(r))
        kl = torch.zeros_like(r)
        if s["ref"] is not None:
            q = flat(s["ref"])[used] - lp
            kl = q.expm1() - q
            g = g - s["kl"] * q.expm1()
        policy, kl = (weight * term).sum(), (weight * kl).sum()
        stats = torch.stack((policy + s["kl"] * kl, policy, kl, (weight * ~free).sum()))
        grad = torch.zeros(seq.shape, dtype=f8, device=DEV)
        grad[used] = weight * g
        return stats, grad.reshape(s["logp"].shape)
    bufs = [b.to(f8) for b, _ in s["flat"].values()]
    norm = torch.linalg.vector_norm(torch.stack([torch.linalg.vector_norm(b) for b in bufs]))
    scale = min(1.0, s["max_norm"] / (float(norm) + 1e-6))
    return [norm] + [b * scale for b in bufs]
