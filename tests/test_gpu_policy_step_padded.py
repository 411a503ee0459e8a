"""A policy step through the final norm on the GPU: hidden states of rows that
take no part may hold anything."""

import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("d", [128, 136])
def test_rows_without_a_token_reach_no_gradient(fs, torch_cuda, d, rms):
    torch = torch_cuda
    from lm_head_exact_gb300 import policy_step as ps
    g = torch.Generator(device="cuda").manual_seed(d)
    n, V, S = 120, 500, 8
    h = torch.randn(n, d, generator=g, device="cuda").bfloat16()
    W = (torch.randn(V, d, generator=g, device="cuda") * 0.1).bfloat16()
    norm = ps.FinalNorm(torch.rand(d, generator=g, device="cuda") + 0.5,
                        None if rms else torch.randn(d, generator=g, device="cuda"), rms=rms)
    temp = torch.full((n,), 0.9, device="cuda")
    temp[3::10] = -1.0                                         # no token is drawn there
    mask = torch.ones(n, dtype=torch.bool, device="cuda")
    mask[5::15] = False
    starts = torch.arange(0, n + 1, n // S, device="cuda")
    off = (temp < 0) | ~mask
    out = []
    for fill in (1.0, float("nan"), float("inf")):
        x = h.clone()
        x[off] = fill
        r = ps.roll_out(x, W, temp, starts, lambda ids: (ids.view(S, -1) % 7).float().mean(1), 1, 2, norm=norm)
        r.mask, r.advantages = mask, torch.linspace(-1, 1, S, device="cuda")
        r.old_logp = r.old_logp - 0.05
        out.append(ps.policy_step(r, W, norm=norm))
    for other in out[1:]:
        for name in ("grad_h", "grad_W", "grad_norm_weight") + (() if rms else ("grad_norm_bias",)):
            a, b = getattr(out[0], name), getattr(other, name)
            assert bool(b.isfinite().all()) and torch.equal(a, b), name
        assert torch.equal(out[0].stats, other.stats)
    assert bool((out[0].grad_h[off] == 0).all()) and bool((out[0].grad_norm_weight != 0).any())
    assert fs.device_error() == 0
