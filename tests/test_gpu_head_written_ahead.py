"""An LM head that one of the norm's or the 8-bit product's calls writes, read by
a sampler two calls on.  The sampler between them lets the next one start, and
read its head, before its own wait, so the call that writes must have ended by
then.  (The call right before a sampler must not write its head: see
fs_set_launch_overlap.)"""

import pytest

pytestmark = pytest.mark.gpu

V, D = 64000, 1024


def _writers(fs, torch, k):
    """Calls that write a [V, D] bf16 matrix: by name, with inputs of their own."""
    g = torch.Generator(device="cuda").manual_seed(40 + k)
    x = torch.randn(V, D, generator=g, device="cuda").bfloat16()
    weight = torch.rand(D, generator=g, device="cuda") + 0.5
    mean, rstd = fs.layer_norm(x, weight)[1:]
    a8 = fs.quantize_fp8(torch.randn(V, 256, generator=g, device="cuda").bfloat16())
    b8 = fs.quantize_fp8(torch.randn(D, 256, generator=g, device="cuda").bfloat16() * 0.06, block_rows=128)
    odd = torch.randn(V * D + 1, generator=g, device="cuda").bfloat16()[1:].view(V, D)
    return {"norm": lambda out: fs.layer_norm(x, weight, out=out),
            "norm off boundaries": lambda out: fs.layer_norm(odd, weight, out=out),
            "gradient": lambda out: fs.layer_norm_backward(x, x, weight, mean, rstd, out=out),
            "gradient alone": lambda out: fs.layer_norm_backward(x, x, weight, mean, rstd, need_weight=False, need_bias=False,
                                                                 out=out),
            "product": lambda out: fs.fp8_matmul(*a8, *b8, out=out)}


@pytest.mark.parametrize("B", [1, 16, 100, 300])
@pytest.mark.parametrize("kind", ["norm", "norm off boundaries", "gradient", "gradient alone", "product"])
def test_a_head_written_two_calls_ahead(fs, torch_cuda, kind, B):
    torch = torch_cuda
    g = torch.Generator(device="cuda").manual_seed(B)
    h = torch.randn(B, D, generator=g, device="cuda").bfloat16() * 0.1
    other = torch.randn(500, D, generator=g, device="cuda").bfloat16()
    temp = torch.ones(B, device="cuda")
    calls = [_writers(fs, torch, k)[kind] for k in range(2)]
    W = torch.empty(V * D + 1, dtype=torch.bfloat16, device="cuda")
    W = (W[1:] if kind == "norm off boundaries" else W[:-1]).view(V, D)
    # the sampler's head begins on a 16-byte boundary: where the call's cannot, it is a row further in
    head = W if W.data_ptr() % 16 == 0 else W.view(-1)[7:7 + (V - 1) * D].view(V - 1, D)
    alone = []
    for call in calls:
        call(W)
        torch.cuda.synchronize()
        alone.append(fs.sample(h, head, temp, 11, 3))
        torch.cuda.synchronize()
    got = []
    for turn in range(8):
        calls[turn % 2](W)
        fs.sample(h, other, temp, 1, 2)
        got.append(fs.sample(h, head, temp, 11, 3))
    torch.cuda.synchronize()
    for turn, (ids, mx) in enumerate(got):
        assert torch.equal(ids, alone[turn % 2][0]) and torch.equal(mx, alone[turn % 2][1])
    assert not torch.equal(alone[0][1], alone[1][1]) and fs.device_error() == 0
