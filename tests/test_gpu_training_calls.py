"""Calls of the training operators from several host threads, on given streams
and after failures."""

import threading

import pytest

pytestmark = pytest.mark.gpu


def _in_a_thread(work):
    """What work() returns on a new host thread; its exception is raised here."""
    out = []

    def body():
        try:
            out.append((work(), None))
        except Exception as e:                             # noqa: BLE001  (raised by the test's thread)
            out.append((None, e))

    t = threading.Thread(target=body)
    t.start()
    t.join()
    if out[0][1] is not None:
        raise out[0][1]
    return out[0][0]


@pytest.mark.parametrize("what", ["scores", "gradients", "sample"])
def test_first_call_of_a_host_thread(fs, torch_cuda, what):
    """A thread that has made no CUDA call before: none of its own has bound
    the device's context to it."""
    torch = torch_cuda
    h, W = torch.ones(20, 64, device="cuda").bfloat16(), torch.ones(300, 64, device="cuda").bfloat16()
    ids, temp = torch.arange(20, device="cuda"), torch.ones(20, device="cuda")
    logp, lse = fs.token_logprobs(h, W, ids, temp)
    out = {"scores": (torch.empty_like(temp), torch.empty_like(temp)),
           "gradients": (torch.empty_like(h), torch.empty_like(W)),
           "sample": (torch.empty_like(ids), torch.empty_like(temp))}[what]
    call = {"scores": lambda: fs.token_logprobs(h, W, ids, temp, out=out),
            "gradients": lambda: fs.token_logprobs_backward(h, W, ids, temp, logp, lse, temp, out=out),
            "sample": lambda: fs.sample(h, W, temp, 1, 2, out=out)}[what]
    want = [t.clone() for t in call()]
    torch.cuda.synchronize()
    for t in out:
        t.zero_()
    torch.cuda.synchronize()
    _in_a_thread(call)
    torch.cuda.synchronize()
    for a, b in zip(want, out):
        assert torch.equal(a, b)
