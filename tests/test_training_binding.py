"""The binding of the training operators, where no kernel runs."""

import pytest

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("which", ["forward", "backward"])
def test_workspace_sizes_are_those_of_the_current_device(monkeypatch, which):
    """A device that holds more pairs of SMs at a time needs more workspace
    for the same sizes than the one asked first."""
    from lm_head_exact_gb300 import binding as fs
    device = [0]

    class Library:
        @staticmethod
        def fs_token_logprobs_workspace_bytes(n, d, V):
            return (1 << 20) + 1000 * device[0]

        fs_token_logprobs_backward_workspace_bytes = fs_token_logprobs_workspace_bytes

        @staticmethod
        def fs_token_logprobs(*args):
            asked.append(args[-2])
            return 0

        fs_token_logprobs_backward = fs_token_logprobs

    asked = []
    monkeypatch.setattr(fs, "library", lambda: Library)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: device[0])
    monkeypatch.setattr(fs, "_arg", lambda t, *a: 16)
    monkeypatch.setattr(fs, "_stream_of", lambda *a: 0)
    h, W = torch.zeros(3, 8, dtype=torch.bfloat16), torch.zeros(77, 8, dtype=torch.bfloat16)
    ids, f = torch.zeros(3, dtype=torch.int64), torch.ones(3)
    for device[0] in (0, 1, 0):
        if which == "forward":
            fs.token_logprobs(h, W, ids, f)
        else:
            fs.token_logprobs_backward(h, W, ids, f, f, f, f)
    fs._forward_bytes.cache_clear()
    fs._backward_bytes.cache_clear()
    assert asked == [1 << 20, (1 << 20) + 1000, 1 << 20]
