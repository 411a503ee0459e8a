"""What the training operators refuse, on the host before any kernel runs."""

import ctypes

import pytest

Z = ctypes.c_void_p(0)


def _last(lib):
    return lib.fs_last_error().decode()


@pytest.fixture(scope="module")
def lib(built_library):
    from lm_head_exact_gb300 import binding
    return binding.library()


def test_scores_refuse(lib):
    def call(n, d, V):
        return lib.fs_token_logprobs(Z, Z, n, d, V, Z, Z, Z, 0, Z, Z, Z, Z, 0, Z)

    def back(n, d, V):
        return lib.fs_token_logprobs_backward(Z, Z, n, d, V, Z, Z, Z, 0, Z, Z, Z, Z, Z, Z, Z, 0, Z)

    for f in (call, back):
        assert f(-1, 64, 10) == 1 and "B >= 0" in _last(lib)
        assert f(4, 0, 10) == 1
        assert f(4, 12, 10) == 2 and "multiple of 8" in _last(lib)
        assert f(4, 64, 1 << 31) == 2
        assert f(4, 64, (1 << 31) - 1023) == 2 and f((1 << 31) - 1023, 64, 10) == 2 and "n and V" in _last(lib)
        assert f(4, 65544, 10) == 2
        assert f(4, 64, 10) == 1 and "h is NULL" in _last(lib)
        assert f(0, 64, 10) == 0
    assert lib.fs_logprob_buffer_elems(3, 65) == 3 * 128
    assert lib.fs_logprob_buffer_elems(0, 65) == 0 and lib.fs_logprob_buffer_elems(3, 0) == 0
    assert lib.fs_token_logprobs_workspace_bytes(0, 64, 10) == 0
    assert lib.fs_token_logprobs_workspace_bytes(5, 64, 10) >= 5 * 12
    assert lib.fs_token_logprobs_backward_workspace_bytes(5, 64, 10) >= 5 * (4 + 128 + 128 + 256)
    # a large batch takes its vocabulary in pieces: ds does not grow without bound
    assert lib.fs_token_logprobs_backward_workspace_bytes(1 << 17, 64, 1 << 20) < 8 << 30


def test_policy_refuses(lib):
    def call(S=2, N=8, low=0.2, high=0.2, kl=0.0, mean=0, per_seq=1):
        return lib.fs_policy_loss(Z, Z, Z, Z, per_seq, Z, Z, S, N, low, high, kl, mean, Z, Z, Z, 0, Z)

    assert call(N=-1) == 1 and call(S=-1) == 1
    assert call(S=0) == 1 and "n_seqs" in _last(lib)
    assert call(S=3) == 1 and "multiple" in _last(lib)
    for low in (-0.1, 1.0, float("nan")):
        assert call(low=low) == 1 and "clip_low" in _last(lib)
    for high in (-0.1, float("inf"), float("nan")):
        assert call(high=high) == 1 and "clip_high" in _last(lib)
    assert call(kl=float("nan")) == 1 and "finite" in _last(lib)
    assert call(kl=0.1) == 1 and "ref_logp" in _last(lib)
    assert call(mean=3) == 1 and call(mean=-1) == 1
    assert call(per_seq=2) == 1
    assert call(N=1 << 40, S=1) == 2
    assert call() == 1 and "stats is NULL" in _last(lib)
    assert lib.fs_policy_loss_workspace_bytes(0) == 0 and lib.fs_policy_loss_workspace_bytes(3) >= 12


def test_clip_refuses(lib):
    one = (ctypes.c_void_p * 1)(16)
    n4, neg, far = (ctypes.c_int64 * 1)(4), (ctypes.c_int64 * 1)(-4), (ctypes.c_int64 * 1)(1 << 40)
    f32, odd = (ctypes.c_int * 1)(0), (ctypes.c_int * 1)(3)

    def call(g=one, o=one, s=n4, t=f32, n=1, max_norm=1.0, kind=0):
        return lib.fs_clip_grad_norm(g, o, s, t, n, max_norm, kind, Z, Z)

    assert call(n=-1) == 1
    for m in (-1.0, float("nan")):
        assert call(max_norm=m) == 1 and "max_norm" in _last(lib)
    assert call(kind=2) == 1 and "norm type" in _last(lib)
    assert call(g=None) == 1 and call(s=None) == 1 and call(t=None) == 1
    assert call(s=neg) == 1 and "negative" in _last(lib)
    assert call(s=far) == 2
    assert call(t=odd) == 1 and "type" in _last(lib)
    assert call() == 1 and "norm is NULL" in _last(lib)


def test_binding_refuses_cpu_tensors_and_wrong_shapes(built_library):
    torch = pytest.importorskip("torch")
    from lm_head_exact_gb300 import binding as fs
    h, W = torch.zeros(2, 8, dtype=torch.bfloat16), torch.zeros(4, 8, dtype=torch.bfloat16)
    ids, t, g = torch.zeros(2, dtype=torch.int64), torch.ones(2), torch.ones(2)
    for call in (lambda: fs.token_logprobs(h, W, ids, t),
                 lambda: fs.token_logprobs_backward(h, W, ids, t, t, t, g),
                 lambda: fs.policy_loss(t, t, t), lambda: fs.clip_grad_norm([g], 1.0)):
        with pytest.raises(fs.FlashSampleError, match="CUDA tensor"):
            call()
    with pytest.raises(fs.FlashSampleError, match=r"\[V, d\]"):
        fs.token_logprobs(h, W[:, :4], ids, t)
    with pytest.raises(fs.FlashSampleError, match="bias must be"):
        fs.token_logprobs(h, W, ids, t, bias=torch.zeros(3, 4))
    with pytest.raises(fs.FlashSampleError, match="norm_type"):
        fs.clip_grad_norm([g], 1.0, norm_type=1.0)


@pytest.mark.parametrize("what,grads,outs,sizes,types,max_norm,refused", [
    ("listed twice", [4096, 4096], [4096, 4096], [8, 8], [0, 0], 1.0, True),
    ("listed twice, only measured", [4096, 4096], [4096, 4096], [8, 8], [0, 0], float("inf"), False),
    ("listed twice, written elsewhere", [4096, 4096], [8192, 8224], [8, 8], [0, 0], 1.0, False),
    ("one output for two", [4096, 5000], [8192, 8192], [8, 8], [0, 0], 1.0, True),
    ("one output for two, unscaled", [4096, 5000], [8192, 8192], [8, 8], [0, 0], float("inf"), True),
    ("overlapping views in place", [4096, 4112], [4096, 4112], [8, 8], [0, 1], 1.0, True),
    ("neighbours in place", [4096, 4112], [4096, 4112], [8, 8], [1, 1], 1.0, False),
    ("an output on another gradient", [4096, 8192], [8200, 6000], [8, 8], [0, 0], 1.0, True),
    ("an output on its gradient's rest", [4096], [4100], [8], [0], 1.0, True),
    ("a large one around a small one", [4096, 4200], [4096, 4200], [1000, 2], [0, 2], 1.0, True),
    ("empty ones anywhere", [4096, 4096, 4100], [4096, 4096, 4100], [8, 0, 0], [0, 0, 0], 1.0, False),
])
def test_clip_refuses_memory_that_would_be_scaled_twice(lib, what, grads, outs, sizes, types, max_norm, refused):
    n = len(grads)
    status = lib.fs_clip_grad_norm((ctypes.c_void_p * n)(*grads), (ctypes.c_void_p * n)(*outs),
                                   (ctypes.c_int64 * n)(*sizes), (ctypes.c_int * n)(*types), n, max_norm, 0, Z, Z)
    assert status == 1
    assert ("overlaps" in _last(lib)) == refused and ("norm is NULL" in _last(lib)) != refused
