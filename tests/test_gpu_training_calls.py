"""Calls of the training operators from several host threads, on given streams
and after failures."""

import threading

import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _streams_left_as_new(fs):
    """PyTorch hands its streams out in turn: what these tests leave on them is
    given back."""
    yield
    fs.check(fs.library().fs_workspace_release())


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


def _run_threads(torch, jobs, rounds):
    """Every job `rounds` times on a host thread of its own, all on one stream;
    the results of each, in order."""
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    results = [[] for _ in jobs]
    errors = []
    start = threading.Barrier(len(jobs))

    def work(job, out):
        try:
            with torch.cuda.stream(stream):
                start.wait()
                for _ in range(rounds):
                    out.append(job())
        except Exception as e:                             # noqa: BLE001  (reported by the test's thread)
            errors.append(e)

    threads = [threading.Thread(target=work, args=a) for a in zip(jobs, results)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    torch.cuda.synchronize()
    return results


@pytest.mark.parametrize("what", ["clip", "policy", "scores"])
def test_threads_that_share_a_stream(fs, torch_cuda, what):
    """What a call leaves in the stream's workspace for its next launch is not
    another thread's: every result is the one of the call made alone."""
    torch = torch_cuda
    gen = torch.Generator(device="cuda").manual_seed(11)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    jobs = []
    for k in range(2):
        if what == "clip":
            grads = [rand(3000) * (k + 1), rand(500)]
            jobs.append(lambda g=grads, m=0.5 + 4 * k: (lambda o: [fs.clip_grad_norm(g, m, out=o)] + o)(
                [torch.empty_like(x) for x in g]))
        elif what == "policy":
            old = -rand(6, 300).abs()
            args = old + 0.2 * rand(6, 300), old, rand(6)
            mask = torch.rand(6, 300, generator=gen, device="cuda") < 0.2 + 0.6 * k
            jobs.append(lambda a=args, m=mask, mean=("token", "sequence")[k]: fs.policy_loss(*a, mask=m, mean=mean))
        else:
            h, W = rand(20 + 4 * k, 64).bfloat16(), rand(700, 64).bfloat16()
            ids, temp = torch.arange(h.shape[0], device="cuda"), torch.full((h.shape[0],), 0.7 + k, device="cuda")
            jobs.append(lambda a=(h, W, ids, temp): fs.token_logprobs(*a))
    alone = [job() for job in jobs]
    torch.cuda.synchronize()
    for want, got in zip(alone, _run_threads(torch, jobs, 400)):
        for r in got:
            for a, b in zip(want, r):
                assert torch.equal(a, b)
    assert fs.device_error() == 0


@pytest.mark.parametrize("what", ["topk", "unfused", "host", "growing"])
def test_threads_that_sample_on_one_stream(fs, torch_cuda, what):
    """Staging, logits and candidate lists of one thread's call stay its own;
    a batch that makes the workspace grow leaves the other thread's call
    whole."""
    torch = torch_cuda
    gen = torch.Generator(device="cuda").manual_seed(12)
    jobs, alone = [], []
    rounds = 30 if what == "growing" else 200
    for k in range(2):
        h = torch.randn(2000, 64, generator=gen, device="cuda").bfloat16()
        W = torch.randn(900, 64, generator=gen, device="cuda").bfloat16()
        temp = torch.full((2000,), 0.5 + k, device="cuda")
        n = 12 + 8 * k
        if what == "topk":
            job = lambda i, h=h, W=W, t=temp, n=n: fs.sample_topk(h[:n], W, t[:n], 5, 6, 4)  # noqa: E731
        elif what == "unfused":
            job = lambda i, h=h, W=W, t=temp, n=n: fs.sample_unfused(h[:n], W, t[:n], 5, 6)  # noqa: E731
        elif what == "host":
            hh, th = h[:n].cpu(), temp[:n].cpu()
            job = lambda i, hh=hh, W=W, th=th: [torch.from_numpy(a) for a in fs.sample_host(hh, W, th, 5, 6)]  # noqa: E731
        else:
            job = lambda i, h=h, W=W, t=temp, k=k: (lambda n: fs.sample(h[:n], W, t[:n], 5, 6))(  # noqa: E731
                16 + 60 * i * k)
        jobs.append((lambda f, at: lambda: f(next(at)))(job, iter(range(rounds))))
        alone.append([job(i) for i in range(rounds if what == "growing" else 1)])
    torch.cuda.synchronize()
    for want, got in zip(alone, _run_threads(torch, jobs, rounds)):
        assert len(got) == rounds
        for i, r in enumerate(got):
            for a, b in zip(want[i % len(want)], r):
                assert torch.equal(a, b)
    assert fs.device_error() == 0


def test_the_per_thread_stream_is_each_threads_own(fs, torch_cuda):
    """One handle, two streams: calls that run at the same time share neither
    counts nor tickets."""
    torch = torch_cuda
    per_thread = torch.cuda.ExternalStream(2)              # cudaStreamPerThread
    gen = torch.Generator(device="cuda").manual_seed(13)
    rounds, S, L = 100, 64, 500
    cases, outs, alone = [], [], []
    for k in range(2):
        old = -torch.rand(S, L, generator=gen, device="cuda")
        logp = old + 0.2 * torch.randn(S, L, generator=gen, device="cuda")
        adv = torch.randn(S, generator=gen, device="cuda")
        mask = torch.rand(S, L, generator=gen, device="cuda") < 0.2 + 0.6 * k
        cases.append((logp, old, adv, mask))
        outs.append([(torch.zeros(4, device="cuda"), torch.zeros(S, L, device="cuda")) for _ in range(rounds)])
        alone.append(fs.policy_loss(logp, old, adv, mask=mask))
    torch.cuda.synchronize()

    def work(k):
        logp, old, adv, mask = cases[k]
        for out in outs[k]:
            fs.policy_loss(logp, old, adv, mask=mask, out=out, stream=per_thread)

    threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for want, got in zip(alone, outs):
        for r in got:
            for a, b in zip(want, r):
                assert torch.equal(a, b)
    fs.check(fs.library().fs_workspace_release())
    assert fs.device_error() == 0


@pytest.mark.parametrize("mean", ["token", "sequence"])
def test_a_loss_launch_that_fails_leaves_no_count(fs, torch_cuda, mean):
    """The counting launch has run, the one that takes the count away has not:
    the next call counts from zero."""
    torch = torch_cuda
    gen = torch.Generator(device="cuda").manual_seed(14)
    old = -torch.rand(5, 40, generator=gen, device="cuda")
    mask = torch.rand(5, 40, generator=gen, device="cuda") < 0.5
    args = old + 0.1, old, torch.randn(5, generator=gen, device="cuda")
    want = fs.policy_loss(*args, mask=mask, mean=mean)
    for _ in range(2):
        fs.debug_set_fault(fs.FS_FAULT_LATER_LAUNCH)
        try:
            with pytest.raises(fs.FlashSampleError) as e:
                fs.policy_loss(*args, mask=mask, mean=mean)
        finally:
            fs.debug_set_fault(fs.FS_FAULT_NONE)
        assert e.value.status == "FS_ERR_CUDA"
    for a, b in zip(want, fs.policy_loss(*args, mask=mask, mean=mean)):
        assert torch.equal(a, b)


def _on_another_stream(torch, shapes, call, use):
    """call(stream)'s results, made while the current stream has yet to read
    tensors of these shapes and types that the program has dropped: none of
    the results may lie in their memory."""
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    dropped = [torch.full(s, 3.0, device="cuda").to(t) for s, t in shapes for _ in range(3)]
    addresses = {t.data_ptr() for t in dropped}
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)                          # some 10 ms of the current stream
    read = [t.clone() for t in dropped]
    dropped.clear()
    results = call(side)
    assert not addresses & {t.data_ptr() for t in results}
    torch.cuda.current_stream().wait_stream(side)
    got = [t.clone() for t in results]
    del results
    torch.cuda.synchronize()
    assert all(bool((t == 3).all()) for t in read)
    for a, b in zip(use, got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("what", ["scores", "gradients", "policy", "clip"])
def test_results_on_a_given_stream(fs, torch_cuda, what):
    """With stream=, the results' memory is not still in use on the current
    stream, and the results are the same."""
    torch = torch_cuda
    gen = torch.Generator(device="cuda").manual_seed(15)
    n, d, V = 200, 64, 3000
    h, W = (torch.randn(m, d, generator=gen, device="cuda").bfloat16() for m in (n, V))
    ids, temp = torch.randint(0, V, (n,), generator=gen, device="cuda"), torch.ones(n, device="cuda")
    logp, lse = fs.token_logprobs(h, W, ids, temp)
    old = logp - 0.1                                       # (every input is there before the current stream is held up)
    f32, bf16 = torch.float32, torch.bfloat16
    if what == "scores":
        shapes = [((n,), f32)]
        call = lambda s=None: list(fs.token_logprobs(h, W, ids, temp, stream=s))  # noqa: E731
    elif what == "gradients":
        shapes = [((n, d), bf16), ((V, d), bf16), ((fs.logprob_buffer(n, V).numel(),), f32)]

        def call(s=None):
            kept = fs.logprob_buffer(n, V, stream=s)
            a, b = fs.token_logprobs(h, W, ids, temp, kept=kept, stream=s)
            return [*fs.token_logprobs_backward(h, W, ids, temp, a, b, temp, kept=kept, stream=s)]
    elif what == "policy":
        shapes = [((4,), f32), ((n,), f32)]
        call = lambda s=None: list(fs.policy_loss(logp, old, lse, stream=s))  # noqa: E731
    else:
        shapes = [((), f32)]
        call = lambda s=None: [fs.clip_grad_norm([logp], float("inf"), stream=s)]  # noqa: E731
    want = call()
    _on_another_stream(torch, shapes, call, want)


@pytest.mark.parametrize("what", ["sample", "logits", "topk", "combine", "norms"])
def test_samples_on_a_given_stream(fs, torch_cuda, what):
    torch = torch_cuda
    gen = torch.Generator(device="cuda").manual_seed(16)
    n, d, V = 40, 64, 700
    h, W = (torch.randn(m, d, generator=gen, device="cuda").bfloat16() for m in (n, V))
    temp = torch.ones(n, device="cuda")
    ids, mx = fs.sample(h, W, temp, 1, 2)
    ids, mx = torch.stack((ids, ids)), torch.stack((mx, mx - 1))
    i64, f32 = torch.int64, torch.float32
    shapes, call = {
        "sample": ([((n,), i64), ((n,), f32)], lambda s=None: [*fs.sample(h, W, temp, 1, 2, stream=s)]),
        "logits": ([((n,), i64), ((n,), f32), ((n, V), f32)],
                   lambda s=None: [*fs.debug_fused_logits(h, W, temp, 1, 2, stream=s)]),
        "topk": ([((n, 3), i64), ((n, 3), f32)], lambda s=None: [*fs.sample_topk(h, W, temp, 1, 2, 3, stream=s)]),
        "combine": ([((n,), i64), ((n,), f32)], lambda s=None: [*fs.combine_shards(mx, ids, stream=s)]),
        "norms": ([((V,), f32)], lambda s=None: [fs.row_norms(W, stream=s)])}[what]
    want = call()
    _on_another_stream(torch, shapes, call, want)


def test_reserve_within_a_capture(fs, torch_cuda):
    """On a stream that has sampled before there is nothing left to grow for
    sampling: reserving within a capture succeeds, and the graph samples."""
    torch = torch_cuda
    h, W = torch.ones(8, 64, device="cuda").bfloat16(), torch.ones(300, 64, device="cuda").bfloat16()
    temp = torch.ones(8, device="cuda")
    torch.cuda.synchronize()
    fs.check(fs.library().fs_workspace_release())
    stream = torch.cuda.Stream()
    want = fs.sample(h, W, temp, 1, 2, stream=stream)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        fs.workspace_reserve(8, 300)
        got = fs.sample(h, W, temp, 1, 2)
        with pytest.raises(fs.FlashSampleError) as e:      # the block of the training calls is not there
            fs.clip_grad_norm([temp], 1.0)
        assert e.value.status == "FS_ERR_WORKSPACE"
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
