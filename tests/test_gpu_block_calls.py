"""Calls of the query/key and gated operators as programs make them: handles of streams, several host threads."""
import threading
import time

import pytest
import torch

import activation_sparse_gemm_b200 as rl

pytestmark = pytest.mark.gpu


def normal(gen, *shape, scale=1.0):
    return (scale * torch.randn(*shape, device="cuda", generator=gen)).bfloat16()


def gated_inputs(M, D, F, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (normal(gen, M, D), normal(gen, F, D, scale=D ** -0.5), normal(gen, F, D, scale=D ** -0.5),
            normal(gen, D, F, scale=F ** -0.5))


def test_handle_zero_is_the_default_stream():
    """torch.cuda.default_stream().cuda_stream is 0: the call runs there, not on a stream of its own."""
    handle = torch.cuda.default_stream().cuda_stream
    assert handle == 0
    args = gated_inputs(40, 136, 264)
    with rl._on(args[0], handle):
        assert torch.cuda.current_stream() == torch.cuda.default_stream()
    want = rl.gated_mlp(*args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # the handle given, not the current stream, is where the call runs
        got = rl.gated_mlp(*args, stream=handle)
    assert torch.equal(got, want)


SPARSE = [(1, 264, 520), (12, 264, 520), (200, 264, 520), (40, 2056, 520), (700, 264, 1032), (300, 1032, 2056)]


def sparse_call(M, D, F, R=16, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(100 + seed)
    args = gated_inputs(M, D, F, seed)
    pair = dict(L_A=normal(gen, D, R, scale=0.1), L_B=normal(gen, R, F, scale=0.1)) if R else {}
    return args, lambda **more: rl.gated_mlp(*args, mode_down=rl.MODE_SPARSE, **pair, **more)


@pytest.mark.parametrize("R", [0, 16])
@pytest.mark.parametrize("M,D,F", SPARSE)
def test_sparse_down_in_captured_graphs(M, D, F, R):
    """Captured on a stream that has made no call before, two graphs hold a workspace each: replayed at once on two
    streams, behind larger eager calls on the stream of the capture, both give the eager result."""
    (X, *_), call = sparse_call(M, D, F, R)
    call()
    _, larger = sparse_call(4 * M + 3, D + 8, F + 136, seed=1)
    torch.cuda.synchronize()
    capture = torch.cuda.Stream()
    graphs, outs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=capture):
            outs.append(call())
        graphs.append(graph)
    for seed in range(2):
        with torch.cuda.stream(capture):
            X.copy_(normal(torch.Generator(device="cuda").manual_seed(seed), M, D))
            want = call()
            larger()
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in graphs]
        for _ in range(4):
            for graph, stream in zip(graphs, streams):
                with torch.cuda.stream(stream):
                    graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out, want) for out in outs)
    assert rl.rtlynx_stream_status() == rl.OK


def in_threads(works):
    """Runs the functions in a host thread each, at once; what they returned."""
    results = [None] * len(works)

    def run(i):
        try:
            results[i] = works[i]()
        except Exception as e:  # reported by the caller's comparison
            results[i] = e

    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(works))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    return results


@pytest.mark.parametrize("M,D,F", [(128, 256, 256), (300, 264, 520), (12, 264, 520), (200, 264, 520), (700, 264, 1032)])
def test_first_call_of_a_host_thread(M, D, F):
    """A call that is all the CUDA work its thread has done, with nothing left to set up but the thread itself."""
    X, gate, up, down = gated_inputs(M, D, F)
    q = X[:, :256].unflatten(1, (2, 128))
    positions, plan = torch.arange(M, device="cuda")[:, None], rl.Rope((128,))
    _, saved = rl.gated_mlp(X, gate, up, down, save=True)
    calls = [lambda: rl.linear(X, gate), lambda: rl.linear(X, gate, mode=rl.MODE_DENSE_SKIP),
             lambda: rl.gated_mlp(X, gate, up, down),
             lambda: rl.gated_mlp_backward(X, X, gate, up, down, saved)[0],
             lambda: rl.gated_mlp(X, gate, up, down, mode_down=rl.MODE_SPARSE),
             lambda: rl.rope(q, None, positions, plan)[0]]
    want = [call() for call in calls]
    torch.cuda.synchronize()
    for call, ref in zip(calls, want):
        got, = in_threads([call])
        assert isinstance(got, torch.Tensor), got
        assert torch.equal(got, ref)


def test_lora_pair_of_the_sparse_down_projection():
    """Taken where the sparse form is asked for, left out where the dense one is, and refused in any other shape."""
    M, D, F, R = 40, 264, 520, 16
    (X, *W), call = sparse_call(M, D, F, R)
    plain = rl.gated_mlp(X, *W, mode_down=rl.MODE_SPARSE)
    assert not torch.equal(call(), plain)
    gen = torch.Generator(device="cuda").manual_seed(9)
    A, B = normal(gen, D, R), normal(gen, R, F)
    assert torch.equal(rl.gated_mlp(X, *W, mode_down=rl.MODE_DENSE_SKIP, L_A=A, L_B=B), rl.gated_mlp(X, *W))
    assert torch.equal(rl.gated_mlp(X, *W, mode_down=rl.MODE_SPARSE, L_A=A[:, :0], L_B=B[:0]), plain)
    for la, lb in ((A, None), (None, B), (A, B.flatten()), (A[:, :8], B), (A, B[:8]), (A.T, B), (A, B.T), (A.float(), B),
                   (A, B.cpu()), (A, B[:0])):
        with pytest.raises(ValueError):
            rl.gated_mlp(X, *W, mode_down=rl.MODE_SPARSE, L_A=la, L_B=lb)
    with pytest.raises(ValueError):
        rl.gated_mlp(X, *W, L_A=A, L_B=B)


@pytest.mark.parametrize("which", ["rope", "gated_mlp"])
def test_other_host_threads_run_while_a_launch_waits(which):
    """More launches than a stream's queue holds, behind a kernel of about a second: one of them waits for it, and this
    thread meanwhile goes on.  Held up, it would stand still as long as that call."""
    X, *W = gated_inputs(2, 64, 128)
    out = torch.empty_like(X)
    positions, plan = torch.zeros(2, 1, dtype=torch.int32, device="cuda"), rl.Rope((64,))
    q, q_out = X.view(2, 1, 64), out.view(2, 1, 64)
    calls = {"rope": lambda: rl.rope(q, None, positions, plan, out=(q_out, None)),
             "gated_mlp": lambda: rl.gated_mlp(X, *W, out=out)}
    call = calls[which]
    call()
    torch.cuda.synchronize()
    waited = 0.0

    def work():
        nonlocal waited
        torch.cuda._sleep(2_000_000_000)
        for _ in range(4000):
            before = time.perf_counter()
            call()
            waited = max(waited, time.perf_counter() - before)

    thread = threading.Thread(target=work)
    thread.start()
    stood, last = 0.0, time.perf_counter()
    while thread.is_alive():
        time.sleep(0.002)
        now = time.perf_counter()
        stood, last = max(stood, now - last), now
    torch.cuda.synchronize()
    assert waited > 0.2, "nothing waited: the queue is longer than this test takes it to be"
    assert stood < waited / 2


@pytest.mark.parametrize("mode", [rl.MODE_DENSE_SKIP, rl.MODE_SPARSE])
def test_host_threads_on_one_stream(mode):
    """Each of several threads gets its own results, whatever the others launch between its kernels."""
    stream = torch.cuda.Stream()
    jobs = []
    for i, (M, D, F) in enumerate(SPARSE):
        args = gated_inputs(M, D, F, seed=i)
        jobs.append((args, rl.gated_mlp(*args, mode_down=mode)))
    torch.cuda.synchronize()

    def work(args, want):
        for _ in range(40):
            got = [rl.gated_mlp(*args, mode_down=mode, stream=stream) for _ in range(5)]
            stream.synchronize()
            if not all(torch.equal(y, want) for y in got):
                return "wrong"
        return "right"

    assert in_threads([lambda job=job: work(*job) for job in jobs]) == ["right"] * len(jobs)
    assert rl.rtlynx_stream_status() == rl.OK
