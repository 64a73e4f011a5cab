"""Calls of the query/key and gated operators as programs make them: handles of streams, several host threads."""
import threading

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
