"""Calls of the query/key and gated operators as programs make them: handles of streams, several host threads."""
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
