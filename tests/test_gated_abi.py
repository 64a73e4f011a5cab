"""CPU-only checks of the gated feed-forward block's entry points: what they
refuse, before touching a GPU (the addresses are never dereferenced)."""
import pytest

import activation_sparse_gemm_b200 as rl
from activation_sparse_gemm_b200 import build as rl_build

M, D, F = 6, 64, 128
NAMES = ("X", "W_gate", "W_up", "W_down", "G", "U", "low", "H", "Y", "dY", "dX", "dW_gate", "dW_up", "dW_down", "ws")
AT = {n: (i + 1) << 24 for i, n in enumerate(NAMES)}


@pytest.fixture(scope="module")
def lib():
    rl_build.build()
    return rl.lib()


def forward(lib, sizes=(M, D, F), R=0, act=rl.ACT_SILU, mode=rl.MODE_DENSE_SKIP, la=None, lb=None, ws_bytes=None,
            **at):
    a = dict(AT, **at)
    if ws_bytes is None:
        ws_bytes = lib.rtlynx_gated_mlp_block_workspace_size(*sizes, mode)
    return lib.rtlynx_gated_mlp_block(a["X"], a["W_gate"], a["W_up"], a["W_down"], la, lb, a["G"], a["U"], a["low"],
                                      a["H"], a["Y"], *sizes, R, act, mode, a["ws"], ws_bytes, None)


def backward(lib, sizes=(M, D, F), act=rl.ACT_SILU, ws_bytes=None, **at):
    a = dict(AT, **at)
    if ws_bytes is None:
        ws_bytes = max(lib.rtlynx_gated_mlp_backward_workspace_size(M, D, F), 1)
    return lib.rtlynx_gated_mlp_backward(a["dY"], a["X"], a["W_gate"], a["W_up"], a["W_down"], a["G"], a["U"], a["low"],
                                         a["H"], a["dX"], a["dW_gate"], a["dW_up"], a["dW_down"], *sizes, act, a["ws"],
                                         ws_bytes, None)


def test_valid_calls_pass_the_checks(lib):
    import torch
    if torch.cuda.is_available():
        pytest.skip("would launch")
    assert forward(lib) != rl.ERR_INVALID_ARG
    assert forward(lib, G=None, U=None, low=None) != rl.ERR_INVALID_ARG
    assert backward(lib) != rl.ERR_INVALID_ARG
    assert backward(lib, dX=None, dW_gate=None, dW_up=None, dW_down=None) == rl.OK


@pytest.mark.parametrize("call", [forward, backward])
@pytest.mark.parametrize("sizes", [(0, D, F), (M, 0, F), (M, D, 0), (M, 60, F), (M, D, 124), (-1, D, F)])
def test_bad_sizes(lib, call, sizes):
    assert call(lib, sizes=sizes) == rl.ERR_INVALID_ARG
    if sizes[0] > 0:
        assert lib.rtlynx_gated_mlp_backward_workspace_size(*sizes) == 0


@pytest.mark.parametrize("call", [forward, backward])
def test_unsupported_sizes_and_bad_activations(lib, call):
    assert call(lib, sizes=((1 << 28) + 1, D, F)) == rl.ERR_UNSUPPORTED
    assert call(lib, sizes=(M, D, (1 << 22) + 8)) == rl.ERR_UNSUPPORTED
    for act in (-1, 2):
        assert call(lib, act=act) == rl.ERR_INVALID_ARG


@pytest.mark.parametrize("name", ["X", "W_gate", "W_up", "W_down", "H", "Y"])
def test_forward_pointers(lib, name):
    assert forward(lib, **{name: None}) == rl.ERR_INVALID_ARG
    assert forward(lib, **{name: AT[name] + 8}) == rl.ERR_INVALID_ARG


def test_forward_saves_the_projections_whole_or_not_at_all(lib):
    assert forward(lib, G=None) == rl.ERR_INVALID_ARG
    assert forward(lib, U=None) == rl.ERR_INVALID_ARG
    assert forward(lib, low=None) == rl.ERR_INVALID_ARG
    assert forward(lib, G=None, U=None) == rl.ERR_INVALID_ARG
    assert forward(lib, G=AT["G"] + 2) == rl.ERR_INVALID_ARG


def test_down_layer_is_checked_as_a_linear_layer(lib):
    assert forward(lib, mode=5) == rl.ERR_INVALID_ARG
    assert forward(lib, mode=rl.MODE_SPARSE, R=16) == rl.ERR_INVALID_ARG  # a rank without factors
    assert forward(lib, mode=rl.MODE_SPARSE, R=12, la=20 << 24, lb=21 << 24) == rl.ERR_UNSUPPORTED
    assert forward(lib, mode=rl.MODE_SPARSE, R=16, la=AT["H"], lb=21 << 24) == rl.ERR_INVALID_ARG


SIZE = {"X": 2 * M * D, "Y": 2 * M * D, "dY": 2 * M * D, "dX": 2 * M * D, "G": 2 * M * F, "U": 2 * M * F,
        "low": 2 * M * F, "H": 2 * M * F, "W_gate": 2 * D * F, "W_up": 2 * D * F, "W_down": 2 * D * F, "dW_gate": 2 * D * F,
        "dW_up": 2 * D * F, "dW_down": 2 * D * F}


@pytest.mark.parametrize("out", ["G", "U", "low", "H", "Y"])
def test_forward_overlaps(lib, out):
    for other in ("X", "W_gate", "W_up", "W_down", "G", "U", "low", "H", "Y"):
        if other != out:
            for at in (AT[other] + SIZE[other] - 16, AT[other] - SIZE[out] + 16):
                assert forward(lib, **{out: at}) == rl.ERR_INVALID_ARG, other


@pytest.mark.parametrize("out", ["dX", "dW_gate", "dW_up", "dW_down"])
def test_backward_overlaps(lib, out):
    for other in SIZE:
        if other not in (out, "Y"):
            for at in (AT[other] + SIZE[other] - 16, AT[other] - SIZE[out] + 16):
                assert backward(lib, **{out: at}) == rl.ERR_INVALID_ARG, other
    assert backward(lib, **{out: AT["ws"]}) == rl.ERR_INVALID_ARG


def test_backward_pointers_and_workspace(lib):
    for name in ("dY", "X", "W_gate", "W_up", "W_down", "G", "U", "low", "H", "ws"):
        assert backward(lib, **{name: None}) == rl.ERR_INVALID_ARG
    need = lib.rtlynx_gated_mlp_backward_workspace_size(M, D, F)
    assert backward(lib, ws_bytes=need - 1) == rl.ERR_INVALID_ARG
    assert backward(lib, ws=AT["ws"] + 16) == rl.ERR_INVALID_ARG
    assert backward(lib, ws=AT["H"]) == rl.ERR_INVALID_ARG


def test_forward_workspace(lib):
    """Split down-projections need one: few tiles of a long K."""
    sizes = (100, 64, 8192)
    need = lib.rtlynx_gated_mlp_block_workspace_size(*sizes, rl.MODE_DENSE_SKIP)
    assert need > 0 and need % 256 == 0
    assert lib.rtlynx_gated_mlp_block_workspace_size(*sizes, rl.MODE_SPARSE) == 0
    assert lib.rtlynx_gated_mlp_block_workspace_size(100, 60, 8192, rl.MODE_DENSE_SKIP) == 0
    assert lib.rtlynx_gated_mlp_block_workspace_size(1, 64, 8192, rl.MODE_DENSE_SKIP) == 0
    assert lib.rtlynx_gated_mlp_block_workspace_size(100000, 5120, 8192, rl.MODE_DENSE_SKIP) == 0
    for change in (dict(ws=None), dict(ws=AT["ws"] + 16), dict(ws_bytes=need - 1), dict(ws=AT["W_up"]),
                   dict(ws=AT["Y"]), dict(ws=AT["H"])):
        assert forward(lib, sizes=sizes, **change) == rl.ERR_INVALID_ARG, change


def test_cpu_tensors_are_refused():
    import torch
    x, w = torch.zeros(4, 64).bfloat16(), torch.zeros(128, 64).bfloat16()
    with pytest.raises(ValueError):
        rl.gated_mlp(x, w, w, w.T.contiguous())
