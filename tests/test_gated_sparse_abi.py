"""CPU-only checks of the gated feed-forward block with a sparse down-projection: the workspace of the call is the
caller's, never the one that the linear layer's call keeps for each stream."""
import pytest

import activation_sparse_gemm_b200 as rl
from tests.test_gated_abi import AT, forward, lib  # noqa: F401  (lib is a fixture)

LA, LB = 20 << 24, 21 << 24


@pytest.mark.parametrize("sizes", [(1, 64, 128), (6, 64, 128), (300, 520, 1032)], ids=str)
@pytest.mark.parametrize("R", [0, 16])
def test_workspace_of_the_sparse_layer(lib, sizes, R):  # noqa: F811
    import torch
    M, D, F = sizes
    need = rl.rtlynx_workspace_size(M, F, D, R, rl.MODE_SPARSE)
    assert need > 0
    assert R == 0 or need > rl.rtlynx_workspace_size(M, F, D, 0, rl.MODE_SPARSE)
    far = {n: (i + 1) << 30 for i, n in enumerate(AT)}
    call = dict(far, sizes=sizes, mode=rl.MODE_SPARSE, R=R, la=LA if R else None, lb=LB if R else None)
    if not torch.cuda.is_available():  # else it would launch
        assert forward(lib, **call, ws_bytes=need) != rl.ERR_INVALID_ARG
    for change in (dict(ws=None), dict(ws=None, ws_bytes=0), dict(ws_bytes=0), dict(ws_bytes=need - 1),
                   dict(ws=far["ws"] + 16), dict(ws=far["H"]), dict(ws=far["Y"]), dict(ws=far["W_down"]),
                   dict(ws=far["low"] - need + 256)):
        assert forward(lib, **dict(dict(call, ws_bytes=need), **change)) == rl.ERR_INVALID_ARG, change
    if R:
        assert forward(lib, **dict(call, ws=LB), ws_bytes=need) == rl.ERR_INVALID_ARG
