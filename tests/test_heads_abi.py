"""CPU-only checks of the query and key heads' entry points: what they refuse,
before touching a GPU (the addresses are never dereferenced)."""
import ctypes
import math

import pytest

import activation_sparse_gemm_b200 as rl
from activation_sparse_gemm_b200 import build as rl_build

B, S, H, D = 2, 6, 4, 64
ROW = 3 * H * D  # queries, keys and values of one token side by side
Q, K, QO, KO = 1 << 24, 2 << 24, 3 << 24, 4 << 24
GQ, GK = 5 << 24, 6 << 24
POS, W, WS, DW = 7 << 24, 8 << 24, 9 << 24, 10 << 24


@pytest.fixture(scope="module")
def lib():
    rl_build.build()
    return rl.lib()


def view(ptr, heads=H, sb=S * H * D, ss=H * D, sh=D):
    return rl.HeadsView(ptr, heads, sb, ss, sh)


def spec(axes=(16, 24, 24), pairing=rl.ROPE_INTERLEAVED, pos_type=rl.POS_INT32, theta=1e4, n_axes=None):
    dims = (ctypes.c_int32 * rl.MAX_AXES)(*axes[:rl.MAX_AXES])
    return rl.RopeSpec(len(axes) if n_axes is None else n_axes, dims, pairing, pos_type, theta, None)


def norm_rope(lib, q=None, k=None, qo=None, ko=None, w=W, sizes=(B, S, D), dtype=rl.BF16, eps=1e-6, sp=None,
              positions=POS, strides=(S * 3, 3, 1)):
    return lib.rtlynx_qk_norm_rope(q or view(Q), k or view(K), w, w, qo or view(QO), ko or view(KO), *sizes, dtype,
                                   eps, sp or spec(), positions, *strides, None)


def past_the_checks(status):
    """Without a GPU a call that passes every check ends at the device query."""
    return status not in (rl.ERR_INVALID_ARG,)


def test_valid_call_passes_the_checks(lib):
    import torch
    if torch.cuda.is_available():
        pytest.skip("would launch")
    assert past_the_checks(norm_rope(lib))


@pytest.mark.parametrize("sizes", [(0, S, D), (B, 0, D), (B, S, 0), (-1, S, D), (B, S, 60)])
def test_bad_sizes(lib, sizes):
    assert norm_rope(lib, sizes=sizes) == rl.ERR_INVALID_ARG


@pytest.mark.parametrize("change", [
    dict(dtype=3), dict(dtype=-1), dict(eps=0.0), dict(eps=-1e-6), dict(eps=math.nan), dict(eps=math.inf),
    dict(sp=spec(pairing=2)), dict(sp=spec(pos_type=3)), dict(sp=spec(theta=0.0)), dict(sp=spec(theta=math.nan)),
    dict(sp=spec(axes=(15, 17, 32))), dict(sp=spec(axes=(32, 32, 2))), dict(sp=spec(axes=(0, 64))),
    dict(sp=spec(axes=(16,), n_axes=0)), dict(positions=None), dict(positions=POS + 2), dict(strides=(-3, 3, 1)),
    dict(sp=spec(pos_type=rl.POS_INT64), positions=POS + 4), dict(w=W + 2)])
def test_bad_arguments(lib, change):
    assert norm_rope(lib, **change) == rl.ERR_INVALID_ARG


@pytest.mark.parametrize("change", [
    dict(q=view(None)), dict(q=view(Q + 8)), dict(q=view(Q, heads=0)), dict(q=view(Q, sh=60)),
    dict(q=view(Q, ss=-256)), dict(qo=view(QO, heads=H - 1)),
    dict(qo=view(QO, sh=0)), dict(qo=view(QO, ss=0)), dict(qo=view(QO, sb=0)), dict(qo=view(QO, ss=D))])
def test_bad_views(lib, change):
    assert norm_rope(lib, **change) == rl.ERR_INVALID_ARG


def test_unsupported(lib):
    assert norm_rope(lib, sizes=(B, S, 264)) == rl.ERR_UNSUPPORTED
    assert norm_rope(lib, sp=spec(n_axes=5)) == rl.ERR_UNSUPPORTED
    assert norm_rope(lib, sp=spec(axes=(14, 6), pairing=rl.ROPE_HALF)) == rl.ERR_UNSUPPORTED
    assert norm_rope(lib, q=view(Q, heads=65537), qo=view(QO, heads=65537)) == rl.ERR_UNSUPPORTED


@pytest.mark.parametrize("change", [
    dict(qo=view(Q + 16)),                           # shifted by half a head's eighth
    dict(qo=view(Q, sb=S * H * D, ss=H * D + 8)),    # same start, other strides
    dict(qo=view(K)), dict(ko=view(Q)), dict(ko=view(QO)),
    dict(qo=view(W - 32)), dict(qo=view(POS)),
    dict(ko=view(QO + 2 * B * S * H * D - 16)),
])
def test_outputs_that_meet_something_else(lib, change):
    assert norm_rope(lib, **change) == rl.ERR_INVALID_ARG


def packed(ptr, slot, heads_first=False):
    if heads_first:  # [B, 3 H, S, D]
        return rl.HeadsView(ptr + 2 * slot * H * S * D, H, 3 * H * S * D, D, S * D)
    return rl.HeadsView(ptr + 2 * slot * H * D, H, S * ROW, ROW, D)


@pytest.mark.parametrize("heads_first", [False, True])
def test_parts_of_one_packed_buffer_are_told_apart(lib, heads_first):
    import torch
    if torch.cuda.is_available():
        pytest.skip("would launch")
    v = [packed(Q, i, heads_first) for i in range(3)]
    assert past_the_checks(norm_rope(lib, q=v[0], k=v[1], qo=v[0], ko=v[1]))    # in place
    assert past_the_checks(norm_rope(lib, q=v[0], k=v[1], qo=v[2], ko=v[1]))    # into the third part
    # swapped, or reaching into a neighbour's part
    assert norm_rope(lib, q=v[0], k=v[1], qo=v[1], ko=v[0]) == rl.ERR_INVALID_ARG
    shifted = rl.HeadsView(v[0].ptr + 16, H, v[0].stride_b, v[0].stride_s, v[0].stride_h)
    assert norm_rope(lib, q=v[0], k=v[1], qo=shifted, ko=v[1]) == rl.ERR_INVALID_ARG
    assert norm_rope(lib, q=v[0], k=v[1], qo=v[0], ko=shifted) == rl.ERR_INVALID_ARG


def backward(lib, gq=None, gk=None, q=None, k=None, dq=None, dk=None, dw_q=DW, dw_k=DW + 4096, ws=WS, ws_bytes=None):
    if ws_bytes is None:
        ws_bytes = lib.rtlynx_qk_norm_rope_workspace_size(D)
    return lib.rtlynx_qk_norm_rope_backward(gq or view(GQ), gk or view(GK), q or view(Q), k or view(K), W, W,
                                            dq or view(QO), dk or view(KO), dw_q, dw_k, B, S, D, rl.BF16, 1e-6,
                                            spec(), POS, S * 3, 3, 1, ws, ws_bytes, None)


def test_backward_refusals(lib):
    need = lib.rtlynx_qk_norm_rope_workspace_size(D)
    assert need > 0
    for change in (dict(ws=None), dict(ws_bytes=need - 1), dict(ws=WS + 16), dict(ws=Q), dict(ws=GQ), dict(dw_q=W),
                   dict(dw_q=DW, dw_k=DW + 16), dict(dw_q=DW + 4), dict(dw_q=GQ), dict(dw_q=WS), dict(dq=view(GK)),
                   dict(dq=view(K)), dict(gq=view(GQ, heads=2))):
        assert backward(lib, **change) == rl.ERR_INVALID_ARG, change
    null = None
    assert lib.rtlynx_qk_norm_rope_backward(view(GQ), null, view(Q), view(K), W, W, view(QO), view(KO), null, null, B,
                                            S, D, rl.BF16, 1e-6, spec(), POS, S * 3, 3, 1, null, 0,
                                            null) == rl.ERR_INVALID_ARG


def test_workspace_size(lib):
    assert [lib.rtlynx_qk_norm_rope_workspace_size(d) for d in (0, -8, 60, 264)] == [0, 0, 0, 0]
    assert lib.rtlynx_qk_norm_rope_workspace_size(256) % 256 == 0


def test_python_rope_arguments():
    with pytest.raises(ValueError):
        rl.Rope((16, 15))
    with pytest.raises(ValueError):
        rl.Rope((8,) * 5)
    with pytest.raises(ValueError):
        rl.Rope((16,), inv_freq=[1.0] * 7)
    assert rl.Rope((16,), inv_freq=range(8)).specs[0].inv_freq[7] == 7.0


def test_cpu_tensors_are_refused():
    import torch
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        rl.rope(q, None, torch.zeros(4, 1, dtype=torch.int32), rl.Rope((64,)))
