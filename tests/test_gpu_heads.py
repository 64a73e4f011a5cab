"""Rotary positions and the query/key head norm on the GPU, against the
definition in 64 bits.

Tolerances.  h = finfo.eps / 2 is the rounding of the output's type.  In
front of it stand 32-bit steps of 2^-24 each: sine and cosine are off by at
most 2^-22 absolutely, products and sums of a pair add three steps, the norm's
factor about ten (thirteen additions of squares count half under the root,
then the reciprocal root's two): less than 2^-19 of the terms' magnitudes.
fp16 adds half its smallest step, 2^-25."""
import math

import pytest
import torch

import activation_sparse_gemm_b200 as rl

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-6


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    return 2.0 ** -25 if dtype == torch.float16 else 2.0 ** -140


def angles(positions, axes, theta, inv_freq=None):
    """[.., pairs] angles in float64."""
    cols, at = [], 0
    for a, n in enumerate(axes):
        f = torch.tensor([theta ** (-2.0 * j / n) for j in range(n // 2)], dtype=torch.float64)
        if inv_freq is not None:
            f = torch.tensor(inv_freq[at:at + n // 2], dtype=torch.float64)
        at += n // 2
        cols.append(positions[..., a, None].double() * f)
    return torch.cat(cols, -1)


def split(x, pairs, pairing):
    if pairing == rl.ROPE_INTERLEAVED:
        return x[..., 0:2 * pairs:2], x[..., 1:2 * pairs:2]
    return x[..., :pairs], x[..., pairs:2 * pairs]


def join(a, b, rest, pairing):
    turned = torch.stack([a, b], -1).flatten(-2) if pairing == rl.ROPE_INTERLEAVED else torch.cat([a, b], -1)
    return torch.cat([turned, rest], -1)


def turn(x, ang, pairing, sign=1.0):
    pairs = ang.shape[-1]
    a, b = split(x, pairs, pairing)
    c, s = ang.cos()[..., None, :], sign * ang.sin()[..., None, :]
    return join(a * c - b * s, a * s + b * c, x[..., 2 * pairs:], pairing)


def pair_size(x, pairs, pairing):
    """|x0| + |x1| of each channel's pair (|x| of a channel that is not turned)."""
    a, b = split(x.abs(), pairs, pairing)
    return join(a + b, a + b, x[..., 2 * pairs:].abs(), pairing)


def norm(x, w):
    r = (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
    return x * r * w


def check(got, ref, size, dtype, steps=2.0 ** -19):
    err = (got.double().cpu() - ref).abs()
    tol = half_step(dtype) * ref.abs() + steps * size + tiny(dtype)
    assert got.dtype == dtype and got.shape == ref.shape
    worst = (err - tol).max().item()
    assert worst <= 0, f"off by {worst:.3e} beyond the tolerance"


def heads(gen, layout, dtype, B, S, Hq, Hk, D):
    def new(*shape):
        return torch.randn(*shape, generator=gen, dtype=torch.float32).to(dtype).cuda()
    if layout == "packed":
        qkv = new(B, S, Hq + 2 * Hk, D)
        return qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hk]
    if layout == "heads_first":
        return new(B, Hq, S, D).transpose(1, 2), new(B, Hk, S, D).transpose(1, 2)
    if layout == "broadcast":  # one sequence's heads for the whole batch
        return new(1, S, Hq, D).expand(B, S, Hq, D), new(1, S, Hk, D).expand(B, S, Hk, D)
    return new(B, S, Hq, D), new(B, S, Hk, D)


CASES = [
    # dtype, B, S, Hq, Hk, D, axes, pairing, layout
    ("bf16", 1, 1, 1, 1, 8, (8,), rl.ROPE_INTERLEAVED, "plain"),
    ("bf16", 3, 1, 5, 1, 128, (128,), rl.ROPE_HALF, "packed"),
    ("bf16", 2, 37, 6, 3, 128, (44, 42, 42), rl.ROPE_INTERLEAVED, "packed"),
    ("fp16", 2, 33, 7, 2, 128, (32, 48, 48), rl.ROPE_HALF, "heads_first"),
    ("fp32", 1, 65, 3, 3, 128, (16, 56, 56), rl.ROPE_INTERLEAVED, "packed"),
    ("fp32", 2, 19, 4, 4, 64, (64,), rl.ROPE_HALF, "heads_first"),
    ("fp16", 1, 130, 4, 4, 72, (8, 32, 32), rl.ROPE_INTERLEAVED, "plain"),
    ("bf16", 1, 130, 4, 2, 96, (2, 2, 2, 2), rl.ROPE_HALF, "plain"),
    ("bf16", 2, 9, 3, 1, 256, (100, 100), rl.ROPE_HALF, "packed"),
    ("fp32", 1, 11, 2, 1, 200, (50, 6), rl.ROPE_INTERLEAVED, "packed"),
    ("fp16", 1, 700, 40, 8, 24, (6, 6, 6), rl.ROPE_INTERLEAVED, "plain"),
    ("bf16", 1, 3000, 9, 1, 64, (20, 44), rl.ROPE_INTERLEAVED, "heads_first"),
    ("bf16", 4, 13, 2, 2, 16, (16,), rl.ROPE_HALF, "broadcast"),
    ("fp16", 1, 50, 7, 5, 40, (10, 30), rl.ROPE_HALF, "packed"),     # six heads of five lanes a warp pass
    ("fp32", 2, 31, 8, 4, 80, (16, 32, 32), rl.ROPE_HALF, "plain"),  # three of ten
    ("bf16", 1, 70, 33, 1, 8, (2, 4), rl.ROPE_INTERLEAVED, "packed"),  # 32 heads of one lane
    ("bf16", 1, 17, 5, 2, 136, (8, 64, 64), rl.ROPE_INTERLEAVED, "heads_first"),  # one head of 17
]


def make(case, seed=0):
    dtype, B, S, Hq, Hk, D, axes, pairing, layout = case
    dtype = TYPES[dtype]
    gen = torch.Generator().manual_seed(seed)
    q, k = heads(gen, layout, dtype, B, S, Hq, Hk, D)
    w = [(1 + 0.3 * torch.randn(D, generator=gen)).to(dtype).cuda() for _ in range(2)]
    positions = torch.randint(-50, 5000, (B, S, len(axes)), generator=gen, dtype=torch.int32)
    return dtype, q, k, w, positions, rl.Rope(axes, theta=10000.0, pairing=pairing), axes, pairing


@pytest.mark.parametrize("case", CASES, ids=str)
def test_rope(case):
    dtype, q, k, _, positions, plan, axes, pairing = make(case)
    ang = angles(positions, axes, 10000.0)
    for x, y in zip((q, k), rl.rope(q, k, positions.cuda(), plan)):
        x = x.double().cpu()
        check(y, turn(x, ang, pairing), pair_size(x, ang.shape[-1], pairing), dtype)


@pytest.mark.parametrize("case", CASES, ids=str)
def test_rope_backward(case):
    dtype, q, k, _, positions, plan, axes, pairing = make(case)
    ang = angles(positions, axes, 10000.0)
    for g, dx in zip((q, k), rl.rope_backward(q, k, positions.cuda(), plan)):
        g = g.double().cpu()
        check(dx, turn(g, ang, pairing, -1.0), pair_size(g, ang.shape[-1], pairing), dtype)


@pytest.mark.parametrize("case", CASES, ids=str)
def test_norm_rope(case):
    dtype, q, k, w, positions, plan, axes, pairing = make(case)
    ang = angles(positions, axes, 10000.0)
    out = rl.qk_norm_rope(q, k, w[0], w[1], positions.cuda(), plan, eps=EPS)
    for x, wi, y in zip((q, k), w, out):
        n = norm(x.double().cpu(), wi.double().cpu())
        check(y, turn(n, ang, pairing), pair_size(n, ang.shape[-1], pairing), dtype)


def backward_reference(x, g, w, ang, pairing):
    """dx, dw, and the magnitudes that their tolerances scale with."""
    r = (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
    n = x * r
    gt = turn(g, ang, pairing, -1.0)
    size = pair_size(g, ang.shape[-1], pairing)
    gw = gt * w
    dx = r * (gw - n * (gw * n).mean(-1, keepdim=True))
    dx_size = r * (size * w.abs() + n.abs() * (size * w.abs() * n.abs()).mean(-1, keepdim=True))
    return dx, (gt * n).sum((0, 1, 2)), dx_size, (size * n.abs()).sum((0, 1, 2))


@pytest.mark.parametrize("case", CASES, ids=str)
def test_norm_rope_backward(case):
    dtype, q, k, w, positions, plan, axes, pairing = make(case)
    B, S = q.shape[:2]
    gen = torch.Generator().manual_seed(5)
    g = [torch.randn(x.shape, generator=gen).to(dtype).cuda() for x in (q, k)]
    ang = angles(positions, axes, 10000.0)
    dq, dk, dwq, dwk = rl.qk_norm_rope_backward(g[0], g[1], q, k, w[0], w[1], positions.cuda(), plan, eps=EPS)
    for x, gi, wi, dx, dw in ((q, g[0], w[0], dq, dwq), (k, g[1], w[1], dk, dwk)):
        dx_ref, dw_ref, dx_size, dw_size = backward_reference(x.double().cpu(), gi.double().cpu(), wi.double().cpu(),
                                                              ang, pairing)
        check(dx, dx_ref, dx_size, dtype)
        # a lane adds at most one term a head for each of its tokens (two, at these sizes), then come the lanes that
        # share channels, the warps, the rows of partial sums; a term itself is off by less than 2^-19
        chain = 2 * x.shape[2] + 3 + 8 + 64 + 8
        check(dw, dw_ref, dw_size, torch.float32, steps=2.0 ** -19 + chain * 2.0 ** -24)


@pytest.mark.parametrize("pairing", [rl.ROPE_INTERLEAVED, rl.ROPE_HALF])
def test_gradients_against_differences(pairing):
    """(f(x + t v) - f(x - t v)) / 2 t along a random direction equals <df, v>, in 32 bits.

    With t = 2^-8 the difference's own error is t^2 / 6 = 3e-6 of a third derivative of a few units, its rounding
    2^-24 / 2 t = 8e-6 of the outputs; over 4000 independent terms both stay far below 1e-3 of the root of the sum of
    squared terms."""
    gen = torch.Generator().manual_seed(11)
    B, S, H, D, axes = 2, 5, 3, 128, (32, 48, 48)
    def new(*shape):
        return torch.randn(*shape, generator=gen).cuda()
    q, k, gq, gk, vq, vk = (new(B, S, H, D) for _ in range(6))
    wq, wk, uq, uk = (new(D) for _ in range(4))
    positions = torch.randint(0, 900, (S, 3), generator=gen).cuda()
    plan = rl.Rope(axes, pairing=pairing)

    def f(t):
        yq, yk = rl.qk_norm_rope(q + t * vq, k + t * vk, wq + t * uq, wk + t * uk, positions, plan, eps=EPS)
        return (yq.double() * gq.double()).sum() + (yk.double() * gk.double()).sum()

    t = 2.0 ** -8
    numeric = ((f(t) - f(-t)) / (2 * t)).item()
    dq, dk, dwq, dwk = rl.qk_norm_rope_backward(gq, gk, q, k, wq, wk, positions, plan, eps=EPS)
    terms = [(dq * vq).double(), (dk * vk).double(), (dwq * uq).double(), (dwk * uk).double()]
    analytic = sum(x.sum() for x in terms).item()
    scale = math.sqrt(sum(x.square().sum().item() for x in terms))
    assert abs(numeric - analytic) <= 1e-3 * scale + 1e-2


@pytest.mark.parametrize("kind", ["int32", "int64", "fp32"])
@pytest.mark.parametrize("shared", [False, True])
def test_position_types_and_sharing(kind, shared):
    gen = torch.Generator().manual_seed(3)
    B, S, axes = 3, 21, (16, 24, 24)
    q = torch.randn(B, S, 2, 64, generator=gen).cuda()
    shape = (S, 3) if shared else (B, S, 3)
    if kind == "int64":
        positions = torch.randint(-(1 << 40), 1 << 40, shape, generator=gen)
    elif kind == "int32":
        positions = torch.randint(-(1 << 31), (1 << 31) - 1, shape, generator=gen).to(torch.int32)
    else:
        positions = (torch.rand(shape, generator=gen) - 0.5) * 1000
    y, none = rl.rope(q, None, positions.cuda(), rl.Rope(axes))
    assert none is None
    ang = angles(positions.expand(B, S, 3), axes, 10000.0)
    # in 64 bits a far angle is off by a few steps of 2^-53 of itself (frequency, 1 / 2 pi, product), here and in the
    # reference: seven together
    slack = 2.0 ** -19 + ang.abs().max().item() * 2.0 ** -50
    check(y, turn(q.double().cpu(), ang, rl.ROPE_INTERLEAVED), pair_size(q.double().cpu(), 32, rl.ROPE_INTERLEAVED),
          torch.float32, steps=slack)


def test_own_frequencies_and_strided_positions():
    gen = torch.Generator().manual_seed(4)
    S, axes = 40, (8, 4)
    freq = [0.5, 0.25, 0.1, 0.0, 2.0, 1e-3]
    q = torch.randn(S, 3, 16, generator=gen).cuda()
    table = torch.randint(0, 99, (2, S), generator=gen)  # axis first
    y, _ = rl.rope(q, None, table.cuda().T, rl.Rope(axes, inv_freq=freq, pairing=rl.ROPE_INTERLEAVED))
    ang = angles(table.T[None], axes, 1.0, freq)
    x = q.double().cpu()[None]
    check(y[None], turn(x, ang, rl.ROPE_INTERLEAVED), pair_size(x, 6, rl.ROPE_INTERLEAVED), torch.float32)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("layout", ["tokens", "heads_first"])
def test_in_place_in_a_packed_buffer_leaves_the_rest(dtype, layout):
    gen = torch.Generator().manual_seed(9)
    B, S, H, D = 2, 23, 4, 64
    shape = (B, S, 3 * H, D) if layout == "tokens" else (B, 3 * H, S, D)
    buf = torch.randn(*shape, generator=gen).to(TYPES[dtype]).cuda()
    before = buf.clone()

    def part(b, i):
        return b[:, :, i * H:(i + 1) * H] if layout == "tokens" else b[:, i * H:(i + 1) * H].transpose(1, 2)

    positions = torch.randint(0, 99, (S, 2), generator=gen).cuda()
    plan = rl.Rope((32, 16), pairing=rl.ROPE_HALF)
    w = torch.ones(D, dtype=TYPES[dtype], device="cuda") * 1.5
    want = rl.qk_norm_rope(part(before, 0), part(before, 1), w, None, positions, plan)
    rl.qk_norm_rope(part(buf, 0), part(buf, 1), w, None, positions, plan, out=(part(buf, 0), part(buf, 1)))
    assert torch.equal(part(buf, 0), want[0]) and torch.equal(part(buf, 1), want[1])
    assert torch.equal(part(buf, 2), part(before, 2))
    # gradients over their own incoming gradients
    g = torch.randn(*shape, generator=gen).to(TYPES[dtype]).cuda()
    args = (part(before, 0), part(before, 1), w, None, positions, plan)
    want = rl.qk_norm_rope_backward(part(g, 0), part(g, 1), *args)
    rl.qk_norm_rope_backward(part(g, 0), part(g, 1), *args, out=(part(g, 0), part(g, 1)))
    assert torch.equal(part(g, 0), want[0]) and torch.equal(part(g, 1), want[1])
    assert want[3] is None and want[2].shape == (D,)


def test_values_stay_in_their_head_and_pair():
    """NaN and infinity touch only their own head (norm) or pair (rotation); zero heads stay zero."""
    S, H, D = 4, 3, 64
    x = torch.ones(S, H, D, device="cuda")
    x[1, 1, 60] = math.inf        # not turned by the axes below
    x[2, 0, 0] = math.nan
    x[3, 2] = 0
    positions = torch.arange(1, S + 1, device="cuda")[:, None].expand(S, 2)
    for pairing in (rl.ROPE_INTERLEAVED, rl.ROPE_HALF):
        plan = rl.Rope((16, 32), pairing=pairing)
        y, _ = rl.rope(x, None, positions, plan)
        bad = torch.zeros(S, H, D, dtype=torch.bool, device="cuda")
        bad[1, 1, 60] = bad[2, 0, 0] = True
        bad[2, 0, 1 if pairing == rl.ROPE_INTERLEAVED else 24] = True
        assert torch.equal(~torch.isfinite(y), bad) and y[1, 1, 60] == math.inf
        assert (y[3, 2] == 0).all() and torch.equal(y[:, :, 48:][~bad[:, :, 48:]], x[:, :, 48:][~bad[:, :, 48:]])
        z, _ = rl.qk_norm_rope(x, None, None, None, positions, plan)
        spoiled = torch.zeros(S, H, dtype=torch.bool, device="cuda")
        spoiled[1, 1] = spoiled[2, 0] = True
        assert torch.isfinite(z[~spoiled]).all() and (z[3, 2] == 0).all() and z[2, 0].isnan().all()
        dq, _, dw, _ = rl.qk_norm_rope_backward(torch.ones_like(x), None, x, None, torch.ones(D, device="cuda"), None,
                                                positions, plan)
        assert torch.isfinite(dq[~spoiled]).all() and dw.isnan().all()


def test_offsets_beyond_32_bits():
    """Two tokens more than 2^31 elements apart."""
    far = (1 << 31) + 4096
    buf = torch.zeros(far + 2 * 128, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((2, 2, 128), (far, 128, 1))
    x.copy_(torch.randn(2, 2, 128, generator=torch.Generator().manual_seed(1)))
    positions = torch.tensor([[3], [1 << 20]], device="cuda")
    plan = rl.Rope((128,), pairing=rl.ROPE_HALF)
    want, _ = rl.rope(x.contiguous(), None, positions, plan)
    rl.rope(x, None, positions, plan, out=(x, None))
    assert torch.equal(x, want)
    assert buf[256:far].count_nonzero() == 0


def test_equal_calls_give_equal_bits_and_one_token_matches_many():
    gen = torch.Generator().manual_seed(2)
    B, S, H, D = 1, 2500, 10, 128
    q, k, gq, gk = (torch.randn(B, S, H, D, generator=gen).bfloat16().cuda() for _ in range(4))
    w = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    positions = torch.arange(S, device="cuda")[:, None]
    plan = rl.Rope((D,), pairing=rl.ROPE_HALF)
    a = rl.qk_norm_rope_backward(gq, gk, q, k, w, w, positions, plan)
    b = rl.qk_norm_rope_backward(gq, gk, q, k, w, w, positions, plan)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    # without the weights' gradients the inputs' are the same
    c = rl.qk_norm_rope_backward(gq, gk, q, k, w, w, positions, plan, weight_grads=False)
    assert torch.equal(a[0], c[0]) and torch.equal(a[1], c[1]) and c[2] is None and c[3] is None
    full = rl.qk_norm_rope(q, k, w, w, positions, plan)
    for s in (0, 1, S - 1):
        one = rl.qk_norm_rope(q[:, s:s + 1], k[:, s:s + 1], w, w, positions[s:s + 1], plan)
        assert torch.equal(one[0][:, 0], full[0][:, s]) and torch.equal(one[1][:, 0], full[1][:, s])


def test_other_stream_and_captured_graph():
    gen = torch.Generator().manual_seed(6)
    S, H, D = 300, 4, 128
    q, k, gq, gk = (torch.randn(S, H, D, generator=gen).bfloat16().cuda() for _ in range(4))
    w = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    positions = torch.arange(S, device="cuda")[:, None]
    plan = rl.Rope((D,))
    want = rl.qk_norm_rope(q, k, w, w, positions, plan)
    want_grad = rl.qk_norm_rope_backward(gq, gk, q, k, w, w, positions, plan)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, int(side.cuda_stream)):
        got = rl.qk_norm_rope(q, k, w, w, positions, plan, stream=stream)
        grad = rl.qk_norm_rope_backward(gq, gk, q, k, w, w, positions, plan, stream=stream)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got + grad, want + want_grad))
    # two graphs, each with workspace of its own, replayed at once on two streams
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y = rl.qk_norm_rope(q, k, w, w, positions, plan)
            outs.append(y + rl.qk_norm_rope_backward(gq, gk, q, k, w, w, positions, plan))
        graphs.append(g)
    q2 = torch.randn(S, H, D, generator=gen).bfloat16().cuda()
    q.copy_(q2)
    want = rl.qk_norm_rope(q, k, w, w, positions, plan) + rl.qk_norm_rope_backward(gq, gk, q, k, w, w, positions, plan)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for out in outs:
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_refusals_on_the_gpu():
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    positions = torch.zeros(4, 1, dtype=torch.int32, device="cuda")
    plan = rl.Rope((64,))
    with pytest.raises(rl.RtlynxError) as e:
        rl.rope(q, None, positions, plan, out=(torch.empty_like(q[:, :1]).expand(4, 2, 64), None))
    assert e.value.status == rl.ERR_INVALID_ARG
    with pytest.raises(ValueError):
        rl.rope(q, None, positions.short(), plan)
    with pytest.raises(ValueError):
        rl.rope(q, None, positions[:3], plan)
    with pytest.raises(ValueError):
        rl.rope(q, q.half(), positions, plan)
    with pytest.raises(ValueError):
        rl.rope(q.double(), None, positions, plan)
    with pytest.raises(ValueError):
        rl.qk_norm_rope(q, None, torch.ones(64, device="cuda"), None, positions, plan)
    assert rl.rtlynx_stream_status() == rl.OK
