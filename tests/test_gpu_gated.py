"""The gated feed-forward block on the GPU.

Two kinds of inputs.  Small whole numbers, for which every product and sum is
exact in 32 bits, so that each output is one rounding (2^-8 of it, half a step
of bf16) away from the exact value: a single misplaced element shows.  And
normal numbers, where the roundings of the operands between the products
count: each is at most 2^-8 of its value, uniform at worst, so it moves a term
of a sum by a standard deviation of at most 2^-8 / sqrt 3 of the term; n
roundings of each term give 2^-8 sqrt(n / 3) times the root of the sum of the
squared terms, and six standard deviations bound the largest of all elements.
(Measuring an element's error by its own terms, and not by the average
element, matters for few tokens: with one token a weight's gradient is a
single term, up to ten times the average one.)  32-bit accumulation adds
K 2^-23 at most."""
import math

import pytest
import torch

import activation_sparse_gemm_b200 as rl

pytestmark = pytest.mark.gpu

H_STEP = 2.0 ** -8

SIZES = [(1, 8, 8), (1, 64, 136), (2, 1032, 264), (3, 72, 40), (5, 520, 1000), (8, 136, 264), (9, 2056, 552),
         (16, 256, 128), (17, 136, 264), (33, 264, 72), (64, 64, 64), (128, 256, 512), (129, 200, 328), (256, 512, 256),
         (257, 520, 136), (300, 1032, 520), (700, 264, 1160), (1025, 72, 2056), (40, 264, 4104), (520, 136, 6152), (2900, 136, 72),
         (30, 2056, 264), (270, 2312, 520), (24, 136, 2312), (65, 200, 6152), (128, 72, 11016), (10, 4104, 5512),
         (200, 72, 11016), (130, 520, 11144), (380, 520, 4872), (500, 520, 4872), (1024, 264, 1544), (384, 264, 136)]


def ints(gen, shape, low, high, density):
    keep = torch.rand(shape, generator=gen) < density
    return (torch.randint(low, high + 1, shape, generator=gen) * keep).double()


def dev(x):
    return x.to(torch.bfloat16).cuda()


def rounded(x):
    return x.to(torch.bfloat16).double()


def check_exact(got, ref, what):
    err = (got.double().cpu() - ref).abs()
    worst = (err - H_STEP * ref.abs()).max().item()
    assert worst <= 0, f"{what}: off by {worst} beyond a rounding, at {torch.nonzero(err > H_STEP * ref.abs())[:4].tolist()}"


def whole_number_inputs(M, D, F, seed):
    """G >= 32, where SiLU and GELU are the identity in 32 bits (exp(-32) is below a step) with slope 1."""
    gen = torch.Generator().manual_seed(seed)
    X = ints(gen, (M, D), -1, 1, min(1.0, 24 / D))
    Wg = ints(gen, (F, D), -1, 1, 0.5)
    Wu = ints(gen, (F, D), -2, 2, 0.5)
    X[:, 0] = 1
    Wg[:, 0] = 80
    return gen, X, Wg, Wu


@pytest.mark.parametrize("act", [rl.ACT_SILU, rl.ACT_GELU])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_forward_whole_numbers(size, act):
    M, D, F = size
    gen, X, Wg, Wu = whole_number_inputs(M, D, F, M + D)
    Wd = ints(gen, (D, F), -1, 1, 0.5)
    G, U = X @ Wg.T, X @ Wu.T
    assert G.min() >= 32 and G.max() < 256
    H = rounded(G * U)
    for save in (False, True):
        out = rl.gated_mlp(dev(X), dev(Wg), dev(Wu), dev(Wd), act=act, save=save)
        y = out[0] if save else out
        check_exact(y, H @ Wd.T, "Y")
        if save:
            for got, ref, name in zip(out[1], (G, U, 0 * G, H), ("G", "U", "low", "H"), strict=True):
                assert torch.equal(got.double().cpu(), ref), name
    assert rl.rtlynx_stream_status() == rl.OK


@pytest.mark.parametrize("size", SIZES, ids=str)
def test_backward_whole_numbers(size):
    """dG = dH U and dU = dH G hold at G >= 32; sparse dY keeps dH, dG and dU within bf16's whole numbers."""
    M, D, F = size
    gen = torch.Generator().manual_seed(M * 7 + F)
    X = ints(gen, (M, D), -2, 2, 1.0)
    Wg, Wu = ints(gen, (F, D), -2, 2, 1.0), ints(gen, (F, D), -2, 2, 1.0)
    Wd = ints(gen, (D, F), -1, 1, 1.0)
    dY = ints(gen, (M, D), -1, 1, min(1.0, 2 / D))
    G = 32.0 * torch.randint(1, 3, (M, F), generator=gen).double()
    U = ints(gen, (M, F), -2, 2, 1.0)
    H = ints(gen, (M, F), -3, 3, 1.0)
    dH = dY @ Wd
    dG, dU = rounded(dH * U), rounded(dH * G)
    ref = (dG @ Wg + dU @ Wu, dG.T @ X, dU.T @ X, dY.T @ H)
    args = (dev(dY), dev(X), dev(Wg), dev(Wu), dev(Wd), (dev(G), dev(U), torch.zeros(M, F, dtype=torch.int16, device="cuda"), dev(H)))
    got = rl.gated_mlp_backward(*args)
    for a, b, name in zip(got, ref, ("dX", "dW_gate", "dW_up", "dW_down")):
        check_exact(a, b, name)
    for skip in range(4):  # any of them left out changes none of the others
        needs = [i != skip for i in range(4)]
        some = rl.gated_mlp_backward(*args, needs=needs)
        assert some[skip] is None
        assert all(torch.equal(a, b) for a, b, n in zip(got, some, needs) if n)
    only = rl.gated_mlp_backward(*args, needs=(False, False, False, True))
    assert torch.equal(only[3], got[3])
    assert rl.rtlynx_stream_status() == rl.OK


def reference(X, Wg, Wu, Wd, dY, act):
    """The block and its gradients in 64 bits, each with the scale of its operands' roundings.

    An output is a sum of terms a b.  A rounding of 2^-8 moves a term by 2^-8 of itself where it is a factor (H, dG, dU).
    G and U are kept to 2^-15: that of G moves act(G) by 2^-15 |G act'(G)| and act'(G) by 2^-15 |G act''(G)|, where
    |G act''(G)| < 1 for both activations.  With the terms so enlarged, independent roundings add up to at most
    2^-8 sqrt(1 / 3) (1 + 2^-6) times the root of the sum of the squared terms: that root is the scale."""
    f = torch.nn.functional
    leaves = [t.double().requires_grad_(True) for t in (X, Wg, Wu, Wd)]
    x, g, u, d = leaves
    gate, up = x @ g.T, x @ u.T
    a = f.silu(gate) if act == rl.ACT_SILU else f.gelu(gate)
    h = a * up
    y = h @ d.T
    dy = dY.double()
    slope, = torch.autograd.grad(a.sum(), gate, retain_graph=True)
    grads = torch.autograd.grad(y, leaves, dy)
    with torch.no_grad():
        dh = dy @ d
        dg2 = ((dh * up).abs() * (slope.abs() + 1)).square()
        du2 = (dh.abs() * (a.abs() + (gate * slope).abs())).square()
        x2, g2, u2, d2, h2 = (t.square() for t in (x, g, u, d, h))
        scales = [s.sqrt() for s in (h2 @ d2.T, dg2 @ g2 + du2 @ u2, dg2.T @ x2, du2.T @ x2, dy.square().T @ h2)]
    return [(r.detach(), s) for r, s in zip((y,) + grads, scales)]


def check_normal(got, ref, K, what):
    """One rounding of the operands (H, or dG and dU); the output's own is at most 2^-8 of it."""
    ref, scale = ref
    err = (got.double() - ref).abs()
    share = H_STEP * math.sqrt(1 / 3) * (1 + 2.0 ** -6) + K * 2.0 ** -23
    worst = (err - H_STEP * ref.abs() - 6 * share * scale).max().item()
    assert worst <= 0, f"{what}: off by {worst:.2e} beyond six standard deviations"
    # all elements together: twice what is expected of them, as few tokens make the roundings' shares unequal
    bound = 2 * (share ** 2 * scale.square().sum() + H_STEP ** 2 / 3 * ref.square().sum()).sqrt()
    assert err.norm() <= bound, f"{what}: error {err.norm():.3e}, bound {bound:.3e}"


@pytest.mark.parametrize("act", [rl.ACT_SILU, rl.ACT_GELU])
@pytest.mark.parametrize("size", [(1, 520, 1288), (4, 2056, 776), (13, 264, 1032), (40, 1032, 392), (300, 520, 1160),
                                  (1100, 776, 2056), (50, 2312, 776)], ids=str)
def test_normal_inputs(size, act):
    M, D, F = size
    gen = torch.Generator(device="cuda").manual_seed(M)
    def new(*shape, scale=1.0):
        return (scale * torch.randn(*shape, device="cuda", generator=gen)).bfloat16()
    X, dY = new(M, D), new(M, D)
    Wg, Wu, Wd = new(F, D, scale=D ** -0.5), new(F, D, scale=D ** -0.5), new(D, F, scale=F ** -0.5)
    ref = reference(X, Wg, Wu, Wd, dY, act)
    y, saved = rl.gated_mlp(X, Wg, Wu, Wd, act=act, save=True)
    check_normal(y, ref[0], D + F, "Y")
    assert torch.equal(y, rl.gated_mlp(X, Wg, Wu, Wd, act=act))
    grads = rl.gated_mlp_backward(dY, X, Wg, Wu, Wd, saved, act=act)
    for got, want, K, name in zip(grads, ref[1:], (D + 2 * F, D + M, D + M, D + M),
                                  ("dX", "dW_gate", "dW_up", "dW_down")):
        check_normal(got, want, K, name)
    again = rl.gated_mlp_backward(dY, X, Wg, Wu, Wd, saved, act=act)
    assert all(torch.equal(a, b) for a, b in zip(grads, again))


@pytest.mark.parametrize("act", [rl.ACT_SILU, rl.ACT_GELU])
def test_gradients_against_differences(act):
    """A central difference of the 64-bit block along the gradient's own direction: <dY, Y(t) - Y(-t)> / 2 t = |grad|^2,
    off by the roundings' sqrt(2 / 3) 2^-8 < 0.4% and t^2 terms of less than that."""
    M, D, F = 40, 136, 264
    gen = torch.Generator(device="cuda").manual_seed(8)
    def new(*shape, scale=1.0):
        return (scale * torch.randn(*shape, device="cuda", generator=gen)).bfloat16()
    X, dY = new(M, D), new(M, D)
    W = [new(F, D, scale=D ** -0.5), new(F, D, scale=D ** -0.5), new(D, F, scale=F ** -0.5)]
    _, saved = rl.gated_mlp(X, *W, act=act, save=True)
    grads = rl.gated_mlp_backward(dY, X, *W, saved, act=act)
    f = torch.nn.functional

    def loss(x, g, u, d):
        a = f.silu(x @ g.T) if act == rl.ACT_SILU else f.gelu(x @ g.T)
        return (((a * (x @ u.T)) @ d.T) * dY.double()).sum().item()

    point = [t.double() for t in (X, *W)]
    for i, grad in enumerate(grads):
        v = grad.double() / grad.double().norm()
        t = 1e-3
        up = [p + t * v if j == i else p for j, p in enumerate(point)]
        down = [p - t * v if j == i else p for j, p in enumerate(point)]
        numeric = (loss(*up) - loss(*down)) / (2 * t)
        assert abs(numeric - grad.double().norm().item()) <= 0.01 * abs(numeric)


def test_activation_over_its_range():
    """One channel each for gate and up, so that H is the activation itself: against 64 bits over all magnitudes."""
    values = torch.cat([torch.linspace(-30, 30, 4001), torch.tensor([0.0, -0.0, 1e-30, -1e-30, 300.0, -300.0, 1e30])])
    x = values.bfloat16().cuda()
    M = x.numel()
    X = torch.zeros(M, 8, dtype=torch.bfloat16, device="cuda")
    X[:, 0] = x
    X[:, 1] = 1
    Wg = torch.zeros(8, 8, dtype=torch.bfloat16, device="cuda")
    Wu = torch.zeros_like(Wg)
    Wg[:, 0] = 1
    Wu[:, 1] = 1
    Wd = torch.eye(8, dtype=torch.bfloat16, device="cuda")
    for act, fn in ((rl.ACT_SILU, torch.nn.functional.silu), (rl.ACT_GELU, torch.nn.functional.gelu)):
        xd = x.double().requires_grad_(True)
        ref = fn(xd)
        slope, = torch.autograd.grad(ref.sum(), xd)
        y, saved = rl.gated_mlp(X, Wg, Wu, Wd, act=act, save=True)
        # the formula's 1.5e-7 (GELU) times |x|, a few 32-bit steps, and the rounding
        tol = H_STEP * ref.detach().abs() + 2e-7 * x.double().abs().clamp(max=30) + 2.0 ** -22 * ref.detach().abs()
        assert ((saved[3][:, 0].double() - ref.detach()).abs() <= tol).all()
        dX = rl.gated_mlp_backward(torch.ones_like(y) / 8, X, Wg, Wu, Wd, saved, act=act)[0]
        # dH = 1/8, eight equal channels: dX[:, 0] is the slope, rounded in dG and again in dX
        tol = 2 * H_STEP * slope.abs() * (1 + H_STEP) + 1e-6
        assert ((dX[:, 0].double() - slope).abs() <= tol).all()


def test_saturated_rows_and_nan_stay_in_their_row():
    M, D, F = 300, 72, 136
    gen = torch.Generator(device="cuda").manual_seed(1)
    X = torch.randn(M, D, device="cuda", generator=gen).bfloat16()
    W = [torch.randn(s, device="cuda", generator=gen).bfloat16() for s in ((F, D), (F, D), (D, F))]
    want = rl.gated_mlp(X, *W)
    X2 = X.clone()
    X2[7, 3] = math.nan
    X2[131] = math.inf
    got = rl.gated_mlp(X2, *W)
    rows = torch.ones(M, dtype=torch.bool, device="cuda")
    rows[7] = rows[131] = False
    assert torch.equal(got[rows], want[rows]) and got[7].isnan().all()


@pytest.mark.parametrize("act", [rl.ACT_SILU, rl.ACT_GELU])
@pytest.mark.parametrize("M,D", [(1, 264), (12, 264), (200, 264), (40, 2056)])
def test_sparse_down_projection(act, M, D):
    """mode_down = sparse runs the same layer as rl.linear on the same H."""
    F, R = 520, 16
    gen = torch.Generator(device="cuda").manual_seed(M)
    def new(*shape, scale=1.0):
        return (scale * torch.randn(*shape, device="cuda", generator=gen)).bfloat16()
    X, LA, LB = new(M, D), new(D, R, scale=0.1), new(R, F, scale=0.1)
    W = new(F, D, scale=D ** -0.5), new(F, D, scale=D ** -0.5), new(D, F, scale=F ** -0.5)
    for la, lb in ((None, None), (LA, LB)):
        y, (_, _, _, H) = rl.gated_mlp(X, *W, act=act, L_A=la, L_B=lb, mode_down=rl.MODE_SPARSE, save=True)
        assert torch.equal(y, rl.linear(H, W[2], la, lb, mode=rl.MODE_SPARSE))


@pytest.mark.parametrize("M,D,F", [(1, 264, 520), (9, 264, 520), (70, 264, 520), (140, 264, 520), (140, 2056, 4104),
                                   (300, 1032, 2056)])
def test_other_stream_and_captured_graph(M, D, F):
    gen = torch.Generator(device="cuda").manual_seed(3)
    def new(*shape):
        return torch.randn(*shape, device="cuda", generator=gen).bfloat16()
    X, dY = new(M, D), new(M, D)
    W = new(F, D), new(F, D), new(D, F)

    def step(stream=None):
        y, saved = rl.gated_mlp(X, *W, save=True, stream=stream)
        return (y,) + rl.gated_mlp_backward(dY, X, *W, saved, stream=stream)

    want = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, int(side.cuda_stream)):
        got = step(stream)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step())
        graphs.append(g)
    X.copy_(new(M, D))
    want = step()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(4):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for out in outs:
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    assert rl.rtlynx_stream_status() == rl.OK


@pytest.mark.parametrize("size", [(5, 72, 136), (150, 136, 264), (70, 136, 4104), (70, 2056, 136)], ids=str)
def test_nothing_else_is_written(size):
    """Guard rows around every output stay as they were."""
    M, D, F = size
    def guarded(rows, cols):
        buf = torch.full((rows + 512, cols), 7.0, dtype=torch.bfloat16, device="cuda")
        return buf, buf[256:256 + rows]
    gen = torch.Generator(device="cuda").manual_seed(3)
    def new(*shape):
        return torch.randn(*shape, device="cuda", generator=gen).bfloat16()
    X, dY = new(M, D), new(M, D)
    W = new(F, D), new(F, D), new(D, F)
    bufs = [guarded(M, F) for _ in range(4)] + [guarded(M, D)]
    G, U, low, H, Y = (b[1] for b in bufs)
    n = rl.rtlynx_gated_mlp_block_workspace_size(M, D, F)
    ws = torch.full((n + 4096,), 7, dtype=torch.uint8, device="cuda")
    rl.rtlynx_gated_mlp_block(X, *W, None, None, G, U, low, H, Y, M, D, F, 0, rl.ACT_SILU, rl.MODE_DENSE_SKIP, ws, n)
    assert (ws[n:] == 7).all()
    grads = [guarded(M, D), guarded(F, D), guarded(F, D), guarded(D, F)]
    n = rl.rtlynx_gated_mlp_backward_workspace_size(M, D, F)
    ws = torch.full((n + 4096,), 7, dtype=torch.uint8, device="cuda")
    rl.rtlynx_gated_mlp_backward(dY, X, *W, G, U, low, H, *(b[1] for b in grads), M, D, F, rl.ACT_SILU, ws, n)
    for buf, inner in bufs + grads:
        assert (buf[:256] == 7).all() and (buf[256 + inner.shape[0]:] == 7).all()
        assert inner is low or torch.isfinite(inner).all()
    assert (ws[n:] == 7).all()


def test_refusals_on_the_gpu():
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(128, 64, dtype=torch.bfloat16, device="cuda")
    d = torch.zeros(64, 128, dtype=torch.bfloat16, device="cuda")
    for args in ((x.half(), w, w, d), (x, w, w.T, d), (x, w, w, w), (x, w[:, ::2], w, d)):
        with pytest.raises(ValueError):
            rl.gated_mlp(*args)
    with pytest.raises(rl.RtlynxError):
        rl.gated_mlp(x, w, w, d, out=x)
    with pytest.raises(rl.RtlynxError):
        rl.gated_mlp(x, w, w, d, act=9)
