"""The gated block where a CTA pair takes several tiles, and at the widths of real models.

A pair has two accumulators, so only its third tile waits for one that the epilogue has handed back: the sizes here give
every launch of the tiled kernel three or more 256 x 256 tiles a pair (74 pairs), with main loops shorter and longer than
the epilogue, and ragged edges.  Whole numbers, as in test_gpu_gated.py: one misplaced element shows."""
import math

import pytest
import torch

import activation_sparse_gemm_b200 as rl
from tests.test_gpu_gated import H_STEP, check_exact, dev, ints, reference, rounded, whole_number_inputs

pytestmark = pytest.mark.gpu

# gate and up: tiles of 256 x 128 columns; dH: 256 x 256
SIZES = [
    (2900, 72, 6152),   # 588 tiles of 2 stages; dH 300 of 2
    (4500, 264, 5000),  # 720 of 5; dH 360 of 5
    (2309, 1096, 5000),  # 400 of 18; dH 200 of 18
    (4500, 2056, 264),  # down-projection: 162 tiles of 5 stages
]


def check(got, ref, what):
    check_exact(got, ref.cpu(), what)


@pytest.mark.parametrize("act", [rl.ACT_SILU, rl.ACT_GELU])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_forward_many_tiles(size, act):
    M, D, F = size
    gen, X, Wg, Wu = whole_number_inputs(M, D, F, M + D)
    Wd = ints(gen, (D, F), -1, 1, 0.5)
    x, g, u, d = (t.cuda() for t in (X, Wg, Wu, Wd))
    G, U = x @ g.T, x @ u.T
    assert G.min() >= 32 and G.max() < 256
    H = rounded(G * U)
    args = dev(X), dev(Wg), dev(Wu), dev(Wd)
    y, saved = rl.gated_mlp(*args, act=act, save=True)
    check(y, H @ d.T, "Y")
    for got, ref, name in zip(saved, (G, U, 0 * G, H), ("G", "U", "low", "H"), strict=True):
        assert torch.equal(got.double(), ref), name
    assert torch.equal(rl.gated_mlp(*args, act=act), y)
    assert rl.rtlynx_stream_status() == rl.OK


@pytest.mark.parametrize("size", SIZES, ids=str)
def test_backward_many_tiles(size):
    M, D, F = size
    gen = torch.Generator().manual_seed(M * 7 + F)
    X = ints(gen, (M, D), -2, 2, 1.0)
    Wg, Wu, Wd = ints(gen, (F, D), -2, 2, 1.0), ints(gen, (F, D), -2, 2, 1.0), ints(gen, (D, F), -1, 1, 1.0)
    dY = ints(gen, (M, D), -1, 1, min(1.0, 2 / D))
    G = 32.0 * torch.randint(1, 3, (M, F), generator=gen).double()
    U, H = ints(gen, (M, F), -2, 2, 1.0), ints(gen, (M, F), -3, 3, 1.0)
    x, g, u, d, dy, gate, up, h = (t.cuda() for t in (X, Wg, Wu, Wd, dY, G, U, H))
    dH = dy @ d
    dG, dU = rounded(dH * up), rounded(dH * gate)
    ref = (dG @ g + dU @ u, dG.T @ x, dU.T @ x, dy.T @ h)
    saved = dev(G), dev(U), torch.zeros(M, F, dtype=torch.int16, device="cuda"), dev(H)
    got = rl.gated_mlp_backward(dev(dY), dev(X), dev(Wg), dev(Wu), dev(Wd), saved)
    for a, b, name in zip(got, ref, ("dX", "dW_gate", "dW_up", "dW_down")):
        check(a, b, name)
    assert rl.rtlynx_stream_status() == rl.OK


def accumulation(X, Wg, Wu, Wd, dY, act):
    """How far 32-bit accumulation of G, U and dH can move Y, dX and the weights' gradients, element by element.

    test_gpu_gated.py counts it as a share K 2^-23 of an output's own terms.  That leaves out what is small because long
    sums before it cancel: with one token a weight's gradient is a single product, and where its U (or G, or dH), a sum of
    5120 terms whose squares' root is 1, happens to be 1e-4, the sum's 1e-6 is a hundredth of it (2.6e-7 past that
    tolerance at 5120 -> 13824, one token).  So: each of the D additions of such a sum is off by at most 2^-23 of the
    partial sum, a walk whose size is 0.53 r on average over its D steps, r the root of the terms' squares; D 2^-23 r is
    twice that, taken as if all had one sign.  By the product rule, with |act''| < 0.8, this gives H, dG and dU an
    error each, and independent ones of an output's terms add up to the root of their squares."""
    f = torch.nn.functional
    x, g, u, d, dy = (t.double() for t in (X, Wg, Wu, Wd, dY))
    share = x.shape[1] * 2.0 ** -23
    gate = (x @ g.T).requires_grad_(True)
    a = f.silu(gate) if act == rl.ACT_SILU else f.gelu(gate)
    slope = torch.autograd.grad(a.sum(), gate)[0].abs()
    a, up, dh = a.detach().abs(), (x @ u.T).abs(), (dy @ d).abs()
    x2, g2, u2, d2, dy2 = (t.square() for t in (x, g, u, d, dy))
    e_gate, e_up, e_dh = (share * t.sqrt() for t in (x2 @ g2.T, x2 @ u2.T, dy2 @ d2))
    h2 = (slope * up * e_gate + a * e_up).square()
    du2 = (a * e_dh + dh * slope * e_gate).square()
    dg2 = (up * slope * e_dh + dh * slope * e_up + 0.8 * dh * up * e_gate).square()
    return [t.sqrt() for t in (h2 @ d2.T, dg2 @ g2 + du2 @ u2, dg2.T @ x2, du2.T @ x2, dy2.T @ h2)]


def check_sums(got, ref, moved, K, what):
    """check_normal with the accumulation before the last sum: six standard deviations of both together."""
    ref, scale = ref
    share = H_STEP * math.sqrt(1 / 3) * (1 + 2.0 ** -6) + K * 2.0 ** -23
    err = (got.double() - ref).abs()
    spread = ((share * scale).square() + moved.square()).sqrt()
    worst = (err - H_STEP * ref.abs() - 6 * spread).max().item()
    assert worst <= 0, f"{what}: off by {worst:.2e} beyond six standard deviations"
    bound = 2 * (spread.square().sum() + H_STEP ** 2 / 3 * ref.square().sum()).sqrt()
    assert err.norm() <= bound, f"{what}: error {err.norm():.3e}, bound {bound:.3e}"


@pytest.mark.parametrize("M,D,F,act", [
    (1, 5120, 13824, rl.ACT_SILU), (16, 5120, 13824, rl.ACT_SILU), (200, 5120, 13824, rl.ACT_GELU),
    (4096, 5120, 13824, rl.ACT_SILU), (2047, 1544, 4104, rl.ACT_GELU), (11, 2056, 5512, rl.ACT_GELU)])
def test_normal_numbers_at_real_widths(M, D, F, act):
    gen = torch.Generator(device="cuda").manual_seed(M)

    def new(*shape, scale=1.0):
        return (scale * torch.randn(*shape, device="cuda", generator=gen)).bfloat16()

    X, dY = new(M, D), new(M, D)
    W = new(F, D, scale=D ** -0.5), new(F, D, scale=D ** -0.5), new(D, F, scale=F ** -0.5)
    ref = reference(X, *W, dY, act)
    out = torch.empty_like(X)
    y, saved = rl.gated_mlp(X, *W, act=act, save=True, out=out)
    assert y.data_ptr() == out.data_ptr()
    grads = rl.gated_mlp_backward(dY, X, *W, saved, act=act)
    moved = accumulation(X, *W, dY, act)
    for got, want, by, K, name in zip((out,) + grads, ref, moved, (D + F, D + 2 * F, D + M, D + M, D + M),
                                      ("Y", "dX", "dW_gate", "dW_up", "dW_down")):
        check_sums(got, want, by, K, name)
    assert rl.rtlynx_stream_status() == rl.OK


def test_output_given():
    """out receives what the call returns; one that is not Y's shape, type or place is refused."""
    M, D, F = 37, 136, 264
    gen = torch.Generator(device="cuda").manual_seed(1)
    X = torch.randn(M, D, device="cuda", generator=gen).bfloat16()
    W = [torch.randn(s, device="cuda", generator=gen).bfloat16() for s in ((F, D), (F, D), (D, F))]
    want = rl.gated_mlp(X, *W)
    buf = torch.full((M + 2, D), 7.0, dtype=torch.bfloat16, device="cuda")
    got = rl.gated_mlp(X, *W, out=buf[1:-1])
    assert got.data_ptr() == buf[1:-1].data_ptr() and torch.equal(buf[1:-1], want)
    assert (buf[0] == 7).all() and (buf[-1] == 7).all()
    for bad in (torch.empty(M, D + 8, dtype=torch.bfloat16, device="cuda")[:, :D], buf, buf[1:-1].float(), want.cpu(),
                torch.empty(D, M, dtype=torch.bfloat16, device="cuda").T):
        with pytest.raises(ValueError):
            rl.gated_mlp(X, *W, out=bad)
    for bad in (X, W[2][:M].view(-1)[:M * D].view(M, D)):
        with pytest.raises(rl.RtlynxError):
            rl.gated_mlp(X, *W, out=bad)


def test_hidden_arrays_beyond_32_bits():
    """H, G, U, dG and dU of more than 2^31 elements: the rows past that point are what a call on them alone gives.
    Whole numbers, so that both are exact whatever the kernel."""
    M, D, F, part = 530000, 8, 4104, 300
    assert (M - part) * F > 1 << 31
    gen, X, Wg, Wu = whole_number_inputs(part, D, F, 5)
    W = dev(Wg), dev(Wu), dev(ints(gen, (D, F), -1, 1, 0.5))
    last, dY = dev(X), dev(ints(gen, (part, D), -1, 1, 0.25))
    many = last.repeat(-(-M // part), 1)[:M].contiguous()
    many[-part:] = last
    far = torch.zeros_like(many)
    far[-part:] = dY
    want, kept = rl.gated_mlp(last, *W, save=True)
    got, saved = rl.gated_mlp(many, *W, save=True)
    assert torch.equal(got[-part:], want)
    for a, b in zip(saved, kept):
        assert torch.equal(a[-part:], b)
    grads = rl.gated_mlp_backward(far, many, *W, saved)
    ref = rl.gated_mlp_backward(dY, last, *W, kept)
    assert torch.equal(grads[0][-part:], ref[0]) and not grads[0][:-part].any()
    for a, b in zip(grads[1:], ref[1:]):
        assert torch.equal(a, b)
    assert rl.rtlynx_stream_status() == rl.OK
