"""The gated block's activations far out, where their values are small: relative errors of H and of the slopes.

Tolerances: the tail of the normal distribution to 1e-4 of itself; exp(-x^2 / 2), whose argument (at most 86) is off by
2^-23 of itself and again by 2^-24 in the change of base, by less than 2e-5; a rounding to bf16, and a second one of dG in
dX.  Below 2^-126 numbers may go to zero."""
import pytest
import torch

import activation_sparse_gemm_b200 as rl

pytestmark = pytest.mark.gpu

HALF_STEP = 2.0 ** -8
SMALLEST = 2.0 ** -126


def run(x, act, rows):
    """H and dX of one channel whose G is x and whose U is 1, in calls of `rows` tokens."""
    hs, slopes = [], []
    W = torch.zeros(8, 8, dtype=torch.bfloat16, device="cuda")
    Wg, Wu = W.clone(), W.clone()
    Wg[0, 0] = Wu[0, 1] = 1
    Wd = torch.eye(8, dtype=torch.bfloat16, device="cuda")
    for part in x.split(rows):
        X = torch.zeros(rows, 8, dtype=torch.bfloat16, device="cuda")
        X[:part.numel(), 0] = part
        X[:, 1] = 1
        y, saved = rl.gated_mlp(X, Wg, Wu, Wd, act=act, save=True)
        hs.append(saved[3][:part.numel(), 0])
        slopes.append(rl.gated_mlp_backward(torch.ones_like(y), X, Wg, Wu, Wd, saved, act=act)[0][:part.numel(), 0])
    return torch.cat(hs).double(), torch.cat(slopes).double()


@pytest.mark.parametrize("rows", [8, 40, 600], ids=lambda n: f"{n}tokens")
@pytest.mark.parametrize("act,lowest", [(rl.ACT_GELU, -13.0), (rl.ACT_SILU, -85.0)])
def test_relative_error_of_the_tail(act, lowest, rows):
    x = torch.linspace(lowest, -1.5, 600, device="cuda").bfloat16()
    xd = x.double().requires_grad_(True)
    # erfc and not erf, which leaves nothing of a small tail
    ref = xd * 0.5 * torch.special.erfc(-xd * 0.5 ** 0.5) if act == rl.ACT_GELU else xd / (1 + torch.exp(-xd))
    slope, = torch.autograd.grad(ref.sum(), xd)
    ref = ref.detach()
    H, dX = run(x, act, rows)
    own = 1.2e-4 + 2e-5
    assert ((H - ref).abs() <= (HALF_STEP + own) * ref.abs() + SMALLEST).all()
    # the slope is the sum of two terms of opposite signs, each as far off as above
    terms = (ref / xd.detach()).abs() + (slope - ref / xd.detach()).abs()
    assert ((dX - slope).abs() <= 2 * HALF_STEP * (1 + HALF_STEP) * slope.abs() + own * terms + SMALLEST).all()
