"""The operators together, as a transformer block uses them: qkv layer, norm and
rotation of queries and keys in place in its packed output, attention (plain),
output layer, gated feed-forward block; forward, and the gradient back to the
input through every one of them, against the same block in 64 bits.

Tolerance: along the longest path (qkv, norm and rotation, attention's output,
output layer and residual, H, Y and residual) a value passes about nine
roundings of at most 2^-8 of something no larger than the norm of what it joins,
each uniform, so independent ones add up to sqrt(9 / 3) 2^-8 of the output's
norm; a factor of two allows for their being passed on unevenly.  The gradient
passes the same places once more on its way back."""
import math

import pytest
import torch

import activation_sparse_gemm_b200 as rl

pytestmark = pytest.mark.gpu

EPS = 1e-6


def attention(q, k, v):
    """q [S, H, d], k and v [S, Hk, d], every query head with its group's keys, in their own type."""
    group = q.shape[1] // k.shape[1]
    k, v = k.repeat_interleave(group, 1), v.repeat_interleave(group, 1)
    scores = torch.einsum("shd,thd->hst", q, k) / math.sqrt(q.shape[-1])
    return torch.einsum("hst,thd->shd", scores.softmax(-1), v)


def rotate(x, angle):
    c, s = angle.cos()[:, None], angle.sin()[:, None]
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)


def reference(x, p, positions, axes, sizes):
    S, H, Hk, d = sizes
    angle = torch.cat([positions[:, a, None].double() * torch.tensor(
        [10000.0 ** (-2.0 * j / n) for j in range(n // 2)], dtype=torch.float64, device=x.device)
        for a, n in enumerate(axes)], -1)
    qkv = (x @ p["qkv"].T).view(S, H + 2 * Hk, d)
    q, k, v = qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:]

    def norm(t, w):
        return rotate(t * (t.square().mean(-1, keepdim=True) + EPS).rsqrt() * w, angle)

    y = x + attention(norm(q, p["w_q"]), norm(k, p["w_k"]), v).reshape(S, H * d) @ p["out"].T
    gate = y @ p["gate"].T
    return y + (torch.nn.functional.silu(gate) * (y @ p["up"].T)) @ p["down"].T


@pytest.mark.parametrize("S,H,Hk,d,F,axes", [
    (1, 4, 4, 64, 520, (16, 24, 24)),      # one token
    (13, 6, 2, 72, 776, (8, 32, 32)),      # few tokens, grouped keys, a head of 72
    (301, 4, 4, 128, 1032, (44, 42, 42)),  # the video workload's axes
])
def test_block_forward_and_backward(S, H, Hk, d, F, axes):
    D = H * d
    gen = torch.Generator(device="cuda").manual_seed(S)

    def new(*shape, scale=1.0):
        return (scale * torch.randn(*shape, device="cuda", generator=gen)).bfloat16()

    p = {"qkv": new((H + 2 * Hk) * d, D, scale=D ** -0.5), "out": new(D, D, scale=D ** -0.5),
         "gate": new(F, D, scale=D ** -0.5), "up": new(F, D, scale=D ** -0.5), "down": new(D, F, scale=F ** -0.5),
         "w_q": (1 + 0.2 * torch.randn(d, device="cuda", generator=gen)).bfloat16(),
         "w_k": (1 + 0.2 * torch.randn(d, device="cuda", generator=gen)).bfloat16()}
    x, dy = new(S, D), new(S, D)
    positions = torch.stack([torch.arange(S, device="cuda") % (3 + a) + a for a in range(3)], -1).int()
    plan = rl.Rope(axes)

    # forward
    qkv = rl.linear(x, p["qkv"], mode=rl.MODE_DENSE_SKIP).view(S, H + 2 * Hk, d)
    q, k, v = qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:]
    before = qkv.clone()
    rl.qk_norm_rope(q, k, p["w_q"], p["w_k"], positions, plan, eps=EPS, out=(q, k))
    assert torch.equal(v, before[:, H + Hk:])
    turned = [t.float().requires_grad_(True) for t in (q, k, v)]
    mixed = attention(*turned)
    attn = mixed.detach().reshape(S, D).bfloat16()
    mid = x + rl.linear(attn, p["out"], mode=rl.MODE_DENSE_SKIP)
    ff, saved = rl.gated_mlp(mid, p["gate"], p["up"], p["down"], save=True)
    y = mid + ff

    # backward: dy reaches mid directly and through the feed-forward block
    d_ff = rl.gated_mlp_backward(dy, mid, p["gate"], p["up"], p["down"], saved)
    d_mid = (dy.float() + d_ff[0].float()).bfloat16()
    d_attn = rl.linear(d_mid, p["out"].T.contiguous(), mode=rl.MODE_DENSE_SKIP)
    dq, dk, dv = (g.bfloat16().contiguous() for g in torch.autograd.grad(mixed, turned, d_attn.float().view_as(mixed)))
    d_qkv = torch.empty_like(qkv)
    d_qkv[:, H + Hk:] = dv
    _, _, dw_q, dw_k = rl.qk_norm_rope_backward(dq, dk, before[:, :H], before[:, H:H + Hk], p["w_q"], p["w_k"],
                                                positions, plan, eps=EPS, out=(d_qkv[:, :H], d_qkv[:, H:H + Hk]))
    dx = d_mid.float() + rl.linear(d_qkv.view(S, -1), p["qkv"].T.contiguous(), mode=rl.MODE_DENSE_SKIP).float()

    leaves = {n: t.double().requires_grad_(True) for n, t in p.items()}
    x64 = x.double().requires_grad_(True)
    y64 = reference(x64, leaves, positions, axes, (S, H, Hk, d))
    names = ("gate", "up", "down", "w_q", "w_k")
    grads = torch.autograd.grad(y64, [x64] + [leaves[n] for n in names], dy.double())

    def close(got, want, roundings, what):
        rel = ((got.double() - want).norm() / want.norm()).item()
        assert rel <= 2 * math.sqrt(roundings / 3) * 2.0 ** -8, f"{what}: {rel:.2e}"

    close(y, y64.detach(), 9, "y")
    close(dx, grads[0], 18, "dx")
    if S > 1:  # one token's attention does not depend on its queries and keys: their gradients are zero
        close(dw_q, grads[4], 18, "dw_q")
        close(dw_k, grads[5], 18, "dw_k")
    for got, want, name in zip(d_ff[1:], grads[1:4], names):
        close(got, want, 12, "d" + name)
    assert rl.rtlynx_stream_status() == rl.OK


@pytest.mark.parametrize("M", [1, 12, 60, 200])
def test_forked_and_joined_streams_in_a_graph(M):
    """Calls on two streams that fork and join inside a captured graph, behind copies, replayed with new inputs: the
    kernels' early launches may not outrun what they read, weights included."""
    D, F, H, d = 264, 4104, 3, 88
    gen = torch.Generator(device="cuda").manual_seed(M)

    def new(*shape, scale=1.0):
        return (scale * torch.randn(*shape, device="cuda", generator=gen)).bfloat16()

    fresh = [new(M, D), new(F, D, scale=D ** -0.5), new(F, D, scale=D ** -0.5), new(D, F, scale=F ** -0.5), new(M, D)]
    held = [torch.zeros_like(t) for t in fresh]
    w = new(d)
    positions = torch.arange(M, device="cuda")[:, None]
    plan = rl.Rope((d,), pairing=rl.ROPE_HALF)
    side = torch.cuda.Stream()

    def step():
        for a, b in zip(held, fresh):  # inputs and weights written right before the calls that read them
            a.copy_(b)
        x, gate, up, down, dy = held
        q = x.view(M, H, d)
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        with torch.cuda.stream(side):
            turned, _ = rl.qk_norm_rope(q, None, w, None, positions, plan)
            y2 = rl.gated_mlp(turned.view(M, D), gate, up, down, act=rl.ACT_GELU)
        y, saved = rl.gated_mlp(x, gate, up, down, save=True)
        here.wait_stream(side)
        grads = rl.gated_mlp_backward(dy + y2, x, gate, up, down, saved)
        back = rl.qk_norm_rope_backward(grads[0].view(M, H, d), None, q, None, w, None, positions, plan)
        return (y, y2) + grads + (back[0], back[2])

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(3):
        for t in fresh:
            t.copy_(torch.randn(t.shape, device="cuda", generator=gen) * t.float().std())
        want = [t.clone() for t in step()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    assert rl.rtlynx_stream_status() == rl.OK
