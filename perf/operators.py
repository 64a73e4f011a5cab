"""The operators around a transformer block's linear layers: what is timed, on which inputs, and their plain forms.

Operators and their entry points in the package (``own`` selects them):

  rope          rotary positions with several axes:        rl.rope, rl.rope_backward
  norm_rope     RMS norm of each query and key head, then
                the rotation, in one pass:                 rl.qk_norm_rope, rl.qk_norm_rope_backward
  gated         gated feed-forward block
                Y = (act(X Wg^T) * (X Wu^T)) Wd^T:          rl.gated_mlp, rl.gated_mlp_backward

Where ``own`` is false ``run`` computes the same in elementary torch operations, in 32 bits (rotation angles in 64),
rounded once at the end.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases
def _heads(name, op, direction, dtype, batch, tokens, heads_q, heads_k, dim, axes, pairing, theta, layout, far=0):
    return {"name": name, "op": op, "direction": direction, "dtype": dtype, "batch": batch, "tokens": tokens,
            "heads_q": heads_q, "heads_k": heads_k, "dim": dim, "axes": axes, "pairing": pairing, "theta": theta,
            "layout": layout, "far": far}


def _gated(name, direction, tokens, width, hidden, act):
    return {"name": name, "op": "gated", "direction": direction, "tokens": tokens, "width": width, "hidden": hidden,
            "act": act}


def listed():
    return [
        # --- rotary positions alone
        # every query and key of a 21 x 30 x 52 video latent (32760 tokens, 40 heads of 128: the width of the video
        # workload), read in place from the packed output of the qkv layer
        _heads("rope_video", "rope", "forward", "bf16", 1, 32760, 40, 40, 128, "44,42,42", "interleaved", 10000.0,
               "packed"),
        # the gradient of the same rotation in a training step: two sequences, heads-first layout, grouped keys,
        # half-split pairs, an odd number of tokens and only part of each head rotated
        _heads("rope_grad_half", "rope", "backward", "fp16", 2, 4099, 32, 8, 96, "16,24,24", "half", 10000.0,
               "heads_first"),
        # --- norm and rotation
        # one token at a time for a batch of four, far into a long sequence: a launch's latency
        _heads("norm_rope_token", "norm_rope", "forward", "bf16", 4, 1, 40, 8, 128, "128", "half", 1000000.0, "packed",
               1 << 22),
        # the queries and keys of the video workload
        _heads("norm_rope_video", "norm_rope", "forward", "bf16", 1, 32760, 40, 40, 128, "44,42,42", "interleaved",
               10000.0, "packed"),
        # an image's joint text and image sequence in 32 bits, odd token count, head size of 72
        _heads("norm_rope_fp32", "norm_rope", "forward", "fp32", 1, 4301, 16, 16, 72, "8,32,32", "interleaved", 256.0,
               "plain"),
        # the gradient of the norm and the rotation in a training step, with the weights' gradients
        _heads("norm_rope_grad", "norm_rope", "backward", "bf16", 2, 8192, 40, 40, 128, "32,48,48", "interleaved", 256.0,
               "packed"),
        # --- gated feed-forward block
        # one token: the weights are read once, nothing else counts (5120 and 13824: the video workload's widths)
        _gated("gated_token", "forward", 1, 5120, 13824, "silu"),
        # a handful of tokens, ragged widths
        _gated("gated_few_tokens", "forward", 11, 2056, 5512, "gelu"),
        # the tiny workload's tokens and width
        _gated("gated_tiny", "forward", 128, 256, 512, "silu"),
        # all tokens of the video workload
        _gated("gated_video", "forward", 32760, 5120, 13824, "silu"),
        # a training step on an odd number of tokens at ragged widths
        _gated("gated_train_ragged", "train", 2047, 1544, 4104, "gelu"),
        # a training step at the video workload's widths
        _gated("gated_train", "train", 8192, 5120, 13824, "silu"),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["rope", "norm_rope", "gated"])
    if op == "gated":
        direction = rng.choice(["forward", "forward", "train"])
        while True:
            tokens = _log(rng, 1, 32760)
            width = 8 * _log(rng, 16, 640)
            hidden = 8 * _log(rng, 32, 1728)
            flops = 6.0 * tokens * width * hidden * (3 if direction == "train" else 1)
            if flops <= 6.0 * 32760 * 5120 * 13824 * (0.7 if direction == "train" else 1.0):
                break
        case = _gated("", direction, tokens, width, hidden, rng.choice(["silu", "gelu"]))
    else:
        direction = rng.choice(["forward", "backward"])
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        pairing = rng.choice(["interleaved", "half"])
        dim = 8 * rng.choice([2, 4, 6, 8, 8, 9, 10, 12, 16, 16, 16, 24, 32])
        part = dim if rng.random() < 0.7 else 8 * rng.randint(1, dim // 8)
        n_axes = rng.randint(1, min(4, part // 2))
        cuts = sorted(rng.sample(range(1, part // 2), n_axes - 1)) if n_axes > 1 else []
        axes = ",".join(str(2 * (b - a)) for a, b in zip([0] + cuts, cuts + [part // 2]))
        while True:
            batch, tokens = rng.choice([1, 1, 2, 3, 5]), _log(rng, 1, 32760)
            heads_k = _log(rng, 1, 40)
            heads_q = heads_k * rng.choice([1, 1, 2, 4, 5])
            if batch * tokens * (heads_q + heads_k) * dim <= 32760 * 80 * 128 // (1 if dtype != "fp32" else 2):
                break
        case = _heads("", op, direction, dtype, batch, tokens, heads_q, heads_k, dim, axes, pairing,
                      rng.choice([256.0, 10000.0, 1000000.0]), rng.choice(["plain", "packed", "heads_first"]),
                      rng.choice([0, 0, 5000, 1 << 20, 1 << 24]))
    del case["name"]
    return case


# ------------------------------------------------------------------ inputs
def _axes(case):
    return [int(a) for a in case["axes"].split(",")]


def _positions(case, gen):
    """Grid coordinates of the tokens of each sequence, one column for each axis, from a start of the seed's own."""
    axes = len(_axes(case))
    batch, tokens = case["batch"], case["tokens"]
    side = max(1, int(round(tokens ** (1.0 / axes))))
    t = torch.arange(tokens, device="cuda")
    columns = []
    for _ in range(axes - 1):
        columns.append(t % (side + 3))
        t = t // (side + 3)
    columns.append(t)
    pos = torch.stack(columns[::-1], dim=-1)[None].expand(batch, tokens, axes)
    start = torch.randint(-8, 64, (batch, 1, axes), device="cuda", generator=gen)
    if case["far"]:
        start = start + torch.randint(case["far"] // 2, case["far"], (batch, 1, axes), device="cuda", generator=gen)
    return (pos + start).to(torch.int32).contiguous()


def _normal(gen, *shape, scale=1.0):
    return torch.randn(*shape, device="cuda", generator=gen, dtype=torch.float32) * scale


def _head_tensors(case, gen):
    """Queries and keys [batch, tokens, heads, dim], laid out as the case says; a few channels are much larger."""
    dtype = DTYPES[case["dtype"]]
    b, s, hq, hk, d = (case[k] for k in ("batch", "tokens", "heads_q", "heads_k", "dim"))
    gain = torch.ones(d, device="cuda")
    gain[torch.randperm(d, device="cuda", generator=gen)[: max(1, d // 16)]] = 6.0
    if case["layout"] == "packed":  # the qkv layer's output: queries, keys, values side by side
        qkv = torch.empty(b, s, hq + 2 * hk, d, device="cuda", dtype=dtype)
        for h in range(hq + 2 * hk):
            qkv[:, :, h] = (_normal(gen, b, s, d) * gain).to(dtype)
        return qkv[:, :, :hq], qkv[:, :, hq:hq + hk]
    if case["layout"] == "heads_first":
        q = (_normal(gen, b, hq, s, d) * gain).to(dtype).transpose(1, 2)
        k = (_normal(gen, b, hk, s, d) * gain).to(dtype).transpose(1, 2)
        return q, k
    return (_normal(gen, b, s, hq, d) * gain).to(dtype), (_normal(gen, b, s, hk, d) * gain).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    state = {"case": case}
    if case["op"] == "gated":
        m, d, f = case["tokens"], case["width"], case["hidden"]
        bf16 = torch.bfloat16
        state["X"] = _normal(gen, m, d).to(bf16)
        state["W_gate"] = _normal(gen, f, d, scale=d ** -0.5).to(bf16)
        state["W_up"] = _normal(gen, f, d, scale=d ** -0.5).to(bf16)
        state["W_down"] = _normal(gen, d, f, scale=f ** -0.5).to(bf16)
        if case["direction"] == "train":
            state["dY"] = _normal(gen, m, d, scale=0.1).to(bf16)
        if own:
            import activation_sparse_gemm_b200 as rl
            state["act"] = {"silu": rl.ACT_SILU, "gelu": rl.ACT_GELU}[case["act"]]
        return state
    dtype = DTYPES[case["dtype"]]
    state["q"], state["k"] = _head_tensors(case, gen)
    state["positions"] = _positions(case, gen)
    if case["op"] == "norm_rope":
        state["w_q"] = (1.0 + _normal(gen, case["dim"], scale=0.2)).to(dtype)
        state["w_k"] = (1.0 + _normal(gen, case["dim"], scale=0.2)).to(dtype)
        state["eps"] = 1e-6
    if case["direction"] == "backward":
        state["dq"], state["dk"] = _head_tensors(dict(case, layout="plain"), gen)
    if own:
        import activation_sparse_gemm_b200 as rl
        state["plan"] = rl.Rope(_axes(case), theta=case["theta"], pairing={
            "interleaved": rl.ROPE_INTERLEAVED, "half": rl.ROPE_HALF}[case["pairing"]])
    return state


# ------------------------------------------------------------------ one pass
def run(state):
    case = state["case"]
    if own:
        return _run_own(case, state)
    if case["op"] == "gated":
        return _plain_gated(case, state)
    return _plain_heads(case, state)


def _run_own(case, s):
    import activation_sparse_gemm_b200 as rl
    if case["op"] == "gated":
        weights = (s["W_gate"], s["W_up"], s["W_down"])
        if case["direction"] == "forward":
            return rl.gated_mlp(s["X"], *weights, act=s["act"])
        y, saved = rl.gated_mlp(s["X"], *weights, act=s["act"], save=True)
        return (y,) + tuple(rl.gated_mlp_backward(s["dY"], s["X"], *weights, saved, act=s["act"]))
    if case["op"] == "rope":
        if case["direction"] == "forward":
            return rl.rope(s["q"], s["k"], s["positions"], s["plan"])
        return rl.rope_backward(s["dq"], s["dk"], s["positions"], s["plan"])
    if case["direction"] == "forward":
        return rl.qk_norm_rope(s["q"], s["k"], s["w_q"], s["w_k"], s["positions"], s["plan"], eps=s["eps"])
    return rl.qk_norm_rope_backward(s["dq"], s["dk"], s["q"], s["k"], s["w_q"], s["w_k"], s["positions"], s["plan"],
                                    eps=s["eps"])


def _cos_sin(case, positions):
    """cos and sin [batch, tokens, 1, pairs] in 32 bits of angles in 64."""
    angles = []
    for a, dim in enumerate(_axes(case)):
        i = torch.arange(dim // 2, device="cuda", dtype=torch.float64)
        angles.append(positions[..., a, None].double() * case["theta"] ** (-2.0 * i / dim))
    angle = torch.cat(angles, dim=-1)[:, :, None, :]
    return torch.cos(angle).float(), torch.sin(angle).float()


def _rotate(case, x, cos, sin):
    part = 2 * cos.shape[-1]
    out = x.clone()
    if case["pairing"] == "interleaved":
        a, b = x[..., 0:part:2], x[..., 1:part:2]
        out[..., 0:part:2] = a * cos - b * sin
        out[..., 1:part:2] = a * sin + b * cos
    else:
        a, b = x[..., : part // 2], x[..., part // 2: part]
        out[..., : part // 2] = a * cos - b * sin
        out[..., part // 2: part] = a * sin + b * cos
    return out


def _plain_heads(case, s):
    dtype = DTYPES[case["dtype"]]
    cos, sin = _cos_sin(case, s["positions"])
    norm = case["op"] == "norm_rope"
    if case["direction"] == "forward":
        outs = []
        for x, w in ((s["q"], s.get("w_q")), (s["k"], s.get("w_k"))):
            x = x.float()
            if norm:
                x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * w.float()
            outs.append(_rotate(case, x, cos, sin).to(dtype))
        return tuple(outs)
    grads, weight_grads = [], []
    for x, g, w in ((s["q"], s["dq"], s.get("w_q")), (s["k"], s["dk"], s.get("w_k"))):
        g = _rotate(case, g.float(), cos, -sin)
        if norm:
            x = x.float()
            r = torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"])
            n = x * r
            weight_grads.append((g * n).double().sum(dim=(0, 1, 2)).float())
            gw = g * w.float()
            g = r * (gw - n * (gw * n).mean(-1, keepdim=True))
        grads.append(g.to(dtype))
    return tuple(grads + weight_grads)


def _plain_act(case, x):
    """The activation and its derivative."""
    if case["act"] == "silu":
        sig = 1.0 / (1.0 + torch.exp(-x))
        return x * sig, sig * (1.0 + x * (1.0 - sig))
    cdf = 0.5 * (1.0 + torch.erf(x * math.sqrt(0.5)))
    return x * cdf, cdf + x * torch.exp(-0.5 * x * x) * (1.0 / math.sqrt(2.0 * math.pi))


def _plain_gated(case, s):
    bf16 = torch.bfloat16
    x, wg, wu, wd = (s[k].float() for k in ("X", "W_gate", "W_up", "W_down"))
    gate, up = x @ wg.T, x @ wu.T
    value, slope = _plain_act(case, gate)
    h = value * up
    y = (h @ wd.T).to(bf16)
    if case["direction"] == "forward":
        return y
    dy = s["dY"].float()
    dh = dy @ wd
    dwd = dy.T @ h
    dgate, dup = dh * up * slope, dh * value
    dx = dgate @ wg + dup @ wu
    return y, dx.to(bf16), (dgate.T @ x).to(bf16), (dup.T @ x).to(bf16), dwd.to(bf16)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    if case["op"] == "gated":
        m, d, f = case["tokens"], case["width"], case["hidden"]
        if case["direction"] == "forward":
            return {"bytes": 2 * (2 * m * d + 3 * d * f), "flops": 6 * m * d * f}
        return {"bytes": 2 * (4 * m * d + 6 * d * f), "flops": 18 * m * d * f}
    size = 4 if case["dtype"] == "fp32" else 2
    rows = case["batch"] * case["tokens"]
    n = rows * (case["heads_q"] + case["heads_k"]) * case["dim"]
    positions = 4 * rows * len(_axes(case))
    if case["op"] == "rope":
        return {"bytes": 2 * n * size + positions, "flops": 3 * n}
    if case["direction"] == "forward":
        return {"bytes": 2 * n * size + positions + 2 * case["dim"] * size, "flops": 7 * n}
    return {"bytes": 3 * n * size + positions + 2 * case["dim"] * (size + 4), "flops": 14 * n}


# ------------------------------------------------------------------ the definition in 64 bits
def _turn(case, positions, x, conjugate=False):
    """x [batch, tokens, heads, dim] in float64, its pairs taken as complex numbers and turned."""
    frequencies = torch.cat([torch.pow(torch.tensor(case["theta"], dtype=torch.float64, device="cuda"),
                                       -torch.arange(0, n, 2, dtype=torch.float64, device="cuda") / n)
                             for n in _axes(case)])
    axis = torch.cat([torch.full((n // 2,), a, device="cuda") for a, n in enumerate(_axes(case))])
    angle = positions.double().index_select(-1, axis) * frequencies
    unit = torch.polar(torch.ones_like(angle), -angle if conjugate else angle).unsqueeze(2)
    part = 2 * unit.shape[-1]
    turned, rest = x[..., :part], x[..., part:]
    if case["pairing"] == "interleaved":
        z = torch.view_as_complex(turned.unflatten(-1, (part // 2, 2)).contiguous()) * unit
        turned = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(turned[..., : part // 2].contiguous(), turned[..., part // 2:].contiguous()) * unit
        turned = torch.cat([z.real, z.imag], dim=-1)
    return torch.cat([turned, rest], dim=-1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "gated":
        train = case["direction"] == "train"
        x, wg, wu, wd = (s.pop(k).double().requires_grad_(train) for k in ("X", "W_gate", "W_up", "W_down"))
        act = torch.nn.functional.silu if case["act"] == "silu" else torch.nn.functional.gelu
        linear = torch.nn.functional.linear
        y = linear(act(linear(x, wg)) * linear(x, wu), wd)
        if not train:
            return y
        return (y.detach(),) + torch.autograd.grad(y, (x, wg, wu, wd), s["dY"].double())
    out, weights = [], []
    for x, g, w in (("q", "dq", "w_q"), ("k", "dk", "w_k")):
        if case["op"] == "rope":
            if case["direction"] == "forward":
                out.append(_turn(case, s["positions"], s[x].double()))
            else:
                out.append(_turn(case, s["positions"], s[g].double(), conjugate=True))
            continue
        v = s[x].double()
        weight = s[w].double()
        if case["direction"] == "forward":
            n = v / torch.sqrt(v.square().sum(-1, keepdim=True) / case["dim"] + s["eps"])
            out.append(_turn(case, s["positions"], n * weight))
        else:
            v.requires_grad_(True)
            weight.requires_grad_(True)
            n = v / torch.sqrt(v.square().sum(-1, keepdim=True) / case["dim"] + s["eps"])
            y = _turn(case, s["positions"], n * weight)
            dv, dw = torch.autograd.grad(y, (v, weight), s[g].double())
            out.append(dv)
            weights.append(dw)
    return tuple(out + weights)
