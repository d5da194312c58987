"""Measured cases of the operators around the attention: rotary positions with the RMS normalisation of
queries and keys, and group normalisation with an activation over packed voxel tokens, both with
their gradients.

`listed()` and `draw(rng)` give cases, `prepare(case, seed)` what a program holds before the call,
`run(state)` one pass: in plain torch (`own` false) or through this package (`own` true). `work(case)`
counts the bytes and operations of a pass, `exact(case, seed)` gives its outputs in 64 bits.

The operators (N tokens with voxel coordinates, in packed sequences that do not see each other):

  rotary       q [N, H, D] and k [N, Hk, D]: u = x * rsqrt(mean_d x^2 + eps) * gamma where `norm`, then
               channel pair p of the first `rotary_dim` channels turns by coordinate[axis_p] * freq_p
               and grows by mscale. `interleaved` pairs (2p, 2p+1), `half` pairs (p, p + rotary_dim/2).
               The pairs go to the axes x, y, z in this order: c = 2 floor(rotary_dim/6) channels to
               each of y and z, the rest to x; freq is theta^(-2j/w) for the j-th pair of an axis of
               w channels, scaled for grids larger than the trained one (`frequencies`).
  rotary_grad  its gradients for q and k, and for the weights where `norm`.
  norm         y = act((x - mean) * rstd * gamma + beta), mean and variance of x [N, C] over the tokens of a
               sequence and the channels of a group; also mean and rstd, [sequences, groups], which are
               zero for a sequence of no tokens.
  norm_grad    its gradients for x, gamma and beta.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
THETA, RMS_EPS, NORM_EPS = 10000.0, 1e-6, 1e-5


def _rotary(name, op, seqs, grid, heads, kv_heads, dim, dtype, layout, rotary_dim, scaling, scale, norm, fused):
    return {"name": name, "op": op, "seqs": seqs, "grid": grid, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "dtype": dtype, "layout": layout, "rotary_dim": rotary_dim, "scaling": scaling, "scale": scale,
            "norm": norm, "fused": fused}


def _norm(name, op, seqs, channels, groups, dtype, activation, affine):
    return {"name": name, "op": op, "seqs": seqs, "channels": channels, "groups": groups, "dtype": dtype,
            "activation": activation, "affine": affine}


def listed():
    return [
        # one voxel token added to a running shape: nothing but the latency of a call
        _rotary("rotary one token", "rotary", "1", 32, 22, 22, 96, "f16", "interleaved", 96, "none", 1.0, True, False),
        # a mid-size shell in a grid twice the trained one, queries and keys still inside the fused
        # projection's output, fewer key heads, part of the head rotated
        _rotary("rotary small shell", "rotary", "20000", 128, 8, 4, 64, "bf16", "half", 40, "yarn", 2.0, True, True),
        # the headline shell with the transformer's own prologue
        _rotary("rotary large shell", "rotary", "110000", 192, 22, 22, 96, "f16", "interleaved", 96, "none", 1.0, True,
                False),
        # a ragged training batch in single precision, an empty and a one-token sequence among its four
        _rotary("rotary grad ragged", "rotary_grad", "700,0,1,633", 32, 3, 3, 32, "f32", "interleaved", 32, "linear",
                4.0, True, False),
        # a rotation without weights: its gradient is the rotation back
        _rotary("rotary grad small shell", "rotary_grad", "20000", 128, 8, 8, 64, "bf16", "half", 64, "ntk", 2.0, False,
                True),
        # a training step of the first refinement pass, weights' gradients over 1.76 million rows
        _rotary("rotary grad large shell", "rotary_grad", "80000", 64, 22, 22, 96, "f16", "interleaved", 96, "none", 1.0,
                True, False),
        # the tiny shell's features: one launch's latency
        _norm("norm tiny shell", "norm", "1814", 64, 8, "f32", "none", True),
        # a mid-size decoder layer
        _norm("norm small shell", "norm", "20000", 512, 32, "bf16", "silu", True),
        # the packed batch of four shells at the transformer's width; groups of 66 channels
        _norm("norm packed shells", "norm", "80000,90000,110000,60000", 2112, 32, "f16", "silu", True),
        # a ragged training batch, an empty and a one-token sequence among its four; 67 channels in one group
        _norm("norm grad ragged", "norm_grad", "700,0,1,633", 67, 1, "f32", "gelu", True),
        # the mid-size layer's training step
        _norm("norm grad small shell", "norm_grad", "20000", 512, 32, "bf16", "silu", True),
        # the first refinement pass's training step at the transformer's width
        _norm("norm grad large shell", "norm_grad", "80000", 2112, 32, "f16", "silu", True),
    ]


def _log_int(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _split(rng, n):
    """n tokens in one to five sequences, empty ones among them."""
    parts = rng.choice((1, 1, 2, 3, 5))
    cuts = sorted(rng.randint(0, n) for _ in range(parts - 1))
    if parts > 2 and rng.random() < 0.3:
        cuts[1] = cuts[0]
    edges = [0] + cuts + [n]
    return ",".join(str(b - a) for a, b in zip(edges, edges[1:]))


def draw(rng):
    op = rng.choice(("rotary", "rotary_grad", "norm", "norm_grad"))
    dtype = rng.choice(("f16", "bf16", "f32"))
    if op.startswith("rotary"):
        dim, heads = rng.choice((32, 64, 96, 128)), rng.randint(1, 24)
        kv_heads = rng.choice((heads, rng.randint(1, heads)))
        row = (heads + kv_heads) * dim * BYTES[dtype]
        most = (110000 * 44 if op == "rotary" else 80000 * 44) * 96 * 2 // row
        n = _log_int(rng, 1, min(110000, most))
        scaling = rng.choice(("none", "linear", "ntk", "yarn"))
        c = _rotary("", op, _split(rng, n), rng.choice((192, 256, 1024)), heads, kv_heads, dim, dtype,
                    rng.choice(("interleaved", "half")), dim if rng.random() < 0.5 else 2 * rng.randint(1, dim // 2),
                    scaling, 1.0 if scaling == "none" else rng.choice((2.0, 3.0, 16.0)), rng.random() < 0.6,
                    rng.random() < 0.4)
    else:
        groups = rng.choice((1, 2, 8, 16, 22, 32))
        # a gradient over groups of one or two values is all cancellation
        width = _log_int(rng, 1 if op == "norm" else 4, 2112 // groups)
        most = (340000 if op == "norm" else 80000) * 2112 * 2 // (groups * width * BYTES[dtype])
        n = _log_int(rng, 1, min(340000, most))
        c = _norm("", op, _split(rng, n), groups * width, groups, dtype, rng.choice(("none", "silu", "gelu")),
                  rng.random() < 0.8)
    del c["name"]
    return c


def frequencies(rotary_dim, scaling, scale, extent):
    """Axis and angular frequency of every rotated pair, and the factor on the rotated channels."""
    c = 2 * (rotary_dim // 6)
    axes, freq = [], []
    for axis, w in enumerate((rotary_dim - 2 * c, c, c)):
        for j in range(w // 2):
            f = THETA ** (-2.0 * j / w)
            if scaling == "linear":
                f /= scale
            elif scaling == "ntk" and w > 2:
                f = (THETA * scale ** (w / (w - 2.0))) ** (-2.0 * j / w)
            elif scaling == "yarn":
                keep = min(1.0, max(0.0, (extent * f / (2 * math.pi) - 1.0) / (32.0 - 1.0)))
                f *= keep + (1.0 - keep) / scale
            axes.append(axis)
            freq.append(f)
    return axes, freq, 0.1 * math.log(scale) + 1.0 if scaling == "yarn" else 1.0


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _shell(gen, n, edge):
    """n distinct cells of a grid of this edge: those nearest to a sphere, in a box of at most 192 cells at a
    random place, in lexicographic order."""
    box = min(edge, 192)
    at = torch.arange(box, device="cuda", dtype=torch.float32) + 0.5
    mid = box * (0.45 + 0.1 * torch.rand(3, device="cuda", generator=gen))
    sq = ((at - mid[0]) ** 2)[:, None, None] + ((at - mid[1]) ** 2)[None, :, None] + ((at - mid[2]) ** 2)[None, None, :]
    off = (sq.sqrt() - 0.33 * box).abs().flatten()
    cells = off.topk(n, largest=False).indices.sort().values
    xyz = torch.stack((cells // (box * box), cells // box % box, cells % box), 1).to(torch.int32)
    return xyz + torch.randint(0, edge - box + 1, (1, 3), device="cuda", generator=gen, dtype=torch.int32)


def _edges(case):
    cu = [0]
    for n in case["seqs"].split(","):
        cu.append(cu[-1] + int(n))
    return cu


def _coords(gen, cu, edge):
    parts = [_shell(gen, b - a, edge) for a, b in zip(cu, cu[1:]) if b > a]
    return torch.cat(parts).contiguous()


def _plan(coords, cu, edge):
    import spatial_sparse_attention_b200 as ssa
    if len(cu) == 2:
        return ssa.Plan(coords, grid=(edge,) * 3, r=0)
    return ssa.Plan(coords, r=0, cu_seqlens=cu, grids=[(edge,) * 3] * (len(cu) - 1))


def prepare(case, seed):
    gen, dt, cu = _generator(seed), DTYPES[case["dtype"]], _edges(case)
    n = cu[-1]
    # queries and keys of a normalised projection; features with a mean and a spread of their own per channel
    normal = lambda *shape: torch.randn(*shape, device="cuda", generator=gen)  # noqa: E731
    state = {"case": case, "cu": cu}
    if case["op"].startswith("rotary"):
        h, hk, d, edge = case["heads"], case["kv_heads"], case["dim"], case["grid"]
        state["coords"] = _coords(gen, cu, edge)
        extent = edge / case["scale"]
        axes, freq, state["mscale"] = frequencies(case["rotary_dim"], case["scaling"], case["scale"], extent)
        state["axes"] = torch.tensor(axes, device="cuda")
        state["freq"] = torch.tensor(freq, dtype=torch.float64, device="cuda")

        def pair():
            if case["fused"]:   # views of the projection's output, values behind the keys
                qkv = normal(n, h + 2 * hk, d).to(dt)
                return qkv[:, :h], qkv[:, h:h + hk]
            return normal(n, h, d).to(dt), normal(n, hk, d).to(dt)

        if case["norm"] or case["op"] == "rotary":
            state["q"], state["k"] = pair()
        if case["op"] == "rotary_grad":
            state["dq"], state["dk"] = pair()
        if case["norm"]:
            state["q_gamma"] = 0.5 + torch.rand(d, device="cuda", generator=gen)
            state["k_gamma"] = 0.5 + torch.rand(d, device="cuda", generator=gen)
        if own:
            import spatial_sparse_attention_b200 as ssa
            state["plan"] = _plan(state["coords"], cu, edge)
            state["rotary"] = ssa.Rotary(theta=THETA, layout=case["layout"], dim=case["rotary_dim"],
                                         scaling=case["scaling"], scale=case["scale"], extent=extent)
    else:
        c, g = case["channels"], case["groups"]
        x = normal(n, c)
        x *= 0.5 + torch.rand(c, device="cuda", generator=gen)
        x += 0.5 * normal(c)
        state["x"] = x.to(dt)
        del x
        state["gamma"] = 1.0 + 0.2 * normal(c) if case["affine"] else None
        state["beta"] = 0.2 * normal(c) if case["affine"] else None
        if case["op"] == "norm_grad":
            state["dy"] = normal(n, c).to(dt)
            state["mean"], state["rstd"] = _statistics(state["x"], cu, g)
        if own:
            # any cells will do: only the packing of the sequences is used
            at = torch.arange(max(b - a for a, b in zip(cu, cu[1:])), device="cuda")
            cells = torch.stack((at // 4096, at // 64 % 64, at % 64), 1).to(torch.int32)
            state["plan"] = _plan(torch.cat([cells[:b - a] for a, b in zip(cu, cu[1:])]).contiguous(), cu, 128)
    return state


# ------------------------------------------------------------------------------------------------
# plain forms
# ------------------------------------------------------------------------------------------------

def _turn(x, state, back=False):
    """The rotation of fp32 rows [N, heads, D], or its transpose."""
    case, r = state["case"], state["case"]["rotary_dim"]
    angle = state["coords"].double()[:, state["axes"]] * state["freq"]
    cos = (angle.cos() * state["mscale"]).float()[:, None]
    sin = (angle.sin() * state["mscale"]).float()[:, None]
    if back:
        sin = -sin
    even, odd = (slice(0, r, 2), slice(1, r, 2)) if case["layout"] == "interleaved" else (slice(0, r // 2),
                                                                                       slice(r // 2, r))
    y = x.clone()
    y[..., even] = x[..., even] * cos - x[..., odd] * sin
    y[..., odd] = x[..., even] * sin + x[..., odd] * cos
    return y


def _rotary_plain(state):
    out = []
    for name in ("q", "k"):
        x = state[name].float()
        if state["case"]["norm"]:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + RMS_EPS) * state[name + "_gamma"]
        out.append(_turn(x, state).to(state[name].dtype))
    return out


def _rotary_grad_plain(state):
    grads, weights = [], []
    for name in ("q", "k"):
        g = state["d" + name]
        du = _turn(g.float(), state, back=True)
        if state["case"]["norm"]:
            x, gamma = state[name].float(), state[name + "_gamma"]
            inv = torch.rsqrt((x * x).mean(-1, keepdim=True) + RMS_EPS)
            x = x * inv
            weights.append((du * x).sum((0, 1), dtype=torch.float64).float())
            du = du * gamma
            du = inv * (du - x * (du * x).mean(-1, keepdim=True))
        grads.append(du.to(g.dtype))
    return grads + weights


def _statistics(x, cu, groups):
    mean = torch.zeros(len(cu) - 1, groups, device=x.device)
    rstd = torch.zeros_like(mean)
    for s, (a, b) in enumerate(zip(cu, cu[1:])):
        if b > a:
            v = x[a:b].float().view(b - a, groups, -1)
            m = v.sum((0, 2), dtype=torch.float64) / (v.shape[0] * v.shape[2])
            mean[s] = m.float()
            v = v - mean[s][:, None]
            rstd[s] = ((v * v).sum((0, 2), dtype=torch.float64) / (v.shape[0] * v.shape[2]) + NORM_EPS).rsqrt().float()
    return mean, rstd


def _norm_plain(state):
    case, x, cu = state["case"], state["x"], state["cu"]
    mean, rstd = _statistics(x, cu, case["groups"])
    y = torch.empty_like(x)
    width = case["channels"] // case["groups"]
    for s, (a, b) in enumerate(zip(cu, cu[1:])):
        z = (x[a:b].float() - mean[s].repeat_interleave(width)) * rstd[s].repeat_interleave(width)
        if case["affine"]:
            z = z * state["gamma"] + state["beta"]
        if case["activation"] == "silu":
            z = z * torch.sigmoid(z)
        elif case["activation"] == "gelu":
            z = 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
        y[a:b] = z.to(x.dtype)
    return y, mean, rstd


def _norm_grad_plain(state):
    case, x, cu, groups = state["case"], state["x"], state["cu"], state["case"]["groups"]
    channels = case["channels"]
    width = channels // groups
    gamma = state["gamma"] if case["affine"] else torch.ones(channels, device=x.device)
    beta = state["beta"] if case["affine"] else torch.zeros(channels, device=x.device)
    dx = torch.empty_like(x)
    dgamma = torch.zeros(channels, dtype=torch.float64, device=x.device)
    dbeta = torch.zeros_like(dgamma)
    for s, (a, b) in enumerate(zip(cu, cu[1:])):
        if b == a:
            continue
        rstd = state["rstd"][s].repeat_interleave(width)
        xhat = (x[a:b].float() - state["mean"][s].repeat_interleave(width)) * rstd
        dz = state["dy"][a:b].float()
        if case["activation"] != "none":
            z = xhat * gamma + beta
            if case["activation"] == "silu":
                t = torch.sigmoid(z)
                dz = dz * (t * (1.0 + z * (1.0 - t)))
            else:
                dz = dz * (0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi))
            del z
        db, dg = dz.sum(0, dtype=torch.float64), (dz * xhat).sum(0, dtype=torch.float64)
        dbeta += db
        dgamma += dg
        m = float(b - a) * width
        s1 = ((db * gamma).view(groups, width).sum(1) / m).float().repeat_interleave(width)
        s2 = ((dg * gamma).view(groups, width).sum(1) / m).float().repeat_interleave(width)
        dx[a:b] = (rstd * (dz * gamma - s1 - xhat * s2)).to(x.dtype)
    return dx, dgamma.float(), dbeta.float()


def run(state):
    op = state["case"]["op"]
    if not own:
        return {"rotary": _rotary_plain, "rotary_grad": _rotary_grad_plain, "norm": _norm_plain,
                "norm_grad": _norm_grad_plain}[op](state)
    plan, case = state["plan"], state["case"]
    if op == "rotary":
        return plan.rotary(state["q"], state["k"], state["rotary"], state.get("q_gamma"), state.get("k_gamma"),
                           eps=RMS_EPS)
    if op == "rotary_grad":
        return plan.rotary_backward(state["dq"], state["dk"], state["rotary"], state.get("q"), state.get("k"),
                                    state.get("q_gamma"), state.get("k_gamma"), eps=RMS_EPS)
    if op == "norm":
        return plan.group_norm(state["x"], case["groups"], state["gamma"], state["beta"], eps=NORM_EPS,
                               activation=case["activation"], return_stats=True)
    return plan.group_norm_backward(state["dy"], state["x"], state["mean"], state["rstd"], case["groups"],
                                    state["gamma"], state["beta"], activation=case["activation"])


def work(case):
    n, size = _edges(case)[-1], BYTES[case["dtype"]]
    if case["op"].startswith("rotary"):
        rows, d, r = n * (case["heads"] + case["kv_heads"]), case["dim"], case["rotary_dim"]
        weights = 8 * d if case["norm"] else 0
        if case["op"] == "rotary":
            return {"bytes": 2 * rows * d * size + 12 * n + weights, "flops": rows * (3 * r + (4 * d if case["norm"] else 0))}
        return {"bytes": (3 if case["norm"] else 2) * rows * d * size + 12 * n + 2 * weights,
                "flops": rows * (3 * r + (10 * d if case["norm"] else 0))}
    c, tables = case["channels"], 8 * case["groups"] * len(case["seqs"].split(","))
    weights, act = 8 * case["channels"] if case["affine"] else 0, 0 if case["activation"] == "none" else 6
    if case["op"] == "norm":
        return {"bytes": 2 * n * c * size + weights + tables, "flops": n * c * (7 + act)}
    return {"bytes": 3 * n * c * size + weights + 8 * c + tables, "flops": n * c * (14 + act)}


# ------------------------------------------------------------------------------------------------
# 64 bits
# ------------------------------------------------------------------------------------------------

def _rotary_exact(x, gamma, state):
    """RMS normalisation and rotation of [N, heads, D] fp64 rows: each pair as one complex number."""
    case, r = state["case"], state["case"]["rotary_dim"]
    if gamma is not None:
        x = gamma * x / (x.square().sum(-1, keepdim=True) / x.shape[-1] + RMS_EPS).sqrt()
    turn = torch.polar(torch.full_like(state["freq"], state["mscale"]).expand(x.shape[0], -1),
                       state["coords"][:, state["axes"]].to(torch.float64) * state["freq"])[:, None]
    head, tail = x[..., :r], x[..., r:]
    if case["layout"] == "interleaved":
        z = torch.view_as_complex(head.reshape(*head.shape[:-1], r // 2, 2))
        return torch.cat((torch.view_as_real(z * turn).flatten(-2), tail), -1)
    z = torch.complex(*head.chunk(2, -1)) * turn
    return torch.cat((z.real, z.imag, tail), -1)


def _norm_exact(x, gamma, beta, case, cu, want_stats=False):
    """Group normalisation and activation of fp64 [N, C], sequence by sequence."""
    outs, means, rstds = [], [], []
    g = case["groups"]
    for a, b in zip(cu, cu[1:]):
        if a == b:
            means.append(x.new_zeros(g))
            rstds.append(x.new_zeros(g))
            continue
        v = x[a:b].reshape(b - a, g, -1)
        var, mean = torch.var_mean(v, dim=(0, 2), unbiased=False)
        means.append(mean)
        rstds.append(1.0 / (var + NORM_EPS).sqrt())
        outs.append(((v - mean[:, None]) / (var + NORM_EPS).sqrt()[:, None]).reshape(b - a, -1))
    z = torch.cat(outs)
    if gamma is not None:
        z = z * gamma + beta
    if case["activation"] == "silu":
        z = z / (1.0 + (-z).exp())
    elif case["activation"] == "gelu":
        z = 0.5 * z * torch.special.erfc(-z / math.sqrt(2.0))
    return (z, torch.stack(means), torch.stack(rstds)) if want_stats else z


def exact(case, seed):
    state = prepare(case, seed)
    cu = state["cu"]
    if case["op"].startswith("rotary"):
        outs, weights = [], []
        for name in ("q", "k"):
            gamma = state[name + "_gamma"].double() if case["norm"] else None
            if case["op"] == "rotary":
                outs.append(_rotary_exact(state[name].double(), gamma, state))
                continue
            # the gradient by differentiating the operator; without weights it does not depend on the input
            g = state["d" + name].double()
            x = (state[name].double() if case["norm"] else torch.zeros_like(g)).requires_grad_()
            leaves = [x] + ([gamma.requires_grad_()] if case["norm"] else [])
            grads = torch.autograd.grad(_rotary_exact(x, gamma, state), leaves, g)
            outs.append(grads[0])
            weights += list(grads[1:])
        return outs + weights
    gamma = state["gamma"].double() if case["affine"] else None
    beta = state["beta"].double() if case["affine"] else None
    x = state["x"].double()
    if case["op"] == "norm":
        return _norm_exact(x, gamma, beta, case, cu, True)
    if not case["affine"]:   # weights of one and zero have a gradient too
        gamma, beta = x.new_ones(case["channels"]), x.new_zeros(case["channels"])
    leaves = [t.requires_grad_() for t in (x, gamma, beta)]
    return list(torch.autograd.grad(_norm_exact(*leaves, case, cu), leaves, state["dy"].double()))
