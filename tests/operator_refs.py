"""fp64 restatements (numpy) of the operators around the attention, written from their definitions in
include/ssa.h and sharing nothing with the library, and the error bounds of the kernels' fp32
arithmetic.

The bounds: with u = 2^-24 every fp32 operation is off by at most u relative (sums of n terms by n u of
the terms' magnitudes), and storing the result in a type adds at most half a step, eps/2 of the value
(plus half the smallest subnormal of the type).
"""
from __future__ import annotations

import math

import numpy as np
import torch

U = 2.0 ** -24
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def half_step(dtype: str):
    """(relative, absolute) error of one rounding to the type."""
    f = torch.finfo(DTYPES[dtype])
    return f.eps / 2, float(f.smallest_normal) * f.eps / 2


def f64(t) -> np.ndarray:
    return t.detach().double().cpu().numpy() if isinstance(t, torch.Tensor) else np.asarray(t, np.float64)


def check(got, ref, bound, dtype, what):
    """|got - ref| <= bound + one rounding to the type, on every element."""
    got, ref = f64(got), np.asarray(ref)
    assert got.shape == ref.shape, what
    rel, tiny = half_step(dtype)
    limit = bound * (1 + rel) + rel * np.abs(ref) + tiny
    off = np.abs(got - ref)
    assert np.isfinite(got).all(), f"{what}: not finite"
    worst = float((off / limit).max()) if off.size else 0.0
    print(f"{what}: max|d| {off.max() if off.size else 0:.3e}, {worst:.3f} of the bound ({dtype})")
    assert worst <= 1.0, f"{what}: {worst:.3f} of the bound"


# ---- rotary positions ----------------------------------------------------------------------------

def pair_table(D, theta=10000.0, dim=None, layout="interleaved", scaling=None, scale=1.0, extent=0.0,
               beta_slow=1.0, beta_fast=32.0, mscale=None):
    """[(first channel, second channel, axis, frequency)] of the rotated pairs, and mscale."""
    R = dim or D
    c = 2 * (R // 6)
    pairs, p = [], 0
    for axis, w in ((0, R - 2 * c), (1, c), (2, c)):
        for j in range(w // 2):
            f = math.exp(-2.0 * j / w * math.log(theta))
            if scaling == "linear":
                f = f / scale
            elif scaling == "ntk":
                if w > 2:
                    f = f * scale ** (-2.0 * j / (w - 2))
            elif scaling == "yarn":
                turns = extent * f / (2 * math.pi)
                g = (turns - beta_slow) / (beta_fast - beta_slow)
                g = 0.0 if g < 0 else 1.0 if g > 1 else g
                f = (1 - g) * f / scale + g * f
            pairs.append((2 * p, 2 * p + 1, axis, f) if layout == "interleaved" else (p, p + R // 2, axis, f))
            p += 1
    if mscale is None:
        mscale = 0.1 * math.log(scale) + 1.0 if scaling == "yarn" else 1.0
    return pairs, mscale


def rotate(x, coords, D, back=False, **opt):
    """The rotation of [N, H, D] rows (or its transpose)."""
    pairs, m = pair_table(D, **opt)
    y = np.array(x, np.float64)
    for a, b, axis, f in pairs:
        t = coords[:, axis].astype(np.float64)[:, None] * f
        c, s = m * np.cos(t), m * (-np.sin(t) if back else np.sin(t))
        y[:, :, a], y[:, :, b] = x[:, :, a] * c - x[:, :, b] * s, x[:, :, a] * s + x[:, :, b] * c
    return y


def partner_magnitude(x, D, **opt):
    """|own| + |partner| of every channel, what one rotation's error is relative to."""
    pairs, m = pair_table(D, **opt)
    y = np.abs(x)
    z = np.array(y)
    for a, b, _, _ in pairs:
        z[:, :, a] = z[:, :, b] = m * (y[:, :, a] + y[:, :, b])
    return z


def rotary(x, coords, gamma=None, eps=1e-6, **opt):
    """(output, bound) of the forward for one of q, k."""
    D = x.shape[2]
    u = x if gamma is None else x / np.sqrt((x * x).mean(2, keepdims=True) + eps) * gamma
    # normalisation: a sum of squares in chains of at most 8 + 1 + 4 additions and the mean (14 u) under a square root (7 u),
    # rsqrtf (2 ulp, 4 u), two products (2 u); cosine and sine by series of a 32-bit phase (the phase below 0.1 u, the remainder's
    # rounding and product 1.5 u, the series 2 u) and mscale (2 u); product and sum (2 u): 21 u, 32 u covers them
    return rotate(u, coords, D, **opt), 32 * U * partner_magnitude(u, D, **opt)


def rotary_grad(g, coords, x=None, gamma=None, eps=1e-6, **opt):
    """((dx, bound), (dgamma, sum of the magnitudes of its terms) or None)."""
    D = g.shape[2]
    du, mag = rotate(g, coords, D, back=True, **opt), partner_magnitude(g, D, **opt)
    if gamma is None:
        return (du, 32 * U * mag), None
    inv = 1 / np.sqrt((x * x).mean(2, keepdims=True) + eps)
    n = x * inv
    dot = (du * gamma * n).mean(2, keepdims=True)
    dx = inv * (du * gamma - n * dot)
    # as the forward for every factor, and the mean of the products over the row
    bound = 96 * U * inv * (mag * np.abs(gamma) + np.abs(n) * (mag * np.abs(gamma * n)).mean(2, keepdims=True))
    return (dx, bound), ((du * n).sum((0, 1)), (mag * np.abs(n)).sum((0, 1)))


# ---- group normalisation -------------------------------------------------------------------------

def _phi(z):
    return np.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)


def _cdf(z):
    return torch.special.ndtr(torch.from_numpy(np.ascontiguousarray(z))).numpy()


def _sigma(z):
    e = np.exp(-np.abs(z))
    return np.where(z >= 0, 1 / (1 + e), e / (1 + e))


def activation(z, name):
    return z * _sigma(z) if name == "silu" else z * _cdf(z) if name == "gelu" else z


def activation_grad(z, name):
    if name == "silu":
        return _sigma(z) * (1 + z * (1 - _sigma(z)))
    return _cdf(z) + z * _phi(z) if name == "gelu" else np.ones_like(z)


def activation_error(z, name):
    """Bound, in units u, of the kernels' error of act(z) / |z| and of act'(z): sigma by the hardware's exponential
    (2 ulp, 4 u, and |z| u of its rounded argument) and reciprocal (1 ulp, 2 u); Phi by a polynomial off by up to 6 u and its
    evaluation (8 u), times the exponential of -z^2/2 (2 ulp and z^2 u of its argument) and a reciprocal; a few operations on top.
    |act'| and its terms stay below 1.3 + |z|/4."""
    if name not in ("silu", "gelu"):
        return np.zeros_like(z)
    return (24 + 4 * np.abs(z) + 2 * np.minimum(z * z, 30)) * (1.3 + np.abs(z) / 4)


DEPTH = 64 + 288 + 8    # covers the longest chain of fp32 additions: 48 rows of a thread, up to 256 row lanes of a CTA, the channels


def norm_stats(x, cu, groups):
    """Per (sequence, group): mean, biased variance, mean |x|, max |x - mean|."""
    B = len(cu) - 1
    out = np.zeros((4, B, groups))
    for s in range(B):
        v = x[cu[s]:cu[s + 1]].reshape(cu[s + 1] - cu[s], groups, x.shape[1] // groups)
        if len(v):
            m = v.mean((0, 2))
            d = v - m[:, None]
            out[:, s] = m, (d * d).mean((0, 2)), np.abs(v).mean((0, 2)), np.abs(d).max((0, 2))
    return out


def _rows_of(table, cu, C):
    """[B, G] as [N, C]."""
    t = np.repeat(table, C // table.shape[1], axis=1)
    return np.concatenate([np.broadcast_to(t[s], (b - a, C)) for s, (a, b) in enumerate(zip(cu, cu[1:]))])


def group_norm(x, cu, groups, gamma=None, beta=None, eps=1e-5, act=None):
    """(y, bound), (mean, bound), (rstd, bound). The kernels add a thread's deviations from a pivot among its rows: the mean of
    up to 48 of them is off by 50 u of their size, at most twice the largest deviation, plus 8 u of the values;
    the variance by the cancellation of up to 48 terms, 2 (1 + 4) times 51 u (pivots of random rows are off
    the mean by at most 4 variances on average). Row lanes and channels merge about their means: chains of at most 27 additions and 3 u
    a term. 540 u of the variance, half of that of rstd: below 360 u."""
    C = x.shape[1]
    mean, var, size, most = norm_stats(x, cu, groups)
    empty = (np.diff(cu) == 0)[:, None] | np.zeros_like(mean, bool)
    rstd = np.where(empty, 0.0, 1 / np.sqrt(np.where(empty, 1.0, var + eps)))
    dmean = U * (8 * size + 128 * most)
    drstd = 360 * U * rstd
    g = np.ones(C) if gamma is None else gamma
    b = np.zeros(C) if beta is None else beta
    m, r, dm = (_rows_of(t, cu, C) for t in (mean, rstd, dmean))
    xhat = (x - m) * r
    z = xhat * g + b
    dz = r * np.abs(g) * (dm + U * np.abs(x)) + (360 + 6) * U * np.abs(xhat * g) + 2 * U * np.abs(b)
    bound = 1.13 * dz + U * activation_error(z, act) * np.abs(z)
    return (activation(z, act), bound), (mean, dmean), (rstd, drstd)


def group_norm_grad(dy, x, mean, rstd, cu, groups, gamma=None, beta=None, act=None):
    """(dx, bound), (dgamma, bound), (dbeta, bound) of the formula at the given statistics."""
    N, C = x.shape
    g = np.ones(C) if gamma is None else gamma
    b = np.zeros(C) if beta is None else beta
    m, r = _rows_of(mean, cu, C), _rows_of(rstd, cu, C)
    xhat = (x - m) * r
    exhat = U * (2 * np.abs(xhat) + (np.abs(x) + np.abs(m)) * r)
    z = xhat * g + b
    ez = np.abs(g) * exhat + 2 * U * (np.abs(xhat * g) + np.abs(b))
    dz = dy * activation_grad(z, act)
    # |act''| <= 0.8
    edz = np.abs(dy) * ((0.8 * ez if act in ("silu", "gelu") else 0) + U * activation_error(z, act)) + U * np.abs(dz)
    t1, e1 = dz * g, edz * np.abs(g)
    t2, e2 = t1 * xhat, e1 * np.abs(xhat) + np.abs(t1) * exhat
    n = np.maximum(np.diff(cu), 1)[:, None] * (C // groups)

    def means(t):
        return np.stack([t[a:c].reshape(c - a, groups, C // groups).sum((0, 2)) for a, c in zip(cu, cu[1:])]) / n

    S1, S2 = _rows_of(means(t1), cu, C), _rows_of(means(t2), cu, C)
    eS1 = _rows_of(means(e1 + DEPTH * U * np.abs(t1)), cu, C)
    eS2 = _rows_of(means(e2 + DEPTH * U * np.abs(t2)), cu, C)
    dx = r * (t1 - S1 - xhat * S2)
    edx = r * (e1 + eS1 + np.abs(xhat) * eS2 + exhat * np.abs(S2) + 6 * U * (np.abs(t1) + np.abs(S1) + np.abs(xhat * S2)))
    w = dz * xhat
    ew = edz * np.abs(xhat) + np.abs(dz) * exhat
    return ((dx, edx), (w.sum(0), (ew + DEPTH * U * np.abs(w)).sum(0)), (dz.sum(0), (edz + DEPTH * U * np.abs(dz)).sum(0)))
