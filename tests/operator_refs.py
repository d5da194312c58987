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
    # normalisation: a sum of up to 16 + 4 terms and a division under a square root (11 u), rsqrtf
    # (2 ulp, 4 u), two products; the angle (3 u), sincospif (2 ulp) and mscale, product and sum: 32 u covers them
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
