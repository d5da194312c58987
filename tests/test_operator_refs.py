"""The fp64 references of the operators against independent statements of the same things: the
oracle's prologue, central differences, closed forms; and the library's host-side frequencies."""
import ctypes

import numpy as np
import pytest
import torch

import operator_refs as ref
import oracle
import spatial_sparse_attention_b200 as ssa

OPTS = [dict(), dict(layout="half"), dict(dim=20, layout="half", scaling="linear", scale=3.0),
        dict(dim=2, scaling="ntk", scale=2.0), dict(dim=26, scaling="ntk", scale=4.0, theta=500.0),
        dict(layout="half", scaling="yarn", scale=3.0, extent=64.0, beta_fast=8.0)]


def _rows(n, h, d, seed):
    rng = np.random.default_rng(seed)
    return rng.standard_normal((n, h, d)), rng.integers(0, 200, (n, 3))


@pytest.mark.parametrize("D", [32, 64, 96, 128])
def test_rotary_is_the_oracles_prologue(D):
    x, c = _rows(7, 2, D, D)
    gamma = np.linspace(0.5, 1.5, D).astype(np.float32)
    want = oracle.qk_prologue(x, c.astype(np.int32), gamma, eps=1e-6, theta=1000.0)
    got, _ = ref.rotary(x, c, gamma.astype(np.float64), 1e-6, theta=1000.0)
    np.testing.assert_allclose(got, want, rtol=0, atol=1e-12)


@pytest.mark.parametrize("opt", OPTS)
def test_layouts_are_channel_permutations(opt):
    D = 32
    x, c = _rows(5, 3, D, 1)
    R = opt.get("dim", D)
    perm = np.concatenate([np.arange(0, R, 2), np.arange(1, R, 2), np.arange(R, D)])
    a = ref.rotate(x, c, D, **{**opt, "layout": "interleaved"})
    b = ref.rotate(x[:, :, perm], c, D, **{**opt, "layout": "half"})
    np.testing.assert_allclose(a[:, :, perm], b, rtol=0, atol=1e-13)


@pytest.mark.parametrize("opt", OPTS)
@pytest.mark.parametrize("norm", [False, True])
def test_rotary_gradient_against_differences(opt, norm):
    D = 32
    x, c = _rows(3, 2, D, 2)
    rng = np.random.default_rng(3)
    g = rng.standard_normal(x.shape)
    gamma = rng.random(D) + 0.5 if norm else None
    (dx, _), dg = ref.rotary_grad(g, c, x, gamma, **opt)
    f = lambda v, w: float((ref.rotary(v, c, w, **opt)[0] * g).sum())  # noqa: E731
    h = 1e-5
    for _ in range(4):
        d = rng.standard_normal(x.shape)
        num = (f(x + h * d, gamma) - f(x - h * d, gamma)) / (2 * h)
        # third derivatives times h^2 and the rounding of f over h: below 1e-7 of the terms' size
        assert abs(num - (dx * d).sum()) <= 1e-6 * np.abs(dx * d).sum()
        if norm:
            d = rng.standard_normal(D)
            num = (f(x, gamma + h * d) - f(x, gamma - h * d)) / (2 * h)
            assert abs(num - (dg[0] * d).sum()) <= 1e-6 * np.abs(dg[0] * d).sum()


@pytest.mark.parametrize("opt", OPTS)
@pytest.mark.parametrize("D", [32, 96])
def test_library_frequencies(opt, D):
    pairs, m = ref.pair_table(D, **opt)
    r = ssa.Rotary(**opt)
    axis, freq = r.frequencies(D)
    assert axis == [p[2] for p in pairs]
    np.testing.assert_allclose(freq, [p[3] for p in pairs], rtol=1e-13)
    assert r.mscale == pytest.approx(m, rel=1e-6)


def test_scaled_frequencies_at_the_ends():
    """Linear divides all, ntk keeps the first and divides the last of an axis, yarn keeps what turns often and
    divides what does not."""
    base = ssa.Rotary().frequencies(96)[1]
    lin = ssa.Rotary(scaling="linear", scale=4.0).frequencies(96)[1]
    np.testing.assert_allclose(lin, np.array(base) / 4, rtol=1e-15)
    ntk = ssa.Rotary(scaling="ntk", scale=4.0).frequencies(96)[1]
    assert ntk[0] == 1.0 and ntk[15] == pytest.approx(base[15] / 4, rel=1e-12)
    yarn = ssa.Rotary(scaling="yarn", scale=4.0, extent=1000.0, beta_slow=1.0, beta_fast=32.0).frequencies(96)[1]
    turns = 1000.0 * np.array(base) / (2 * np.pi)
    assert (turns >= 32).any() and (turns <= 1).any()
    np.testing.assert_allclose(np.array(yarn)[turns >= 32], np.array(base)[turns >= 32], rtol=1e-14)
    np.testing.assert_allclose(np.array(yarn)[turns <= 1], np.array(base)[turns <= 1] / 4, rtol=1e-14)


@pytest.mark.parametrize("field,value", [
    ("theta", 1.0), ("theta", float("nan")), ("theta", float("inf")), ("mscale", 0.0), ("mscale", float("inf")),
    ("dim", 3), ("dim", 98), ("dim", -2), ("layout", 2), ("scaling", 4), ("scaling", -1)])
def test_frequencies_refuse(field, value):
    r = ssa.Rotary()
    setattr(r, field, value)
    with pytest.raises(ssa.SSAError, match="INVALID_ARG"):
        ssa._check(ssa.lib.ssa_rotary_frequencies(ctypes.addressof(r), 96, None, None), "x")


@pytest.mark.parametrize("opt", [dict(scaling="linear", scale=0.0), dict(scaling="ntk", scale=-1.0),
                                 dict(scaling="linear", scale=float("inf")),
                                 dict(scaling="linear", scale=5e-324), dict(scaling="ntk", scale=5e-324),
                                 dict(scaling="yarn", scale=2.0, extent=0.0),
                                 dict(scaling="yarn", scale=2.0, extent=64.0, beta_slow=8.0, beta_fast=8.0),
                                 dict(scaling="yarn", scale=2.0, extent=64.0, beta_slow=-1.0)])
def test_scaling_refuses(opt):
    with pytest.raises(ssa.SSAError, match="INVALID_ARG"):
        ssa.Rotary(**opt).frequencies(96)


def test_head_dim_and_names_refused():
    with pytest.raises(ssa.SSAError, match="UNSUPPORTED"):
        ssa.Rotary().frequencies(80)
    for bad in (dict(layout="pairs"), dict(scaling="log"), dict(dim=0)):
        with pytest.raises(ValueError):
            ssa.Rotary(**bad)


def test_operators_refuse_a_null_plan_before_any_device_work():
    r = ssa.Rotary()
    v = ssa._Heads(16, 96, 96, 1)
    a = ctypes.addressof
    assert ssa.lib.ssa_rotary(None, a(v), None, None, None, 1e-6, a(r), 96, 1, a(v), None, None) == 1
    assert ssa.lib.ssa_rotary_backward(None, a(v), None, None, None, None, None, 1e-6, a(r), 96, 1, a(v), None, None,
                                       None, None) == 1


# ---- group normalisation -------------------------------------------------------------------------

@pytest.mark.parametrize("act", [None, "silu", "gelu"])
def test_group_norm_is_torchs_per_sequence(act):
    rng = np.random.default_rng(1)
    cu = np.array([0, 5, 5, 6, 20])
    x, w, b = rng.standard_normal((20, 12)) * 3 + 1, rng.random(12) + 0.5, rng.standard_normal(12)
    (y, _), (mean, _), (rstd, _) = ref.group_norm(x, cu, 3, w, b, 1e-3, act)
    f = {None: lambda t: t, "silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu}[act]
    for s, (a, e) in enumerate(zip(cu, cu[1:])):
        if a == e:
            assert (mean[s] == 0).all() and (rstd[s] == 0).all()
            continue
        t = torch.from_numpy(x[a:e].T[None])
        want = f(torch.nn.functional.group_norm(t, 3, torch.from_numpy(w), torch.from_numpy(b), 1e-3))[0].T.numpy()
        np.testing.assert_allclose(y[a:e], want, rtol=0, atol=1e-12)


@pytest.mark.parametrize("act", [None, "silu", "gelu"])
@pytest.mark.parametrize("affine", [False, True])
def test_group_norm_gradient_against_differences(act, affine):
    rng = np.random.default_rng(2)
    cu = np.array([0, 7, 7, 8, 19])
    x, dy = rng.standard_normal((19, 8)), rng.standard_normal((19, 8))
    w, b = (rng.random(8) + 0.5, rng.standard_normal(8)) if affine else (np.ones(8), np.zeros(8))
    _, (mean, _), (rstd, _) = ref.group_norm(x, cu, 2, w, b, 1e-2, act)
    grads = ref.group_norm_grad(dy, x, mean, rstd, cu, 2, *((w, b) if affine else (None, None)), act)
    f = lambda *a: float((ref.group_norm(a[0], cu, 2, a[1], a[2], 1e-2, act)[0][0] * dy).sum())  # noqa: E731
    h = 1e-5
    for i, v in enumerate((x, w, b)):
        for _ in range(4):
            d = rng.standard_normal(v.shape)
            at = lambda s: f(*[u + s * d if j == i else u for j, u in enumerate((x, w, b))])  # noqa: E731
            num = (at(h) - at(-h)) / (2 * h)
            assert abs(num - (grads[i][0] * d).sum()) <= 1e-6 * np.abs(grads[i][0] * d).sum() + 1e-7


def test_group_norm_refuses_a_null_plan_before_any_device_work():
    v, a = ssa._Rows(16, 8), ctypes.addressof
    assert ssa.lib.ssa_group_norm(None, a(v), 8, 2, None, None, 1e-5, 0, 0, a(v), None, None, None) == 1
    assert ssa.lib.ssa_group_norm_backward(None, a(v), a(v), 16, 16, 8, 2, None, None, 0, 0, a(v), 16, 16, None) == 1
