"""ssa_rotary and ssa_rotary_backward through the C ABI against the fp64 references, on every element."""
import ctypes

import numpy as np
import pytest
import torch

import operator_refs as ref
import workloads
from ssa_testlib import coords_of, make_plan, tensors_of, to_gpu

pytestmark = pytest.mark.gpu

import spatial_sparse_attention_b200 as ssa  # noqa: E402


def cells(n, edge, seed):
    """n distinct cells of a grid, far corner included."""
    rng = np.random.default_rng(seed)
    at = rng.choice(edge ** 3, size=n, replace=False)
    at[0] = edge ** 3 - 1
    at = np.unique(at)
    while len(at) < n:
        at = np.unique(np.append(at, rng.integers(edge ** 3)))
    return np.stack([at // edge ** 2, at // edge % edge, at % edge], 1).astype(np.int32)


def one_plan(n, edge=64, seed=0):
    c = cells(n, edge, seed)
    return ssa.Plan(torch.from_numpy(c).cuda(), grid=(edge,) * 3, r=0), c


def rows(shape, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(ref.DTYPES[dtype])


def weights(D, seed):
    g = torch.Generator().manual_seed(seed)
    return 0.5 + torch.rand(D, generator=g), 0.5 + torch.rand(D, generator=g)


def check_forward(plan, c, q, k, opt, gammas=(None, None), eps=1e-6, what="", **call):
    dtype = {v: n for n, v in ref.DTYPES.items()}[q.dtype]
    gq, gk = (None if w is None else w.cuda() for w in gammas)
    outs = plan.rotary(q, k, ssa.Rotary(**opt), gq, gk, eps=eps, **call)
    torch.cuda.synchronize()
    for x, got, w, name in zip((q, k), outs, gammas, "qk"):
        want, bound = ref.rotary(ref.f64(x), c, None if w is None else ref.f64(w), eps, **opt)
        ref.check(got, want, bound, dtype, f"{what} {name}")
    return outs


def check_backward(plan, c, up_q, up_k, q, k, opt, gammas=(None, None), eps=1e-6, depth=256, what="", **call):
    """depth: terms of the longest chain of additions of the weights' gradients."""
    dtype = {v: n for n, v in ref.DTYPES.items()}[up_q.dtype]
    gq, gk = (None if w is None else w.cuda() for w in gammas)
    refs = [ref.rotary_grad(ref.f64(g), c, None if w is None else ref.f64(x), None if w is None else ref.f64(w), eps,
                            **opt) for g, x, w in zip((up_q, up_k), (q, k), gammas)]
    outs = plan.rotary_backward(up_q, up_k, ssa.Rotary(**opt), q, k, gq, gk, eps=eps, **call)
    torch.cuda.synchronize()
    for i, name in enumerate("qk"):
        ref.check(outs[i], *refs[i][0], dtype, f"{what} d{name}")
        if gammas[0] is not None:
            dg, mag = refs[i][1]
            ref.check(outs[2 + i], dg, (96 + depth) * ref.U * mag, "f32", f"{what} d{name}_gamma")
    return outs


# ---- refusals first: none of these calls may reach a kernel ------------------------------------

def test_refusals():
    plan, c = one_plan(10)
    q = torch.zeros(10, 3, 96, dtype=torch.float16, device="cuda")
    k = torch.zeros(10, 2, 96, dtype=torch.float16, device="cuda")
    w = torch.ones(96, device="cuda")
    before = ssa.launch_count()
    for bad in (q.cpu(), q[:9], q[0], q[:, :, ::2], q.float(), q.transpose(1, 2)):
        with pytest.raises(ValueError):
            plan.rotary(q, bad)
    with pytest.raises(ValueError):
        plan.rotary(q.cpu(), k.cpu())
    with pytest.raises(ValueError):
        plan.rotary(q, k, q_gamma=w[:95], k_gamma=w)
    with pytest.raises(ValueError):
        plan.rotary(q, k, q_gamma=w.half(), k_gamma=w)
    for kw in (dict(q_gamma=w), dict(k_gamma=w),                      # one weight without the other
               dict(eps=-1.0), dict(eps=float("nan")),
               dict(q_out=k.repeat(1, 2, 1)[:, :1]),                     # another head count
               dict(q_out=torch.zeros(1, 3, 96, dtype=q.dtype, device="cuda").expand(10, 3, 96)),
               dict(q_out=torch.zeros(10, 1, 96, dtype=q.dtype, device="cuda").expand(10, 3, 96))):
        with pytest.raises(ssa.SSAError, match="INVALID_ARG"):
            plan.rotary(q, k, **kw)
    with pytest.raises(ssa.SSAError, match="INVALID_ARG"):
        plan.rotary(q.double(), k.double())
    with pytest.raises(ssa.SSAError, match="INVALID_ARG"):
        plan.rotary(q, k, ssa.Rotary(dim=98))
    with pytest.raises(ssa.SSAError, match="UNSUPPORTED"):
        plan.rotary(q[:, :, :80], k[:, :, :80])
    # outputs that meet what the call reads or writes elsewhere
    buf = torch.zeros(10, 8, 96, dtype=q.dtype, device="cuda")
    with pytest.raises(ssa.SSAError, match="INVALID_ARG"):
        plan.rotary(q, buf[:, 2:4], q_out=buf[:, :3])                # q_out over k's first head
    with pytest.raises(ssa.SSAError, match="INVALID_ARG"):
        plan.rotary(buf[:, :3], k, q_out=buf[:, 1:4])                # q_out shifted over q
    with pytest.raises(ssa.SSAError, match="INVALID_ARG"):
        plan.rotary(q, k, q_out=buf[:, :3], k_out=buf[:, 2:4])
    # the gradient with weights needs the inputs
    with pytest.raises(ssa.SSAError, match="INVALID_ARG"):
        plan.rotary_backward(q, k, None, None, None, w, w)
    with pytest.raises(ssa.SSAError, match="INVALID_ARG"):
        plan.rotary_backward(q, k, None, q, k, w, None)
    with pytest.raises(ssa.SSAError, match="INVALID_ARG"):
        plan.rotary_backward(q, k, None, q, k[:, :1], w, w)
    assert ssa.launch_count() == before


def test_c_refusals():
    """What the binding cannot express: null views, misaligned data, negative strides, a queries-only call with a
    key output."""
    plan, _ = one_plan(4)
    x = torch.zeros(4, 2, 32, device="cuda")
    r, a = ssa.Rotary(), ctypes.addressof
    ok = ssa._Heads(x.data_ptr(), 64, 32, 2)
    call = lambda q, k, qo, ko, dt=0: ssa.lib.ssa_rotary(plan._h, q and a(q), k and a(k), None, None, 1e-6, a(r), 32, dt,  # noqa: E731
                                                         qo and a(qo), ko and a(ko), None)
    before = ssa.launch_count()
    assert call(None, None, ok, None) == 1
    assert call(ok, None, None, None) == 1
    assert call(ok, None, ok, ok) == 1
    assert call(ok, ok, ok, None) == 1
    for bad in (ssa._Heads(None, 64, 32, 2), ssa._Heads(x.data_ptr() + 2, 64, 32, 2), ssa._Heads(x.data_ptr(), -64, 32, 2),
                ssa._Heads(x.data_ptr(), 64, -32, 2), ssa._Heads(x.data_ptr(), 64, 32, 0),
                ssa._Heads(x.data_ptr(), 1 << 40, 32, 2)):
        assert call(bad, None, ok, None) == 1
        assert call(ok, None, bad, None) == 1
    assert call(ok, None, ok, None, dt=3) == 1
    assert ssa.lib.ssa_rotary(plan._h, a(ok), None, None, None, 1e-6, None, 32, 0, a(ok), None, None) == 1
    assert ssa.launch_count() == before


def test_c_refuses_misaligned_weights_and_an_infinite_eps():
    plan, _ = one_plan(4)
    x = torch.zeros(4, 2, 32, device="cuda")
    w = torch.ones(160, device="cuda")
    r, a, p = ssa.Rotary(), ctypes.addressof, w.data_ptr()
    v = ssa._Heads(x.data_ptr(), 64, 32, 2)
    before = ssa.launch_count()
    assert ssa.lib.ssa_rotary(plan._h, a(v), None, p + 1, None, 1e-6, a(r), 32, 0, a(v), None, None) == 1
    assert ssa.lib.ssa_rotary(plan._h, a(v), None, p, None, float("inf"), a(r), 32, 0, a(v), None, None) == 1
    assert ssa.lib.ssa_rotary_backward(plan._h, a(v), None, a(v), None, p, None, 1e-6, a(r), 32, 0, a(v), None, p + 130, None,
                                       None) == 1
    assert ssa.launch_count() == before


# ---- values ------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("D", [32, 64, 96, 128])
@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("norm", [False, True])
def test_types_head_dims_layouts(dtype, D, layout, norm):
    plan, c = one_plan(301, seed=D)
    q, k = rows((301, 5, D), dtype, 1).cuda(), rows((301, 2, D), dtype, 2).cuda()
    dq, dk = rows((301, 5, D), dtype, 3).cuda(), rows((301, 2, D), dtype, 4).cuda()
    g = weights(D, 5) if norm else (None, None)
    opt = dict(layout=layout)
    check_forward(plan, c, q, k, opt, g)
    check_backward(plan, c, dq, dk, q, k, opt, g)


@pytest.mark.parametrize("dtype,D", [("f16", 96), ("f32", 64), ("bf16", 128)])
@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("dim", [2, 4, 6, 8, 10, 26, 32, 40, 50, 62])
def test_part_of_the_head(dtype, D, layout, dim):
    plan, c = one_plan(77, seed=dim)
    q, k = rows((77, 3, D), dtype, 1).cuda(), rows((77, 3, D), dtype, 2).cuda()
    dq, dk = rows((77, 3, D), dtype, 3).cuda(), rows((77, 3, D), dtype, 4).cuda()
    opt = dict(layout=layout, dim=dim)
    g = weights(D, 5)
    q2, _ = check_forward(plan, c, q, k, opt)
    # the channels that pass through keep their bits
    assert torch.equal(q2[:, :, dim:], q[:, :, dim:])
    check_forward(plan, c, q, k, opt, g)
    check_backward(plan, c, dq, dk, q, k, opt, g)


@pytest.mark.parametrize("opt", [dict(scaling="linear", scale=16.0), dict(scaling="ntk", scale=3.0, dim=64),
                                 dict(scaling="yarn", scale=16.0, extent=64.0, layout="half"),
                                 dict(scaling="yarn", scale=2.0, extent=512.0, mscale=0.5, theta=500.0),
                                 dict(scaling="linear", scale=0.01)])
def test_scaled_positions_far_out(opt):
    """Positions up to the far corner of a 1024^3 grid, trained at a part of it."""
    plan, c = one_plan(200, edge=1024, seed=9)
    assert c.max() == 1023
    q, k = rows((200, 4, 96), "f32", 1).cuda(), rows((200, 4, 96), "f32", 2).cuda()
    check_forward(plan, c, q, k, opt, weights(96, 3))
    check_backward(plan, c, q, k, q, k, opt, weights(96, 3))


def test_largest_coordinate():
    c = np.array([[65534, 0, 0], [65533, 1, 2], [40000, 3, 7]], np.int32)
    plan = ssa.Plan(torch.from_numpy(c).cuda(), grid=(65535, 8, 8), r=0)
    q = rows((3, 2, 128), "f32", 1).cuda()
    check_forward(plan, c, q, q.clone(), {})


@pytest.mark.parametrize("n,h,hk", [(1, 1, 1), (1, 22, 22), (2, 1, 7), (17, 40, 1), (600, 1, 1), (2400, 3, 2)])
def test_sizes(n, h, hk):
    """One token to several tiles per CTA, one head to more heads than a warp pass takes."""
    plan, c = one_plan(n, seed=n)
    for dtype in ("f16", "f32"):
        q, k = rows((n, h, 96), dtype, 1).cuda(), rows((n, hk, 96), dtype, 2).cuda()
        check_forward(plan, c, q, k, {}, weights(96, 5))
        check_backward(plan, c, q, k, k[:, :1].expand(n, h, 96), q[:, :1].expand(n, hk, 96), {}, weights(96, 5))


@pytest.mark.slow
def test_large_shell_weights():
    """Many tiles per CTA: the sums over 1.32 million rows. A lane adds at most 2 * 60000 * 22 / (2 * 148 * 40) = 223
    rows, then 40 lanes and up to 14 + 32 CTAs."""
    n, h = 60000, 22
    plan, c = one_plan(n, edge=128, seed=1)
    q, k = rows((n, h, 96), "f16", 1).cuda(), rows((n, 2, 96), "f16", 2).cuda()
    dq, dk = rows((n, h, 96), "f16", 3).cuda(), rows((n, 2, 96), "f16", 4).cuda()
    check_forward(plan, c, q, k, {}, weights(96, 5))
    check_backward(plan, c, dq, dk, q, k, {}, weights(96, 5), depth=512)


def test_packed_sequences_and_rebuild():
    a, b = cells(40, 32, 1), cells(25, 64, 2)
    c = np.concatenate([a, b])
    plan = make_plan(c, [0, 40, 40, 65], [[32] * 3, [8] * 3, [64] * 3], 1)
    q, k = rows((65, 3, 64), "bf16", 1).cuda(), rows((65, 3, 64), "bf16", 2).cuda()
    check_forward(plan, c, q, k, {}, weights(64, 3))
    c2 = np.concatenate([cells(40, 32, 5), cells(25, 64, 6)])
    plan.rebuild(torch.from_numpy(c2).cuda())
    check_forward(plan, c2, q, k, {}, weights(64, 3))
    check_backward(plan, c2, q, k, k, q, {}, weights(64, 3))


# ---- memory: strides, alignment, in place, rows outside ----------------------------------------

@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("dtype", ["f16", "f32"])
def test_views_and_alignment(layout, dtype):
    n, h, D = 50, 3, 64
    plan, c = one_plan(n)
    opt, g = dict(layout=layout), weights(D, 5)
    fused = rows((n, 3 * h, D), dtype, 1).cuda()                       # queries and keys in a fused projection
    per_head = rows((n, h, 3, D), dtype, 2).cuda()                     # q, k, v of a head side by side
    head_major = rows((2, h, n, D), dtype, 3).cuda().transpose(1, 2)   # [h, n, D] storage
    odd = torch.zeros(n * h * D + 1, dtype=fused.dtype, device="cuda")[1:].view(n, h, D)
    odd.copy_(fused[:, :h])                                            # one element off every boundary
    wide = rows((n, h, D + 6), dtype, 4).cuda()[:, :, 2:2 + D]          # rows at 4-byte steps
    repeated = rows((n, 1, D), dtype, 5).cuda().expand(n, h, D)
    one_row = rows((1, 1, D), dtype, 6).cuda().expand(n, h, D)
    for q, k in ((fused[:, :h], fused[:, h:2 * h]), (per_head[:, :, 0], per_head[:, :, 1]), (head_major[0], head_major[1]),
                 (odd, wide), (repeated, one_row), (fused[:, 1:2], odd)):
        check_forward(plan, c, q, k, opt, g)
        check_backward(plan, c, k.contiguous()[:, :1].expand(q.shape), q.contiguous()[:, :1].expand(k.shape), q, k, opt, g)
        check_backward(plan, c, q, k, None, None, opt)
    # outputs in views: the memory between them is left as it was
    out = torch.full((n + 2, h, 3, D), 7.0, dtype=fused.dtype, device="cuda")
    check_forward(plan, c, fused[:, :h], fused[:, h:2 * h], opt, g, q_out=out[1:-1, :, 0], k_out=out[1:-1, :, 2])
    check_backward(plan, c, fused[:, :h], fused[:, h:2 * h], fused[:, h:2 * h], fused[:, :h], opt, g,
                   dq=out[1:-1, :, 2], dk=out[1:-1, :, 0])
    assert (out[:, :, 1] == 7).all() and (out[0] == 7).all() and (out[-1] == 7).all()


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("norm", [False, True])
def test_in_place(layout, norm):
    n, h, D = 700, 4, 96
    plan, c = one_plan(n)
    opt, g = dict(layout=layout, dim=48), weights(D, 5) if norm else (None, None)
    gd = [None if w is None else w.cuda() for w in g]
    r = ssa.Rotary(**opt)
    for src in (rows((n, 3 * h, D), "bf16", 1).cuda(), rows((n, h, 3, D), "bf16", 1).cuda()):
        part = (lambda t, i: t[:, i * h:(i + 1) * h]) if src.dim() == 3 else (lambda t, i: t[:, :, i])
        want = plan.rotary(part(src, 0), part(src, 1), r, *gd)
        buf = src.clone()
        got = plan.rotary(part(buf, 0), part(buf, 1), r, *gd, q_out=part(buf, 0), k_out=part(buf, 1))
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert torch.equal(part(buf, 2), part(src, 2))
        up = rows(src.shape, "bf16", 2).cuda()
        want = plan.rotary_backward(part(up, 0), part(up, 1), r, part(src, 0), part(src, 1), *gd)
        buf = up.clone()
        got = plan.rotary_backward(part(buf, 0), part(buf, 1), r, part(src, 0), part(src, 1), *gd, dq=part(buf, 0),
                                   dk=part(buf, 1))
        assert all(torch.equal(x, y) for x, y in zip(got, want))
        if norm:
            over = src.clone()      # over the forward's inputs
            got = plan.rotary_backward(part(up, 0), part(up, 1), r, part(over, 0), part(over, 1), *gd, dq=part(over, 0),
                                       dk=part(over, 1))
            assert all(torch.equal(x, y) for x, y in zip(got, want))


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("D,dim", [(32, 6), (64, 54), (96, 26), (96, 88), (128, 100), (128, 2)])
def test_half_layout_off_the_vectors(dtype, D, dim):
    """Sides of pairs that do not start at 16 bytes: aligned rows, rows that are not, in place, other rows' memory."""
    n, h = 333, 5
    plan, c = one_plan(n)
    opt = dict(layout="half", dim=dim, scaling="ntk", scale=2.0)
    fused = rows((n, 3 * h, D), dtype, 1).cuda()
    q, k = fused[:, :h], fused[:, h:2 * h - 2]
    odd = torch.zeros(n * h * D + 1, dtype=fused.dtype, device="cuda")[1:].view(n, h, D)
    odd.copy_(q)
    for w in (weights(D, 5), (None, None)):
        check_forward(plan, c, q, k, opt, w)
        check_forward(plan, c, odd, k, opt, w)
        check_backward(plan, c, k[:, :1].expand(n, h, D), q[:, :3], q, k, opt, w)
        r, wd = ssa.Rotary(**opt), [None if v is None else v.cuda() for v in w]
        want = plan.rotary(q, k, r, *wd)
        buf = fused.clone()
        got = plan.rotary(buf[:, :h], buf[:, h:2 * h - 2], r, *wd, q_out=buf[:, :h], k_out=buf[:, h:2 * h - 2])
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert torch.equal(buf[:, 2 * h - 2:], fused[:, 2 * h - 2:])
        grads = plan.rotary_backward(q, k, r, k[:, :1].expand(n, h, D), q[:, :3], *wd)
        buf = fused.clone()
        got = plan.rotary_backward(buf[:, :h], buf[:, h:2 * h - 2], r, k[:, :1].expand(n, h, D), q[:, :3], *wd,
                                   dq=buf[:, :h], dk=buf[:, h:2 * h - 2])
        assert all(torch.equal(a, b) for a, b in zip(got, grads))
        assert torch.equal(buf[:, 2 * h - 2:], fused[:, 2 * h - 2:])


def test_queries_only():
    plan, c = one_plan(33)
    q, k = rows((33, 3, 64), "f16", 1).cuda(), rows((33, 2, 64), "f16", 2).cuda()
    w, _ = weights(64, 3)
    w = w.cuda()
    both = plan.rotary(q, k, None, w, w)
    assert torch.equal(plan.rotary(q, None, None, w), both[0])
    assert torch.equal(plan.rotary(q), plan.rotary(q, k)[0])
    grads = plan.rotary_backward(q, k, None, q, k, w, w)
    dq, dw = plan.rotary_backward(q, None, None, q, None, w)
    assert torch.equal(dq, grads[0])
    # the queries alone are summed by other CTAs: the same terms in another order
    assert torch.allclose(dw, grads[2], rtol=1e-4, atol=1e-4)
    assert torch.equal(plan.rotary_backward(q), plan.rotary_backward(q, k)[0])


def test_large_strides():
    """Offsets that pass 32 bits: 40 tokens 2^27 elements apart in a 10.7 GB buffer."""
    n, D = 40, 64
    plan, c = one_plan(n)
    big = torch.empty((n - 1) * 2 ** 27 + 2 * D, dtype=torch.float16, device="cuda")
    q = torch.as_strided(big, (n, 2, D), (2 ** 27, D, 1))
    q.copy_(rows((n, 2, D), "f16", 1))
    check_forward(plan, c, q, q[:, :1], {}, weights(D, 2))
    src = q.clone()
    want = plan.rotary(src)
    plan.rotary(q, q_out=q)
    assert torch.equal(q, want)


# ---- special values ----------------------------------------------------------------------------

@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_infinities_and_nan_stay_in_their_row_and_pair(layout):
    n, h, D = 20, 3, 64
    plan, c = one_plan(n)
    x = rows((n, h, D), "f16", 1)
    x[3, 1, 2] = float("inf")       # a turned channel
    x[5, 0, 63] = float("nan")      # channels that pass through
    x[6, 2, 50] = -float("inf")
    r = ssa.Rotary(layout=layout, dim=48)
    clean = rows((n, h, D), "f16", 1).cuda()
    got, want = plan.rotary(x.cuda(), None, r), plan.rotary(clean, None, r)
    mate = 3 if layout == "interleaved" else 26
    touched = torch.zeros(n, h, D, dtype=torch.bool, device="cuda")
    touched[3, 1, 2] = touched[3, 1, mate] = touched[5, 0, 63] = touched[6, 2, 50] = True
    assert torch.equal(got[~touched], want[~touched])
    assert got[6, 2, 50] == -float("inf") and got[5, 0, 63].isnan() and not got[3, 1, 2].isfinite()
    w = weights(D, 2)[0].cuda()
    got, want = plan.rotary(x.cuda(), None, r, w), plan.rotary(clean, None, r, w)
    rowmask = touched.any(2)
    assert torch.equal(got[~rowmask], want[~rowmask])
    dq, dw = plan.rotary_backward(clean, None, r, x.cuda(), None, w)
    dq0, _ = plan.rotary_backward(clean, None, r, clean, None, w)
    assert torch.equal(dq[~rowmask], dq0[~rowmask])
    assert not dw.isfinite().all()      # the weights' sums see every row


def test_zero_rows():
    plan, c = one_plan(9)
    z = torch.zeros(9, 2, 32, device="cuda")
    w = torch.ones(32, device="cuda")
    assert torch.equal(plan.rotary(z, None, None, w), z)
    g = rows((9, 2, 32), "f32", 1).cuda()
    check_backward(plan, c, g, g.clone(), z, z, {}, (w.cpu(), w.cpu()))
    # large and small magnitudes of the type
    big = torch.full((9, 2, 32), 3e4, dtype=torch.float16, device="cuda")
    check_forward(plan, c, big, big.clone(), {}, (w.cpu(), w.cpu()))
    small = torch.full((9, 2, 32), 6e-8, dtype=torch.float16, device="cuda")
    check_forward(plan, c, small, small.clone(), {}, (w.cpu(), w.cpu()), eps=0.0)


# ---- streams, graphs, repeats --------------------------------------------------------------------

def test_equal_bits_and_side_streams():
    n = 3000
    c = cells(n, 64, 3)
    s = torch.cuda.Stream()
    plan = ssa.Plan(torch.from_numpy(c).cuda(), grid=(64,) * 3, r=0)
    q, k = rows((n, 8, 64), "bf16", 1).cuda(), rows((n, 8, 64), "bf16", 2).cuda()
    w = [v.cuda() for v in weights(64, 3)]
    want = plan.rotary_backward(q, k, None, k, q, *w)
    torch.cuda.synchronize()
    outs = []
    for i in range(6):      # two streams at once, each call with buffers of its own
        with torch.cuda.stream(s) if i % 2 else torch.cuda.stream(torch.cuda.default_stream()):
            outs.append(plan.rotary_backward(q, k, None, k, q, *w))
    torch.cuda.synchronize()
    for got in outs:
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    # a plan bound to a stream
    with torch.cuda.stream(s):
        cd = torch.from_numpy(c).cuda()
    s.synchronize()
    bound = ssa.Plan(cd, grid=(64,) * 3, r=0, stream=s)
    got = bound.rotary_backward(q, k, None, k, q, *w)
    s.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_captured_and_replayed():
    """Two graphs of one plan, replayed at the same time on two streams, on changed inputs."""
    n = 2000
    plan, c = one_plan(n)
    w = [v.cuda() for v in weights(64, 3)]
    sets = []
    for i in range(2):
        q, k = rows((n, 8, 64), "f16", 10 + i).cuda(), rows((n, 8, 64), "f16", 20 + i).cuda()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            plan.rotary_backward(q, k, None, k, q, *w)
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            f = plan.rotary(q, k, None, *w)
            b = plan.rotary_backward(f[0], f[1], None, q, k, *w)
        sets.append((q, k, s, graph, f, b))
    for i, (q, k, *_ ) in enumerate(sets):
        q.copy_(rows((n, 8, 64), "f16", 30 + i))
        k.copy_(rows((n, 8, 64), "f16", 40 + i))
    torch.cuda.synchronize()
    for _ in range(5):
        for q, k, s, graph, f, b in sets:
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for q, k, s, graph, f, b in sets:
        ff = plan.rotary(q, k, None, *w)
        bb = plan.rotary_backward(ff[0], ff[1], None, q, k, *w)
        assert all(torch.equal(x, y) for x, y in zip(list(f) + list(b), list(ff) + list(bb)))


# ---- with the attention --------------------------------------------------------------------------

@pytest.mark.parametrize("name,dtype", [("tiny", "f32"), ("small", "bf16")])
def test_operator_then_attention_is_the_fused_prologue(name, dtype):
    """ssa_rotary followed by ssa_forward against ssa_forward_prologue. Both round the transformed
    queries and keys to the type; where their fp32 arithmetic differs an element may round to the other
    neighbour, one step, which moves the output within the stated tolerance of the method."""
    cfg = workloads.CONFIGS[name]
    c, cu, g = coords_of(name)
    t = to_gpu(tensors_of(name))
    plan = make_plan(c, cu, g, cfg.radius)
    D = t["Q"].shape[2]
    w = [v.cuda() for v in weights(D, 7)]
    fused, sel0 = plan.forward_prologue(t["Q"], t["K"], t["V"], t["gates"], t["Wc"], cfg.topk, *w, return_sel=True)
    q, k = plan.rotary(t["Q"], t["K"], None, *w, eps=1e-6)
    out, sel = plan.forward(q, k, t["V"], t["gates"], t["Wc"], cfg.topk, return_sel=True)
    torch.cuda.synchronize()
    same = (sel0 == sel).all(2)
    assert same.float().mean() > 0.9
    d = (out.double() - fused.double())[same]
    assert d.abs().max() <= (1e-5 if dtype == "f32" else 2e-2)
    assert d.norm() <= (1e-5 if dtype == "f32" else 5e-3) * fused.double()[same].norm()


def test_training_step_through_prologue_and_attention():
    """Gradients of sum(dO * ssa(rotary(q), rotary(k), v)) with respect to q, k and the weights, with all blocks
    selected (the selection is then no function of the inputs), against central differences of the
    kernels' own fp32 forward along random directions."""
    c, cu, g = coords_of("tiny")
    t = to_gpu(tensors_of("tiny", with_grad_out=True))
    n = 400
    lo = np.sort(np.random.default_rng(1).choice(len(c), n, replace=False))
    c = np.ascontiguousarray(c[lo])
    topk = 32
    plan = make_plan(c, [0, n], g, 2)
    keep = torch.from_numpy(c[:, 2] < 16).cuda()
    assert plan.num_blocks > 0
    q, k, v, gates, dO = (t[x][torch.from_numpy(lo).cuda()].contiguous() for x in ("Q", "K", "V", "gates", "dO"))
    if plan.num_blocks > topk:      # keep the shell's lower half: at most 32 blocks
        idx = keep.nonzero()[:, 0]
        c = np.ascontiguousarray(c[idx.cpu().numpy()])
        q, k, v, gates, dO = (x[idx].contiguous() for x in (q, k, v, gates, dO))
        plan = make_plan(c, [0, len(c)], g, 2)
    assert plan.num_blocks <= topk
    w = [x.cuda() for x in weights(32, 3)]
    rot = ssa.Rotary(layout="half", scaling="ntk", scale=2.0)

    def loss(q, k, gq, gk):
        a, b = plan.rotary(q, k, rot, gq, gk)
        return float((plan.forward(a, b, v, gates, t["Wc"], topk).double() * dO.double()).sum())

    a, b = plan.rotary(q, k, rot, *w)
    da, db, _ = plan.backward(a, b, v, gates, t["Wc"], dO, topk)
    grads = plan.rotary_backward(da, db, rot, q, k, *w)
    args = [q, k, *w]
    gen = torch.Generator(device="cuda").manual_seed(5)
    h = 2e-2
    for i in range(4):
        # along the gradient, where the change is largest, and along a mix of it and noise
        noise = torch.randn(args[i].shape, device="cuda", generator=gen)
        for d in (grads[i], grads[i] + noise * grads[i].norm() / noise.norm()):
            d = d / d.norm() * args[i].norm() ** 0.5
            f = lambda s: loss(*[x + s * d if j == i else x for j, x in enumerate(args)])  # noqa: E731
            # fourth-order differences: truncation h^4, rounding 2^-24 * sqrt(terms) of the loss over h
            num = (8 * (f(h) - f(-h)) - (f(2 * h) - f(-2 * h))) / (12 * h)
            want = float((grads[i].double() * d.double()).sum())
            print(i, num, want)
            assert abs(num - want) <= 2e-2 * abs(want)
