"""ssa_group_norm and ssa_group_norm_backward through the C ABI against the fp64 references, on every element."""
import ctypes

import numpy as np
import pytest
import torch

import operator_refs as ref
import workloads
from ssa_testlib import coords_of, make_plan, tensors_of, to_gpu

pytestmark = pytest.mark.gpu

import spatial_sparse_attention_b200 as ssa  # noqa: E402

RAGGED = (700, 0, 1, 633)
_plans = {}


def plan_of(seqs):
    """A plan of sequences of these lengths; the cells do not matter."""
    if seqs not in _plans:
        cu = np.concatenate([[0], np.cumsum(seqs)])
        at = np.concatenate([np.arange(n) for n in seqs])
        c = np.stack([at // 4096, at // 64 % 64, at % 64], 1).astype(np.int32)
        _plans[seqs] = make_plan(c, cu.tolist(), [[128] * 3] * len(seqs), 0), cu
    return _plans[seqs]


def features(n, C, dtype, seed):
    """Rows with a mean and a spread of their own per channel."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, C, generator=g) * (0.5 + torch.rand(C, generator=g)) + 0.5 * torch.randn(C, generator=g)
    return x.to(ref.DTYPES[dtype])


def weights(C, seed):
    g = torch.Generator().manual_seed(seed)
    return 1 + 0.2 * torch.randn(C, generator=g), 0.2 * torch.randn(C, generator=g)


def dev(w):
    return [None if v is None else v.cuda() for v in w]


def f64s(w):
    return [None if v is None else ref.f64(v) for v in w]


def check_forward(plan, cu, x, groups, w=(None, None), eps=1e-5, act=None, what="", **call):
    dtype = {v: n for n, v in ref.DTYPES.items()}[x.dtype]
    want = ref.group_norm(ref.f64(x), cu, groups, *f64s(w), eps, act)
    y, mean, rstd = plan.group_norm(x, groups, *dev(w), eps=eps, activation=act, return_stats=True, **call)
    torch.cuda.synchronize()
    ref.check(y, *want[0], dtype, f"{what} y")
    ref.check(mean, *want[1], "f32", f"{what} mean")
    ref.check(rstd, *want[2], "f32", f"{what} rstd")
    return y, mean, rstd


def check_backward(plan, cu, dy, x, groups, w=(None, None), eps=1e-5, act=None, what="", **call):
    dtype = {v: n for n, v in ref.DTYPES.items()}[x.dtype]
    _, mean, rstd = plan.group_norm(x, groups, *dev(w), eps=eps, activation=act, return_stats=True)
    want = ref.group_norm_grad(ref.f64(dy), ref.f64(x), ref.f64(mean), ref.f64(rstd), cu, groups, *f64s(w), act)
    got = plan.group_norm_backward(dy, x, mean, rstd, groups, *dev(w), activation=act, **call)
    torch.cuda.synchronize()
    for name, a, b, t in zip(("dx", "dgamma", "dbeta"), got, want, (dtype, "f32", "f32")):
        ref.check(a, *b, t, f"{what} {name}")
    return got


# ---- refusals first: none of these calls may reach a kernel ------------------------------------

def test_refusals():
    plan, _ = plan_of(RAGGED)
    small, _ = plan_of((1,))
    n = sum(RAGGED)
    x = torch.zeros(n, 64, device="cuda")
    w, st = torch.ones(64, device="cuda"), torch.zeros(4, 8, device="cuda")
    before = ssa.launch_count()
    for bad in (x.cpu(), x[:-1], x[0], x[:, ::2], x.t(), x[:, None]):
        with pytest.raises(ValueError):
            plan.group_norm(bad, 8)
    for kw in (dict(gamma=w[:8], beta=w), dict(gamma=w.half(), beta=w), dict(gamma=w.cpu(), beta=w),
               dict(out=x[:, :32]), dict(out=x.half()), dict(activation="relu")):
        with pytest.raises(ValueError):
            plan.group_norm(x, 8, **kw)
    for groups in (0, -1):
        with pytest.raises(ValueError):
            plan.group_norm(x, groups)
    for call in (lambda: plan.group_norm(x, 5), lambda: plan.group_norm(x, 128), lambda: plan.group_norm(x.double(), 8),
                 lambda: plan.group_norm(x, 8, eps=-1.0), lambda: plan.group_norm(x, 8, eps=float("nan")),
                 lambda: plan.group_norm(x, 8, eps=float("inf")), lambda: plan.group_norm(x, 8, gamma=w),
                 lambda: plan.group_norm(x, 8, beta=w), lambda: plan.group_norm(x.half(), 8, out=x[:1].half().expand(n, 64))):
        with pytest.raises(ssa.SSAError, match="INVALID_ARG"):
            call()
    buf = torch.zeros(n + 1, 96, device="cuda")
    for a, b in ((buf[:-1, :64], buf[1:, :64]), (buf[:-1, :64], buf[:-1, 32:])):     # overlapping, not the same
        with pytest.raises(ssa.SSAError, match="INVALID_ARG"):
            plan.group_norm(a, 8, out=b)
        with pytest.raises(ssa.SSAError, match="INVALID_ARG"):
            plan.group_norm_backward(a, x, st, st, 8, dx=b)
        with pytest.raises(ssa.SSAError, match="INVALID_ARG"):
            plan.group_norm_backward(x, a, st, st, 8, dx=b)
    for m in (st[:3], st.half(), st.cpu(), None):
        with pytest.raises(ValueError):
            plan.group_norm_backward(x, x, m, st, 8)
    with pytest.raises(ValueError):
        plan.group_norm_backward(x.half(), x, st, st, 8)
    with pytest.raises(ssa.SSAError, match="UNSUPPORTED"):
        small.group_norm(torch.zeros(1, 65537, device="cuda"), 1)
    assert ssa.launch_count() == before


def test_c_refusals():
    plan, _ = plan_of((4,))
    x = torch.zeros(4, 16, device="cuda")
    s = torch.zeros(2, device="cuda")
    a = ctypes.addressof
    ok = ssa._Rows(x.data_ptr(), 16)

    def fwd(x_, y_, mean=None, rstd=None, act=0, dt=0):
        return ssa.lib.ssa_group_norm(plan._h, x_ and a(x_), 16, 2, None, None, 1e-5, act, dt, y_ and a(y_), mean, rstd, None)

    def bwd(dy, x_, dx, mean=s.data_ptr(), rstd=s.data_ptr(), dg=s.data_ptr(), db=s.data_ptr()):
        return ssa.lib.ssa_group_norm_backward(plan._h, dy and a(dy), x_ and a(x_), mean, rstd, 16, 2, None, None, 0, 0,
                                               dx and a(dx), dg, db, None)

    before = ssa.launch_count()
    assert fwd(None, ok) == 1 and fwd(ok, None) == 1
    assert fwd(ok, ok, mean=s.data_ptr()) == 1 and fwd(ok, ok, rstd=s.data_ptr()) == 1
    assert fwd(ok, ok, act=3) == 1 and fwd(ok, ok, act=-1) == 1 and fwd(ok, ok, dt=3) == 1
    for bad in (ssa._Rows(None, 16), ssa._Rows(x.data_ptr() + 2, 16), ssa._Rows(x.data_ptr(), -16), ssa._Rows(x.data_ptr(), 1 << 40)):
        assert fwd(bad, ok) == 1 and fwd(ok, bad) == 1
        assert bwd(bad, ok, ok) == 1 and bwd(ok, bad, ok) == 1 and bwd(ok, ok, bad) == 1
    assert fwd(ok, ssa._Rows(x.data_ptr(), 15)) == 1
    assert bwd(None, ok, ok) == 1 and bwd(ok, None, ok) == 1 and bwd(ok, ok, None) == 1
    for kw in (dict(mean=None), dict(rstd=None), dict(dg=None), dict(db=None)):
        assert bwd(ok, ok, ok, **kw) == 1
    assert ssa.launch_count() == before


def test_c_refuses_misaligned_arrays():
    plan, _ = plan_of((4,))
    x = torch.zeros(4, 16, device="cuda")
    w = torch.ones(64, device="cuda")
    a, p = ctypes.addressof, w.data_ptr()
    v = ssa._Rows(x.data_ptr(), 16)
    before = ssa.launch_count()
    for bad in range(4):
        at = [p, p + 64, p + 128, p + 160]
        at[bad] += 2
        assert ssa.lib.ssa_group_norm(plan._h, a(v), 16, 2, at[0], at[1], 1e-5, 0, 0, a(v), at[2], at[3], None) == 1
        assert ssa.lib.ssa_group_norm_backward(plan._h, a(v), a(v), p + 128, p + 160, 16, 2, at[0], at[1], 0, 0, a(v), at[2],
                                               at[3], None) == 1
    assert ssa.launch_count() == before


# ---- values ------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("act", [None, "silu", "gelu"])
@pytest.mark.parametrize("C,groups", [(64, 8), (67, 1), (96, 32), (2112, 32), (22, 22), (4, 2), (1, 1), (130, 2), (1040, 16)])
def test_types_activations_widths(dtype, act, C, groups):
    plan, cu = plan_of(RAGGED)
    x, dy, w = features(cu[-1], C, dtype, C).cuda(), features(cu[-1], C, dtype, C + 1).cuda(), weights(C, 3)
    check_forward(plan, cu, x, groups, w, act=act)
    check_backward(plan, cu, dy, x, groups, w, act=act)


@pytest.mark.parametrize("seqs", [(1,), (2,), (0, 3), (5, 0), (0, 1, 0, 1, 0), (1,) * 300, (17, 300, 2, 2000), (4096,)])
@pytest.mark.parametrize("C,groups", [(64, 8), (264, 1), (33, 3)])
def test_sequences(seqs, C, groups):
    """One token to a few tiles; empty sequences first, between and last; many sequences in one tile."""
    plan, cu = plan_of(seqs)
    for dtype in ("f16", "f32"):
        x, dy, w = features(cu[-1], C, dtype, 5).cuda(), features(cu[-1], C, dtype, 6).cuda(), weights(C, 3)
        check_forward(plan, cu, x, groups, w, act="silu")
        check_backward(plan, cu, dy, x, groups, w, act="silu")
        check_forward(plan, cu, x, groups)
        check_backward(plan, cu, dy, x, groups)


@pytest.mark.parametrize("C,groups,dtype", [(2112, 32, "f16"), (512, 32, "bf16"), (100, 4, "f32"), (2112, 1, "f16"), (8, 8, "f32")])
def test_longer_sequences(C, groups, dtype):
    """Several tiles per sequence with whole rows per thread."""
    plan, cu = plan_of((9000, 1, 14500))
    x, dy, w = features(cu[-1], C, dtype, 1).cuda(), features(cu[-1], C, dtype, 2).cuda(), weights(C, 3)
    check_forward(plan, cu, x, groups, w, act="silu")
    check_backward(plan, cu, dy, x, groups, w, act="silu")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("C,groups", [(100, 4), (36, 2), (1658, 1), (211, 1), (2045, 5), (12, 12)])
def test_rows_of_every_alignment(dtype, C, groups):
    """Rows that start at multiples of 2, 4, 8 and 16 bytes, with a part of a vector at their ends."""
    plan, cu = plan_of((17, 300, 2, 2000))
    buf = torch.full((2319 + 1, C), 7.0, dtype=ref.DTYPES[dtype], device="cuda")
    x, dy, w = features(2319, C, dtype, C).cuda(), features(2319, C, dtype, 2).cuda(), weights(C, 3)
    check_forward(plan, cu, x, groups, w, act="gelu", out=buf[:-1])
    assert (buf[-1] == 7).all()
    buf.fill_(7.0)
    check_backward(plan, cu, dy, x, groups, w, act="gelu", dx=buf[1:])
    assert (buf[0] == 7).all()


def test_wide_rows():
    plan, cu = plan_of((3, 2))
    for C, groups in ((65536, 1), (65535, 3), (65536, 65536)):
        x, dy = features(5, C, "f16", 1).cuda(), features(5, C, "f16", 2).cuda()
        check_forward(plan, cu, x, groups, act="gelu")
        if groups < C:
            check_backward(plan, cu, dy, x, groups, act="gelu")


def test_values_far_from_zero():
    """A mean a thousand times the spread: a difference of large sums would lose the variance in fp32."""
    plan, cu = plan_of((4096,))
    x = (1000 + torch.randn(4096, 64, generator=torch.Generator().manual_seed(1))).cuda()
    check_forward(plan, cu, x, 8)
    x[:, 8:16] = 5.0          # a group without variance
    y, mean, rstd = plan.group_norm(x, 8, return_stats=True)
    assert (y[:, 8:16] == 0).all() and mean[0, 1] == 5.0 and float(rstd[0, 1]) == pytest.approx(1e-5 ** -0.5, rel=1e-6)
    # one large value among small ones, first and last: the mean and the variance keep the small ones' part
    for at in (0, 4095):
        x = torch.randn(4096, 64, generator=torch.Generator().manual_seed(2))
        x[at, 3] = 3e4
        xd = x.double().numpy()
        _, mean, rstd = plan.group_norm(x.cuda(), 8, return_stats=True)
        m, var, *_ = ref.norm_stats(xd, cu, 8)
        # the pivot's thread: 64 terms of 3e4 (mean, of 32768 values), and 64 (70 u) of its square
        assert abs(float(mean[0, 0]) - m[0, 0]) <= 64 * 64 * ref.U * 3e4 / 32768 + 200 * ref.U
        assert abs(float(rstd[0, 0]) ** -2 - 1e-5 - var[0, 0]) <= (64 * 70 + 8) * ref.U * var[0, 0]


def test_activation_tails():
    """Values where exp overflows or the distribution function underflows."""
    plan, cu = plan_of((64,))
    b = torch.tensor([-200.0, -90.0, -30.0, -12.0, -5.0, -3.0, 0.0, 3.0, 12.0, 30.0, 90.0, 200.0])
    x = features(64, 12, "f32", 1).cuda()
    for act in ("silu", "gelu"):
        y = check_forward(plan, cu, x, 3, (torch.full((12,), 0.1), b), act=act)[0]
        assert y.isfinite().all()
        check_backward(plan, cu, features(64, 12, "f32", 2).cuda(), x, 3, (torch.full((12,), 0.1), b), act=act)


@pytest.mark.parametrize("dtype", ["f16", "f32"])
def test_nan_stays_in_its_sequence_and_group(dtype):
    plan, cu = plan_of((50, 60, 40))
    x, dy = features(150, 64, dtype, 1).cuda(), features(150, 64, dtype, 2).cuda()
    w = dev(weights(64, 3))
    clean = plan.group_norm(x, 8, *w, activation="silu", return_stats=True)
    cg = plan.group_norm_backward(dy, x, *clean[1:], 8, *w, activation="silu")
    for bad in (float("nan"), float("inf"), -float("inf")):
        z = x.clone()
        z[70, 20] = bad
        got = plan.group_norm(z, 8, *w, activation="silu", return_stats=True)
        hit = torch.zeros(150, 64, dtype=torch.bool, device="cuda")
        hit[50:110, 16:24] = True
        assert torch.equal(got[0][~hit], clean[0][~hit]) and got[0][hit].isnan().all()
        for a, b in zip(got[1:], clean[1:]):
            a = a.clone()
            assert not a[1, 2].isfinite()
            a[1, 2] = b[1, 2]
            assert torch.equal(a, b)
        gg = plan.group_norm_backward(dy, z, *got[1:], 8, *w, activation="silu")
        assert torch.equal(gg[0][~hit], cg[0][~hit])
        out = torch.ones(64, dtype=torch.bool, device="cuda")
        out[16:24] = False
        assert torch.equal(gg[1][out], cg[1][out]) and torch.equal(gg[2][out], cg[2][out])
        assert gg[0][hit].isnan().all() and gg[1][~out].isnan().all()


# ---- memory --------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_views_and_alignment(dtype):
    plan, cu = plan_of(RAGGED)
    n, C = cu[-1], 96
    fused = features(n, 3 * C, dtype, 1).cuda()
    odd = torch.zeros(n * C + 1, dtype=fused.dtype, device="cuda")[1:].view(n, C)
    odd.copy_(fused[:, :C])
    wide = features(n, C + 7, dtype, 2).cuda()[:, 3:3 + C]
    same_row = features(1, C, dtype, 3).cuda().expand(n, C)
    w = weights(C, 4)
    for x, dy in ((fused[:, C:2 * C], fused[:, :C]), (odd, wide), (wide, odd), (fused[:, :C], same_row)):
        check_forward(plan, cu, x, 8, w, act="silu")
        check_backward(plan, cu, dy, x, 8, w, act="silu")
    buf = torch.full((n + 2, 3 * C), 7.0, dtype=fused.dtype, device="cuda")
    check_forward(plan, cu, fused[:, :C], 8, w, out=buf[1:-1, C:2 * C])
    check_backward(plan, cu, fused[:, :C], fused[:, C:2 * C], 8, w, dx=buf[1:-1, C:2 * C])
    assert (buf[:, :C] == 7).all() and (buf[:, 2 * C:] == 7).all() and (buf[0] == 7).all() and (buf[-1] == 7).all()


def test_one_row_repeated():
    """A broadcast input: no variance over the tokens, all of it over the channels."""
    plan, cu = plan_of((300,))
    x = features(1, 64, "f32", 3).cuda().expand(300, 64)
    check_forward(plan, cu, x, 4, act="silu")
    check_backward(plan, cu, features(300, 64, "f32", 4).cuda(), x, 4, act="silu")


@pytest.mark.parametrize("C,groups", [(96, 8), (67, 1), (2112, 32)])
def test_in_place(C, groups):
    plan, cu = plan_of((2000, 3000))
    x, dy, w = features(5000, C, "f16", 1).cuda(), features(5000, C, "f16", 2).cuda(), dev(weights(C, 3))
    want = plan.group_norm(x, groups, *w, activation="silu", return_stats=True)
    grads = plan.group_norm_backward(dy, x, *want[1:], groups, *w, activation="silu")
    buf = x.clone()
    got = plan.group_norm(buf, groups, *w, activation="silu", out=buf, return_stats=True)
    assert got[0].data_ptr() == buf.data_ptr() and all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.equal(plan.group_norm(x, groups, *w, activation="silu"), want[0])
    for over in (0, 1):
        bufs = [dy.clone(), x.clone()]
        got = plan.group_norm_backward(*bufs, *want[1:], groups, *w, activation="silu", dx=bufs[over])
        assert all(torch.equal(a, b) for a, b in zip(got, grads))
    same = plan.group_norm_backward(x, x, *want[1:], groups, *w, activation="silu")   # one tensor as both inputs
    other = plan.group_norm_backward(x.clone(), x, *want[1:], groups, *w, activation="silu")
    assert all(torch.equal(a, b) for a, b in zip(same, other))


def test_large_strides():
    """Offsets that pass 32 bits: 40 tokens 2^27 elements apart in a 10.7 GB buffer."""
    plan, cu = plan_of((39, 1))
    big = torch.empty(39 * 2 ** 27 + 64, dtype=torch.float16, device="cuda")
    x = torch.as_strided(big, (40, 64), (2 ** 27, 1))
    x.copy_(features(40, 64, "f16", 1))
    src = x.clone()
    want = plan.group_norm(src, 4, return_stats=True)
    check_forward(plan, cu, x, 4)
    check_backward(plan, cu, features(40, 64, "f16", 2).cuda(), x, 4)
    plan.group_norm(x, 4, out=x)
    assert torch.equal(x, want[0])


# ---- streams, graphs, repeats --------------------------------------------------------------------

def test_equal_bits_and_side_streams():
    plan, cu = plan_of((9000, 1, 14500))
    n = cu[-1]
    x, dy, w = features(n, 512, "bf16", 1).cuda(), features(n, 512, "bf16", 2).cuda(), dev(weights(512, 3))

    def both(p):
        y, m, r = p.group_norm(x, 32, *w, activation="silu", return_stats=True)
        return (y, m, r) + p.group_norm_backward(dy, x, m, r, 32, *w, activation="silu")

    want = both(plan)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    outs = []
    for i in range(6):
        with torch.cuda.stream(s) if i % 2 else torch.cuda.stream(torch.cuda.default_stream()):
            outs.append(both(plan))
    torch.cuda.synchronize()
    for got in outs:
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    at = np.concatenate([np.arange(k) for k in (9000, 1, 14500)])
    c = np.stack([at // 4096, at // 64 % 64, at % 64], 1).astype(np.int32)
    cd = torch.from_numpy(c).cuda()
    torch.cuda.synchronize()
    bound = ssa.Plan(cd, r=0, cu_seqlens=cu.tolist(), grids=[[128] * 3] * 3, stream=s)
    got = both(bound)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("C,groups,seqs", [(512, 32, (2000, 0, 900)), (64, 8, (300,)), (2112, 32, (9000, 1, 14500))])
def test_captured_and_replayed(C, groups, seqs):
    """Two graphs of one plan, replayed at the same time on two streams, on changed inputs."""
    plan, cu = plan_of(seqs)
    w = dev(weights(C, 3))
    sets = []
    for i in range(2):
        x, dy = features(cu[-1], C, "f16", 10 + i).cuda(), features(cu[-1], C, "f16", 20 + i).cuda()
        s = torch.cuda.Stream()
        torch.cuda.synchronize()

        def both():
            y, m, r = plan.group_norm(x, groups, *w, activation="gelu", return_stats=True)
            return (y, m, r) + plan.group_norm_backward(dy, x, m, r, groups, *w, activation="gelu")

        with torch.cuda.stream(s):
            both()
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            outs = both()
        sets.append((x, dy, s, graph, outs, both))
    for i, (x, dy, *_) in enumerate(sets):
        x.copy_(features(cu[-1], C, "f16", 30 + i))
        dy.copy_(features(cu[-1], C, "f16", 40 + i))
    torch.cuda.synchronize()
    for _ in range(5):
        for x, dy, s, graph, outs, both in sets:
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for x, dy, s, graph, outs, both in sets:
        assert all(torch.equal(a, b) for a, b in zip(outs, both()))


# ---- with the other operators ----------------------------------------------------------------------

def test_profiled_by_name():
    plan, cu = plan_of((300,))
    x = features(300, 64, "f32", 1).cuda()
    ssa.profile_reset()
    ssa.profile_enable(True)
    try:
        _, m, r = plan.group_norm(x, 8, return_stats=True)
        plan.group_norm_backward(x, x, m, r, 8)
        plan.rotary(x.view(300, 2, 32))
        plan.rotary_backward(x.view(300, 2, 32))
        got = ssa.profile_read()
    finally:
        ssa.profile_enable(False)
        ssa.profile_reset()
    for name in ("group_norm", "group_norm_backward", "rotary", "rotary_backward"):
        assert got[name][1] == 1 and got[name][0] > 0


def test_layer_from_features_to_attention_and_back():
    """norm -> activation -> projection -> rotary positions -> attention, forward and gradients, against the same
    chain with the fp64 references at the operators' own roundings: each operator is checked at the
    values that the one before it handed on."""
    cfg = workloads.CONFIGS["small"]
    c, cu, g = coords_of("small")
    t = to_gpu(tensors_of("small", with_grad_out=True))
    plan = make_plan(c, cu, g, cfg.radius)
    n, H, D = t["Q"].shape
    cu = np.asarray(cu)
    C = 96
    x, w = features(n, C, "bf16", 1).cuda(), weights(C, 2)
    proj = (torch.randn(C, 3 * H * D, generator=torch.Generator().manual_seed(3)) / C ** 0.5).bfloat16().cuda()
    gq, gk = (0.5 + torch.rand(D, generator=torch.Generator().manual_seed(4))).cuda(), torch.ones(D, device="cuda")
    rot = ssa.Rotary(layout="half", dim=D // 2, scaling="yarn", scale=2.0, extent=64.0)
    opt = dict(layout="half", dim=D // 2, scaling="yarn", scale=2.0, extent=64.0)
    y, mean, rstd = check_forward(plan, cu, x, 8, w, act="silu", what="norm")
    qkv = (y @ proj).view(n, 3 * H, D)
    q, k = qkv[:, :H], qkv[:, H:2 * H]
    qr, kr = plan.rotary(q, k, rot, gq, gk)
    for a, b, gam in ((q, qr, gq), (k, kr, gk)):
        ref.check(b, *ref.rotary(ref.f64(a), c, ref.f64(gam), **opt), "bf16", "rotary")
    v = qkv[:, 2 * H:].contiguous()
    o = plan.forward(qr, kr, v, t["gates"], t["Wc"], cfg.topk)
    assert o.isfinite().all()
    dq, dk, dv = plan.backward(qr, kr, v, t["gates"], t["Wc"], t["dO"], cfg.topk)
    dqkv = torch.empty_like(qkv)
    dqkv[:, 2 * H:] = dv
    _, _, dgq, dgk = plan.rotary_backward(dq, dk, rot, q, k, gq, gk, dq=dqkv[:, :H], dk=dqkv[:, H:2 * H])
    for up, a, gam, got, dw in ((dq, q, gq, dqkv[:, :H], dgq), (dk, k, gk, dqkv[:, H:2 * H], dgk)):
        r, (dg, mag) = ref.rotary_grad(ref.f64(up), c, ref.f64(a), ref.f64(gam), **opt)
        ref.check(got, *r, "bf16", "rotary gradient")
        ref.check(dw, dg, 512 * ref.U * mag, "f32", "weights' gradient")
    dy = dqkv.view(n, -1) @ proj.t()
    grads = plan.group_norm_backward(dy, x, mean, rstd, 8, *dev(w), activation="silu")
    want = ref.group_norm_grad(ref.f64(dy), ref.f64(x), ref.f64(mean), ref.f64(rstd), cu, 8, *f64s(w), "silu")
    for a, b, dt in zip(grads, want, ("bf16", "f32", "f32")):
        ref.check(a, *b, dt, "norm gradient")


def test_gradient_against_differences_of_the_forward():
    """sum(dy * group_norm(x)) in fp32 along the gradient and along noise, fourth-order differences."""
    plan, cu = plan_of((120, 0, 1, 80))
    x, dy, w = features(201, 24, "f32", 1).cuda(), features(201, 24, "f32", 2).cuda(), dev(weights(24, 3))
    for act in (None, "silu", "gelu"):
        args = [x, *w]
        _, m, r = plan.group_norm(x, 3, *w, activation=act, return_stats=True)
        grads = plan.group_norm_backward(dy, x, m, r, 3, *w, activation=act)
        f = lambda a: float((plan.group_norm(a[0], 3, a[1], a[2], activation=act).double() * dy.double()).sum())  # noqa: E731
        h = 2e-2
        gen = torch.Generator(device="cuda").manual_seed(5)
        for i in range(3):
            noise = torch.randn(args[i].shape, device="cuda", generator=gen)
            for d in (grads[i], grads[i] + noise * grads[i].norm() / noise.norm()):
                d = d / d.norm()
                at = lambda s: f([v + s * d if j == i else v for j, v in enumerate(args)])  # noqa: E731
                num = (8 * (at(h) - at(-h)) - (at(2 * h) - at(-2 * h))) / (12 * h)
                want = float((grads[i].double() * d.double()).sum())
                # h^4 of the fifth derivative (of order one per unit step) and, over h, the fp32 rounding of
                # 4824 outputs of size one: sqrt(4824) * 2^-24 * 1.5 / h = 3e-4
                assert abs(num - want) <= 2e-3 * abs(want) + 1e-3
