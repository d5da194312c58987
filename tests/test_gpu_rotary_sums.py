"""The weights' gradients of the rotary gradient over many rows: the sums keep their precision however many rows a
thread adds up."""
import pytest
import torch

import operator_refs as ref
from test_gpu_rotary import check_backward, check_forward, one_plan, rows, weights

pytestmark = pytest.mark.gpu

import spatial_sparse_attention_b200 as ssa  # noqa: E402


@pytest.mark.parametrize("n,heads,keys,D,dtype", [(200000, 1, 32, 128, "f32"), (200000, 1, 40, 96, "bf16"), (60000, 22, 2, 96, "f16")])
def test_equal_terms_over_many_rows(n, heads, keys, D, dtype):
    """Every row the same, in channels that pass through: the gradient of weight c is rows * dy_c * n_c, sums of equal terms whose
    roundings all point one way. Few query heads beside many key heads leave the queries few CTAs, so that a
    thread adds up thousands of rows.

    Error of a term, u = 2^-24: the row's sum of squares (at most 16 / 2 + 1 + 4 additions and the mean, 14 u), halved
    by the root, rsqrtf (2 ulp, 4 u) and x * inv: 12 u. A chain of at most 32 terms in fp32, whose additions are off by u each: 32 u.
    fp64 after that, and one rounding: 45 u. A lost token of 60,000 would be 280 u."""
    plan, c = one_plan(n, edge=128, seed=1)
    w = weights(D, 5)
    x, g = rows((2, 1, D), dtype, 1), rows((2, 1, D), dtype, 2)
    up = [g[i:i + 1].cuda().expand(n, h, D) for i, h in enumerate((heads, keys))]
    xs = [x[i:i + 1].cuda().expand(n, h, D) for i, h in enumerate((heads, keys))]
    outs = plan.rotary_backward(*up, ssa.Rotary(dim=2), *xs, *(v.cuda() for v in w))
    torch.cuda.synchronize()
    for i, h in enumerate((heads, keys)):
        v = ref.f64(x[i, 0])
        norm = v / ((v * v).mean() + 1e-6) ** 0.5
        want = n * h * ref.f64(g[i, 0]) * norm
        off = abs(ref.f64(outs[2 + i]) / want - 1)[2:]
        print(f"{'qk'[i]}: off by {off.max() / ref.U:.1f} u")
        assert off.max() <= 46 * ref.U


@pytest.mark.parametrize("n,heads,keys,D,dtype", [(3, 65535, 7, 32, "f32"), (2, 5, 65535, 96, "f16"), (5, 3001, 2999, 128, "bf16")])
def test_more_heads_than_a_tile_has_rows(n, heads, keys, D, dtype):
    """Tiles of one token with thousands of rows a thread; the sums' chain of 32 is inside the tile. The weights' gradients at
    a bound that does not grow with the rows: 96 u and the chain's 32 u of the terms' magnitudes."""
    plan, c = one_plan(n, seed=n)
    q, k = rows((n, heads, D), dtype, 1).cuda(), rows((n, keys, D), dtype, 2).cuda()
    dq, dk = rows((n, heads, D), dtype, 3).cuda(), rows((n, keys, D), dtype, 4).cuda()
    check_forward(plan, c, q, k, {}, weights(D, 5))
    check_backward(plan, c, dq, dk, q, k, {}, weights(D, 5), depth=32)


@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_large_shell_at_the_short_chains_bound(layout):
    """Many tiles per CTA, its loads running on into the next tile, at the same bound."""
    n, h = 60000, 22
    plan, c = one_plan(n, edge=128, seed=1)
    q, k = rows((n, h, 32), "f16", 1).cuda(), rows((n, 2, 32), "f16", 2).cuda()
    dq, dk = rows((n, h, 32), "f16", 3).cuda(), rows((n, 2, 32), "f16", 4).cuda()
    check_backward(plan, c, dq, dk, q, k, dict(layout=layout, dim=18), weights(32, 5), depth=32)
