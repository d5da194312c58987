"""The weights' gradients of the rotary gradient over many rows: the sums keep their precision however many rows a
thread adds up."""
import pytest
import torch

import operator_refs as ref
from test_gpu_rotary import one_plan, rows, weights

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
