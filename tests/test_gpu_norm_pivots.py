"""Group normalisation of data whose first channel, or first row, is far from the others: the variance comes from
deviations whatever the order of channels and rows."""
import numpy as np
import pytest
import torch

import operator_refs as ref
from test_gpu_norm import check_forward, features, plan_of, weights

pytestmark = pytest.mark.gpu

import spatial_sparse_attention_b200 as ssa  # noqa: E402

# Relative error of rstd, in units u = 2^-24. A thread's rows (at most 48, about the first of them, which lies up to 4
# standard deviations of its channel off): 51 u times 17, of the share that the variance inside the channels has in the
# whole, at most 1 / 30 here: 29 u. The row lanes of a CTA and the channels of a group, about their means: chains of at most 512 / 32 + 5 additions
# of non-negative terms and 3 u for a term each, 24 u. The means themselves are off by some u of the offset, which enters squared, and
# their rounding to fp32 by less. Tiles and column blocks are added in fp64. 77 u and a rounding of the variance, half of that
# and a rounding in its root.
RSTD = 64 * ref.U


def check_rstd(plan, cu, x, groups, limit=RSTD):
    y, mean, rstd = check_forward(plan, cu, x, groups, weights(x.shape[1], 3), act="silu")
    _, var, _, _ = ref.norm_stats(ref.f64(x), cu, groups)
    full = np.diff(cu) > 0
    want = 1 / np.sqrt(var[full] + 1e-5)
    off = np.abs(ref.f64(rstd)[full] / want - 1)
    print(f"rstd off by {off.max() / ref.U:.1f} u")
    assert off.max() <= limit


@pytest.mark.parametrize("offset", [100.0, 1000.0])
@pytest.mark.parametrize("seqs,C,groups,dtype", [
    ((1500,), 339, 1, "f32"), ((1500,), 339, 1, "f16"), ((1700, 0, 300), 2045, 5, "f32"), ((1700, 0, 300), 2045, 5, "bf16"),
    ((9000, 14500), 128, 1, "f32"), ((9000, 14500), 512, 1, "bf16"), ((9000, 14500), 1658, 2, "f32")])
def test_first_channel_of_a_group_far_from_the_others(seqs, C, groups, dtype, offset):
    plan, cu = plan_of(seqs)
    x = features(cu[-1], C, "f32", 1)
    x[:, ::C // groups] += offset
    check_rstd(plan, cu, x.to(ref.DTYPES[dtype]).cuda(), groups)


@pytest.mark.parametrize("C,groups,dtype", [(4, 1, "f32"), (8, 2, "f16"), (3, 1, "f32")])
def test_first_row_far_from_the_others(C, groups, dtype):
    """Narrow rows: a CTA has up to 256 row lanes, here with one row each, and the first lane's is the outlier."""
    plan, cu = plan_of((5000,))
    x = features(cu[-1], C, "f32", 2)
    x[0] += 1000.0
    check_rstd(plan, cu, x.to(ref.DTYPES[dtype]).cuda(), groups)


@pytest.mark.parametrize("n,C,groups,dtype", [(60000, 256, 256, "f32"), (200000, 64, 64, "f32"), (60000, 211, 211, "f16"), (60000, 330, 165, "f32")])
def test_first_row_far_from_its_threads_others(n, C, groups, dtype):
    """Long sequences, up to 48 rows to a thread, of which the first is the outlier and makes up most of the variance: 1000 squared
    over the rows against 1. About it, the thread's squares would cancel by their number. After eight rows the deviations are
    from their mean, which is an eighth of the offset off the others: (8 + 3) u times 8 for the first, (40 + 3) u times 40 / 64 for
    the others, 24 u for the merges: 139 u of the variance, half of that and 2 u of rstd."""
    plan, cu = plan_of((n,))
    x = features(n, C, "f32", 2)
    x[0] += 1000.0
    before = ssa.launch_count()
    check_rstd(plan, cu, x.to(ref.DTYPES[dtype]).cuda(), groups, 72 * ref.U)
    assert ssa.launch_count() - before == 2
