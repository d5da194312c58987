"""Group normalisation of data whose first channel, or first row, is far from the others: the variance comes from
deviations whatever the order of channels and rows."""
import numpy as np
import pytest
import torch

import operator_refs as ref
from test_gpu_norm import check_forward, features, plan_of, weights

pytestmark = pytest.mark.gpu

# Relative error of rstd, in units u = 2^-24. A thread's rows (at most 48, about the first of them, which lies up to 4
# standard deviations of its channel off): 51 u times 17, of the share that the variance inside the channels has in the
# whole, at most 1 / 30 here: 29 u. The row lanes of a CTA and the channels of a group, about their means: chains of at most 512 / 32 + 5 additions
# of non-negative terms and 3 u for a term each, 24 u. The means themselves are off by some u of the offset, which enters squared, and
# their rounding to fp32 by less. Tiles and column blocks are added in fp64. 77 u and a rounding of the variance, half of that
# and a rounding in its root.
RSTD = 64 * ref.U


def check_rstd(plan, cu, x, groups):
    y, mean, rstd = check_forward(plan, cu, x, groups, weights(x.shape[1], 3), act="silu")
    _, var, _, _ = ref.norm_stats(ref.f64(x), cu, groups)
    full = np.diff(cu) > 0
    want = 1 / np.sqrt(var[full] + 1e-5)
    off = np.abs(ref.f64(rstd)[full] / want - 1)
    print(f"rstd off by {off.max() / ref.U:.1f} u")
    assert off.max() <= RSTD


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
