"""The forward of group normalisation in two launches, which inputs beyond the SMs' shared memory take, at every chunk that
rows are read in, with more rows per thread than are in flight at once."""
import numpy as np
import pytest
import torch

import operator_refs as ref
from test_gpu_norm import check_backward, features, dev, f64s, plan_of, weights

pytestmark = pytest.mark.gpu

import spatial_sparse_attention_b200 as ssa  # noqa: E402

SEQS = (9000, 0, 1, 14500)


@pytest.mark.parametrize("C,groups,dtype,chunk", [
    (2112, 32, "bf16", 16), (1044, 9, "f16", 8), (1044, 4, "bf16", 8), (1658, 2, "f16", 4), (1658, 1, "bf16", 4), (2045, 5, "f16", 2),
    (2112, 32, "f32", 16), (1658, 2, "f32", 8), (2045, 5, "f32", 4)])
def test_long_sequences_at_every_chunk(C, groups, dtype, chunk):
    plan, cu = plan_of(SEQS)
    n, es = cu[-1], 4 if dtype == "f32" else 2
    assert C * es % chunk == 0 and (chunk == 16 or C * es % (2 * chunk))
    x, w = features(n, C, dtype, C).cuda(), weights(C, 3)
    buf = torch.full((n + 1, C), 7.0, dtype=x.dtype, device="cuda")
    at = int(chunk < 16)        # the row before or behind the outputs is left as it was
    before = ssa.launch_count()
    y, mean, rstd = plan.group_norm(x, groups, *dev(w), activation="silu", return_stats=True, out=buf[at:n + at])
    assert ssa.launch_count() - before == 2
    want = ref.group_norm(ref.f64(x), cu, groups, *f64s(w), 1e-5, "silu")
    for name, a, b, t in zip(("y", "mean", "rstd"), (y, mean, rstd), want, (dtype, "f32", "f32")):
        ref.check(a, *b, t, name)
    assert (buf[0 if at else n] == 7).all()
    inplace = x.clone()
    plan.group_norm(inplace, groups, *dev(w), activation="silu", out=inplace)
    assert torch.equal(inplace, y)


@pytest.mark.parametrize("C,groups,dtype", [(1044, 9, "f16"), (1658, 2, "bf16"), (1658, 2, "f32"), (2045, 5, "f32"), (1045, 5, "f16")])
def test_gradient_at_narrow_chunks(C, groups, dtype):
    plan, cu = plan_of(SEQS)
    x, dy = features(cu[-1], C, dtype, 1).cuda(), features(cu[-1], C, dtype, 2).cuda()
    check_backward(plan, cu, dy, x, groups, weights(C, 3), act="silu")


def test_rows_of_a_wider_view():
    """Aligned channels in rows that are not: 16-bit rows at steps of 2, 4 and 8 bytes."""
    plan, cu = plan_of(SEQS)
    for pad in (1, 2, 4):
        wide = features(cu[-1], 1056 + pad, "f16", pad).cuda()
        x, w = wide[:, pad:], weights(1056, 3)
        before = ssa.launch_count()
        y, mean, rstd = plan.group_norm(x, 8, *dev(w), activation="gelu", return_stats=True)
        assert ssa.launch_count() - before == 2
        want = ref.group_norm(ref.f64(x), cu, 8, *f64s(w), 1e-5, "gelu")
        for a, b, t in zip((y, mean, rstd), want, ("f16", "f32", "f32")):
            ref.check(a, *b, t, f"pad {pad}")
    assert np.diff(cu)[1] == 0 and (mean[1] == 0).all() and (rstd[1] == 0).all()
