"""The factor on the rotated channels that yarn scaling brings along."""
import math

import pytest

import spatial_sparse_attention_b200 as ssa


@pytest.mark.parametrize("scale", [1.0, 0.999, 0.5, 1e-3, 1e-6])
def test_a_grid_no_larger_than_the_trained_one_keeps_the_factor_at_one(scale):
    """0.1 ln(scale) + 1 is for grids larger than the trained one; below scale 1 it would shrink the channels, and below
    e^-10 turn negative, which the library refuses."""
    r = ssa.Rotary(scaling="yarn", scale=scale, extent=64.0)
    assert r.mscale == 1.0
    r.frequencies(96)


@pytest.mark.parametrize("scale", [1.5, 2.0, 16.0])
def test_a_larger_grid_grows_it(scale):
    assert ssa.Rotary(scaling="yarn", scale=scale, extent=64.0).mscale == pytest.approx(0.1 * math.log(scale) + 1, rel=1e-7)


def test_a_given_factor_stays():
    assert ssa.Rotary(scaling="yarn", scale=0.5, extent=64.0, mscale=0.75).mscale == 0.75
    for scaling in (None, "linear", "ntk"):
        assert ssa.Rotary(scaling=scaling, scale=4.0).mscale == 1.0
