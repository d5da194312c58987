"""fp32 outputs of the operators that meet one another, or what the same launch still reads, are refused."""
import ctypes

import pytest
import torch

import spatial_sparse_attention_b200 as ssa
from test_gpu_norm import plan_of

pytestmark = pytest.mark.gpu


def test_group_norm_refuses_outputs_over_weights_and_statistics():
    plan, _ = plan_of((3, 1))           # statistics [2, 2], weights [16]
    x = torch.zeros(4, 16, device="cuda")
    w = torch.ones(256, device="cuda")
    a, p = ctypes.addressof, w.data_ptr()
    rows = ssa._Rows(x.data_ptr(), 16)
    v = a(rows)
    gamma, beta, mean, rstd, dgamma, dbeta = (p + 4 * 32 * i for i in range(6))

    def fwd(mean, rstd):
        return ssa.lib.ssa_group_norm(plan._h, v, 16, 2, gamma, beta, 1e-5, 0, 0, v, mean, rstd, None)

    def bwd(dgamma, dbeta):
        return ssa.lib.ssa_group_norm_backward(plan._h, v, v, mean, rstd, 16, 2, gamma, beta, 0, 0, v, dgamma, dbeta, None)

    before = ssa.launch_count()
    for m, r in ((gamma, rstd), (mean, beta), (gamma + 60, rstd), (mean, mean), (mean, mean + 12), (beta - 12, rstd)):
        assert fwd(m, r) == 1
    for g, b in ((gamma, dbeta), (dgamma, beta), (beta, gamma), (mean, dbeta), (dgamma, rstd), (dgamma, dgamma), (dgamma, dgamma + 60),
                 (mean - 60, dbeta), (dgamma, rstd + 12)):
        assert bwd(g, b) == 1
    assert ssa.launch_count() == before
    # neighbours are taken
    assert fwd(mean, mean + 16) == 0
    assert fwd(gamma + 64, gamma + 80) == 0
    assert bwd(dgamma, dgamma + 64) == 0
    torch.cuda.synchronize()


def test_rotary_gradient_refuses_weights_gradients_in_one_place():
    c = torch.tensor([[0, 0, 0], [1, 2, 3]], dtype=torch.int32, device="cuda")
    plan = ssa.Plan(c, grid=(8, 8, 8), r=0)
    q, k = torch.ones(2, 2, 32, device="cuda"), torch.ones(2, 2, 32, device="cuda")
    w = torch.ones(96, device="cuda")
    r, a, p = ssa.Rotary(), ctypes.addressof, w.data_ptr()
    vq, vk = ssa._Heads(q.data_ptr(), 64, 32, 2), ssa._Heads(k.data_ptr(), 64, 32, 2)

    def bwd(dq_gamma, dk_gamma):
        return ssa.lib.ssa_rotary_backward(plan._h, a(vq), a(vk), a(vq), a(vk), p, p, 1e-6, a(r), 32, 0, a(vq), a(vk), dq_gamma,
                                           dk_gamma, None)

    before = ssa.launch_count()
    assert bwd(p + 128, p + 128) == 1
    assert bwd(p + 128, p + 252) == 1
    assert ssa.launch_count() == before
    assert bwd(p + 128, p + 256) == 0
    torch.cuda.synchronize()
