"""A call of an operator that the runtime refuses returns its error and leaves none behind for the next call."""
import ctypes

import pytest
import torch

import spatial_sparse_attention_b200 as ssa

pytestmark = pytest.mark.gpu

ALLOC = ctypes.CFUNCTYPE(ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_void_p)
FREE = ctypes.CFUNCTYPE(None, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p)


@pytest.fixture
def plan_without_runtime_allocations():
    """A plan whose memory comes from one buffer, so that a call reaches its launches on a stream where the runtime would
    not allocate."""
    buf = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    used = [0]

    def take(n, stream, ctx):
        at = used[0]
        used[0] += (n + 255) // 256 * 256
        return buf.data_ptr() + at if used[0] <= buf.numel() else None

    alloc, free = ALLOC(take), FREE(lambda p, stream, ctx: None)
    c = torch.stack((torch.arange(64), torch.zeros(64, dtype=torch.int64), torch.arange(64) % 7), 1).int().cuda()
    assert ssa.lib.ssa_set_allocator(alloc, free, None) == 0
    try:
        plan = ssa.Plan(c, grid=(64, 8, 8), r=0)
    finally:
        assert ssa.lib.ssa_set_allocator(None, None, None) == 0
    yield plan
    torch.cuda.synchronize()
    plan.close()
    del buf, alloc, free


def test_a_refused_launch_leaves_no_error_behind(plan_without_runtime_allocations):
    plan = plan_without_runtime_allocations
    x = torch.randn(64, 3, device="cuda").half()        # rows of 2-byte chunks: two launches
    y, up = torch.empty_like(x), torch.randn(64, 3, device="cuda").half()
    q = torch.randn(64, 2, 32, device="cuda").half()
    w, dw = torch.ones(32, device="cuda"), torch.empty(32, device="cuda")
    _, mean, rstd = plan.group_norm(x, 1, return_stats=True)
    dxs = [torch.empty(3, device="cuda") for _ in range(2)]
    want = plan.rotary(q)
    torch.cuda.synchronize()
    a = ctypes.addressof
    rows, up_rows, out_rows = ssa._Rows(x.data_ptr(), 3), ssa._Rows(up.data_ptr(), 3), ssa._Rows(y.data_ptr(), 3)
    heads, rot = ssa._Heads(q.data_ptr(), 64, 32, 2), ssa.Rotary()
    dq = torch.empty_like(q)
    out = ssa._Heads(dq.data_ptr(), 64, 32, 2)
    calls = {
        "group_norm": lambda s: ssa.lib.ssa_group_norm(plan._h, a(rows), 3, 1, None, None, 1e-5, 0, 2, a(out_rows), None, None, s),
        "group_norm_backward": lambda s: ssa.lib.ssa_group_norm_backward(
            plan._h, a(up_rows), a(rows), mean.data_ptr(), rstd.data_ptr(), 3, 1, None, None, 0, 2, a(out_rows), dxs[0].data_ptr(),
            dxs[1].data_ptr(), s),
        "rotary": lambda s: ssa.lib.ssa_rotary(plan._h, a(heads), None, None, None, 1e-6, a(rot), 32, 2, a(out), None, s),
        "rotary_backward": lambda s: ssa.lib.ssa_rotary_backward(
            plan._h, a(heads), None, a(heads), None, w.data_ptr(), None, 1e-6, a(rot), 32, 2, a(out), None, dw.data_ptr(), None, s),
    }
    rt = ctypes.CDLL("libcudart.so.12")
    stream = torch.cuda.Stream().cuda_stream
    handle = ctypes.c_void_p(stream)
    for name, call in calls.items():
        # waiting for a stream that is being captured is an error of the runtime, after which nothing can be queued on it
        # until the capture ends
        assert rt.cudaStreamBeginCapture(handle, 1) == 0
        graph = ctypes.c_void_p()
        try:
            assert rt.cudaStreamSynchronize(handle) != 0
            assert call(stream) == 5, name          # SSA_ERR_CUDA
        finally:
            assert rt.cudaStreamEndCapture(handle, ctypes.byref(graph)) != 0
            rt.cudaGetLastError()
        assert torch.equal(plan.rotary(q), want), name
        assert call(None) == 0, name
    torch.cuda.synchronize()
