"""Cross attention and rotary positions on rows that lie far apart: batch, head and token strides past 2^31 elements,
mask rows past 2^32 bytes, outputs and gradients among them. Bounds as in cross_formula.py."""
import ctypes

import pytest
import torch

import sub_quadratic_two_b200 as sq
from cross_formula import assert_within, backward, bounds, forward, keep_of
from sub_quadratic_two_b200.cross import _desc
from test_cross_gpu import BF16, F32, problem

pytestmark = pytest.mark.gpu

FAR = (1 << 31) + 4096  # elements


def heap_of(shapes, axis, dtype):
    """Views of the shapes in one allocation, filled with 3: rows of an axis (0 batch, 1 head, 2 token) lie FAR apart,
    the others densely in between."""
    size = torch.empty((), dtype=dtype).element_size()
    most = max(s[axis] for s in shapes)
    heap = torch.empty((FAR * (most - 1) + (1 << 20)) * size, dtype=torch.uint8, device="cuda").view(dtype)
    at, views = 0, []
    for s in shapes:
        strides, dense = [0, 0, 0, 1], s[3]
        for i in (2, 1, 0):
            strides[i] = FAR if i == axis else dense
            dense *= 1 if i == axis else s[i]
        views.append(heap[at:].as_strided(s, strides).fill_(3.0))
        at += dense + 127 & ~127
    assert at <= 1 << 20
    return views


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("axis,B,h,hk,n,m", [(0, 2, 2, 1, 70, 150), (1, 1, 2, 2, 130, 140), (1, 2, 4, 2, 3, 1100), (2, 1, 2, 1, 2, 3),
                                             (2, 2, 1, 1, 3, 2)])
def test_cross_attention(cuda_ok, dtype, axis, B, h, hk, n, m):
    d = 64
    code = sq.SQUAD_BF16 if dtype == BF16 else sq.SQUAD_F32
    near = problem(80 + axis, B, h, hk, n, m, d, dtype)
    q, k, v, do, o, dq, dk, dv = far = heap_of([t.shape for t in near] + [near[0].shape, near[0].shape, near[1].shape, near[1].shape],
                                               axis, dtype)
    for x, t in zip(far, near):
        x.copy_(t)
    step = (1 << 32) + 4096  # bytes
    mask = torch.empty(step * (B - 1) + 2048, dtype=torch.uint8, device="cuda").view(torch.bool).as_strided((B, m), (step, 1))
    mask.copy_(torch.rand(B, m, generator=torch.Generator().manual_seed(m)).cuda() < 0.8)
    mask[:, 0] = True
    keep, s = keep_of(B, m, None, mask), d ** -0.5
    desc = _desc(q.shape, k.shape, code, 0.0, step, [t.stride() for t in (q, k, v, o, do, dq, dk, dv)])
    lse = torch.empty(B, h, n, device="cuda")
    ws = [torch.empty(max(1, sq.cross_workspace_size(q, k, w)), dtype=torch.uint8, device="cuda") for w in (0, 1)]
    lib, st = sq.load_library(), torch.cuda.current_stream().cuda_stream
    assert lib.squad_cross_fwd(ctypes.byref(desc), q.data_ptr(), k.data_ptr(), v.data_ptr(), None, mask.data_ptr(),
                               o.data_ptr(), lse.data_ptr(), ws[0].data_ptr(), ws[0].numel(), st) == 0
    assert lib.squad_cross_bwd(ctypes.byref(desc), q.data_ptr(), k.data_ptr(), v.data_ptr(), None, mask.data_ptr(),
                               o.data_ptr(), lse.data_ptr(), do.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                               ws[1].data_ptr(), ws[1].numel(), st) == 0
    sq.poll_device_error()
    bs = bounds(*near[:3], keep, s, near[3])
    assert_within(o, forward(*near[:3], keep, s)[0], bs[0], "o")
    for name, g, r, b in zip(("dq", "dk", "dv"), (dq, dk, dv), backward(*near[:3], keep, s, near[3]), bs[2:]):
        assert_within(g, r, b, name)
    for x, t in zip(far, near):
        assert torch.equal(x, t)  # inputs stay


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("pairing", ["adjacent", "half"])
@pytest.mark.parametrize("axis,B,h,grid", [(0, 2, 3, (2, 5, 7)), (1, 1, 2, (2, 5, 7)), (2, 2, 2, (1, 1, 3))])
def test_rotary(cuda_ok, dtype, pairing, axis, B, h, grid):
    n, d = grid[0] * grid[1] * grid[2], 64
    near = torch.randn(B, h, n, d, generator=torch.Generator(device="cuda").manual_seed(90), device="cuda").to(dtype)
    x, y = heap_of([near.shape] * 2, axis, dtype)
    x.copy_(near)
    rot = sq.rotary_plan(grid, d, (16, 24, 24), pairing=pairing)
    for inverse in (False, True):
        sq.squad_rotary([x], rot, inverse=inverse, out=[y])
        assert torch.equal(y, sq.squad_rotary([near], rot, inverse=inverse)[0])
    assert torch.equal(x, near)
