"""Cross attention and rotary positions at the edges of what a call may be: guarded outputs and workspaces, long
strides, kept calls, captured training, split keys with padding. Bounds as in cross_formula.py."""
import ctypes

import pytest
import torch

import sub_quadratic_two_b200 as sq
from cross_formula import assert_within, backward, bounds, forward, keep_of
from sub_quadratic_two_b200.cross import _desc
from test_cross_gpu import BF16, F32, check, problem

pytestmark = pytest.mark.gpu

GUARD = 512  # bytes before and behind


class Guarded:
    """A dense tensor with a pattern in front of it and behind it."""

    def __init__(self, shape, dtype):
        size = torch.empty((), dtype=dtype).element_size()
        for s in shape:
            size *= s
        self.bytes = torch.full((size + 2 * GUARD,), 0xA5, dtype=torch.uint8, device="cuda")
        self.size = size
        self.t = self.bytes[GUARD:GUARD + size].view(dtype).view(shape)

    def untouched(self):
        return bool((self.bytes[:GUARD] == 0xA5).all() and (self.bytes[GUARD + self.size:] == 0xA5).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,h,hk,n,m,d", [
    (1, 2, 2, 1, 1, 64), (2, 4, 2, 300, 300, 64), (1, 2, 1, 129, 2500, 128), (1, 3, 3, 1, 4099, 64), (2, 2, 2, 1000, 77, 128)])
def test_writes_stay_in_outputs_and_workspaces(cuda_ok, dtype, B, h, hk, n, m, d):
    q, k, v, do = problem(n + m, B, h, hk, n, m, d, dtype)
    code = sq.SQUAD_BF16 if dtype == BF16 else sq.SQUAD_F32
    strides = [t.stride() for t in (q, k, v, q, do, q, k, v)]
    desc = _desc(q.shape, k.shape, code, 0.0, 0, strides)
    lib, st = sq.load_library(), torch.cuda.current_stream().cuda_stream
    o, lse = Guarded(q.shape, dtype), Guarded(q.shape[:3], F32)
    ws = [Guarded((sq.cross_workspace_size(q, k, w),), torch.uint8) for w in (0, 1)]
    grads = [Guarded(t.shape, dtype) for t in (q, k, v)]
    at = lambda g: g.t.data_ptr() if g.size else None  # noqa: E731
    assert lib.squad_cross_fwd(ctypes.byref(desc), q.data_ptr(), k.data_ptr(), v.data_ptr(), None, None, at(o), at(lse),
                               at(ws[0]), ws[0].size, st) == 0
    assert lib.squad_cross_bwd(ctypes.byref(desc), q.data_ptr(), k.data_ptr(), v.data_ptr(), None, None, at(o), at(lse),
                               do.data_ptr(), *[at(g) for g in grads], at(ws[1]), ws[1].size, st) == 0
    torch.cuda.synchronize()
    sq.poll_device_error()
    assert all(g.untouched() for g in [o, lse, *ws, *grads])
    keep, s = keep_of(B, m), d ** -0.5
    bs = bounds(q, k, v, keep, s, do)
    assert_within(o.t, forward(q, k, v, keep, s)[0], bs[0], "o")
    for name, g, r, b in zip(("dq", "dk", "dv"), grads, backward(q, k, v, keep, s, do), bs[2:]):
        assert_within(g.t, r, b, name)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,m,d", [(1, 4097, 64), (130, 5000, 128), (17, 2049, 128)])
def test_split_keys_with_lengths_and_holes(cuda_ok, dtype, n, m, d):
    # parts of the keys that end before, at and behind a length, and parts in which no key is kept
    B = 3
    q, k, v, do = problem(n + m, B, 2, 1, n, m, d, dtype)
    for lens in ([m, 0, 1], [m - 1, 700, 128], [2048, 129, m + 9]):
        check(q, k, v, do, kv_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), backward_too=False)
    mask = torch.zeros(B, m, dtype=torch.bool, device="cuda")
    mask[0, m - 1] = True
    mask[1, 600:1500:3] = True
    check(q, k, v, do, key_mask=mask, backward_too=False)
    check(q, k, v, do, key_mask=mask, kv_lens=torch.tensor([m, 1000, m], dtype=torch.int32, device="cuda"),
          backward_too=False)


@pytest.mark.parametrize("B,h,hk,n,m,d", [
    (1, 1, 1, 16, 700, 32), (1, 2, 2, 300, 300, 64),       # tiles of 16 rows
    (1, 16, 4, 450, 200, 64), (2, 30, 30, 130, 90, 96),    # of 32
    (2, 40, 20, 260, 150, 160), (1, 24, 24, 1000, 77, 128),  # of 64
    (1, 24, 24, 1000, 90, 192)])                           # wide heads
@pytest.mark.parametrize("padded", [False, True])
def test_f32_tiles(cuda_ok, B, h, hk, n, m, d, padded):
    q, k, v, do = problem(m + d, B, h, hk, n, m, d, F32)
    mask = None
    if padded:
        mask = torch.rand(B, m, generator=torch.Generator(device="cuda").manual_seed(m), device="cuda") < 0.7
    check(q, k, v, do, key_mask=mask)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_states_broadcast_over_heads(cuda_ok, dtype):
    # one state for every key head, seen through expand (a head stride of 0)
    q, k, v, do = problem(40, 2, 4, 4, 140, 200, 64, dtype)
    k1, v1 = k[:, :1].expand(-1, 4, -1, -1), v[:, :1].expand(-1, 4, -1, -1)
    check(q, k1, v1, do)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_strides_past_32_bits(cuda_ok, dtype):
    # batch rows, head rows and mask rows more than 2^32 bytes apart in one allocation
    B, h, n, m, d = 2, 2, 70, 150, 64
    far = (1 << 31) + 4096  # elements of the batch stride
    q, k, v, do = problem(41, B, h, h, n, m, d, dtype)
    size = q.element_size()
    heap = torch.empty(far * size + (1 << 22), dtype=torch.uint8, device="cuda")
    at, views = 0, []
    for t in (q, k, v, do, q):
        x = heap[at:].view(dtype).as_strided(t.shape, (far, t.shape[2] * d, d, 1))
        x.copy_(t)
        views.append(x)
        at += t[0].numel() * size + 256 & ~255
    fq, fk, fv, fdo, fo = views
    mask = heap[at:at + 1].view(torch.bool).as_strided((B, m), (far, 1))
    mask.copy_(torch.rand(B, m, device="cuda") < 0.8)
    keep, s = keep_of(B, m, None, mask), d ** -0.5
    o, lse = sq.squad_cross_fwd(fq, fk, fv, key_mask=mask, out=fo)
    grads = sq.squad_cross_bwd(fq, fk, fv, o, lse, fdo, key_mask=mask)
    sq.poll_device_error()
    bs = bounds(q, k, v, keep, s, do)
    assert_within(o, forward(q, k, v, keep, s)[0], bs[0], "o")
    for name, g, r, b in zip(("dq", "dk", "dv"), grads, backward(q, k, v, keep, s, do), bs[2:]):
        assert_within(g, r, b, name)
    rot = sq.rotary_plan((2, 5, 7), d)
    (want,) = sq.squad_rotary([q], rot)
    sq.squad_rotary([fq], rot, out=[fo])
    assert torch.equal(fo, want)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_many_batch_rows(cuda_ok, dtype):
    B, h, n, m, d = 20011, 2, 1, 5, 64
    q, k, v, do = problem(42, B, h, 1, n, m, d, dtype)
    lens = torch.randint(0, m + 1, (B,), generator=torch.Generator().manual_seed(1)).int().cuda()
    check(q, k, v, do, kv_lens=lens)


def test_a_kept_call_still_checks_its_tensors(cuda_ok):
    q, k, v, do = problem(43, 2, 2, 2, 6, 9, 64)
    lens = torch.tensor([9, 9], dtype=torch.int32, device="cuda")
    mask = torch.ones(2, 9, dtype=torch.bool, device="cuda")
    for _ in range(2):
        o, lse = sq.squad_cross_fwd(q, k, v, kv_lens=lens, key_mask=mask)
        sq.squad_cross_bwd(q, k, v, o, lse, do, kv_lens=lens, key_mask=mask)
        flat = torch.randn(q.numel() + 8, device="cuda").to(BF16)
        off = flat[1:1 + q.numel()].view(q.shape)  # the same kind of tensor, 2 bytes off
        with pytest.raises(sq.SquadError):
            sq.squad_cross_fwd(off, k, v, kv_lens=lens, key_mask=mask)
        with pytest.raises(sq.SquadError):
            sq.squad_cross_bwd(q, k, v, o, lse, off, kv_lens=lens, key_mask=mask)
        with pytest.raises(ValueError):
            sq.squad_cross_fwd(q, k, v, kv_lens=lens.cpu(), key_mask=mask)
        with pytest.raises(ValueError):
            sq.squad_cross_fwd(q, k, v, kv_lens=lens, key_mask=mask.cpu())
        with pytest.raises(ValueError):
            sq.squad_cross_fwd(q.cpu(), k, v)
        with pytest.raises(ValueError):
            sq.squad_cross_fwd(None, k, v)
    rot = sq.rotary_plan((1, 2, 3), 64)
    for _ in range(2):
        sq.squad_rotary([q], rot)
        with pytest.raises(sq.SquadError):
            sq.squad_rotary([off], rot)


def test_scale_is_taken_by_value(cuda_ok):
    q, k, v, do = problem(44, 1, 2, 2, 40, 50, 64)
    scale = torch.tensor(0.1)
    for value in (0.1, 0.3):
        scale.fill_(value)
        o, lse = sq.squad_cross_fwd(q, k, v, scale)
        r, rl = sq.squad_cross_fwd(q, k, v, float(scale))
        assert torch.equal(o, r)
        for a, b in zip(sq.squad_cross_bwd(q, k, v, o, lse, do, scale), sq.squad_cross_bwd(q, k, v, o, lse, do, float(scale))):
            assert torch.equal(a, b)
    with pytest.raises(ValueError):
        sq.cross_attention(q, k, v, scale=-0.1)


def test_gradients_are_not_differentiable_again(cuda_ok):
    q, k, v, _ = problem(45, 1, 2, 2, 6, 9, 64, F32)
    for t in (q, k, v):
        t.requires_grad_()
    (g,) = torch.autograd.grad(sq.cross_attention(q, k, v).square().sum(), q, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()
    rot = sq.rotary_plan((1, 2, 3), 64)
    (g,) = torch.autograd.grad(sq.rotary(q, None, rot)[0].square().sum(), q, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()


def test_rotary_of_a_tensor_without_heads(cuda_ok):
    rot = sq.rotary_plan((1, 2, 3), 64)
    x = torch.randn(2, 3, 6, 64, device="cuda")
    none = x[:, :0]
    (want,) = sq.squad_rotary([x], rot)
    for pair in ([x, none], [none, x]):
        for a, b in zip(sq.squad_rotary(pair, rot), pair):
            assert a.shape == b.shape and (a.numel() == 0 or torch.equal(a, want))
    assert sq.squad_rotary([none], rot)[0].shape == none.shape


def test_a_table_changed_before_the_backward_is_refused(cuda_ok):
    rot = sq.rotary_plan((1, 2, 3), 64)
    x = torch.randn(1, 2, 6, 64, device="cuda", requires_grad=True)
    y, _ = sq.rotary(x, None, rot)
    rot.table.mul_(1.0)
    with pytest.raises(RuntimeError):
        y.sum().backward()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_captured_training_step(cuda_ok, dtype):
    """Rotary positions and cross attention, forward and gradients, captured by autograd and replayed on new
    inputs, with leaves of its own while an eager graph of the same memory lives."""
    grid, B, h, m, d = (2, 9, 10), 2, 2, 130, 64
    n = 180
    rot = sq.rotary_plan(grid, d)
    q, k, v, do = problem(46, B, h, h, n, m, d, dtype, "tokens")
    held = [t.detach().clone(memory_format=torch.preserve_format).requires_grad_() for t in (q, k, v)]
    lens = torch.tensor([m, 31], dtype=torch.int32, device="cuda")

    def step():
        leaves = [t.detach().requires_grad_() for t in held]
        o = sq.cross_attention(sq.rotary(leaves[0], None, rot)[0], leaves[1], leaves[2], kv_lens=lens)
        return o, torch.autograd.grad(o, leaves, do)

    alive = sq.cross_attention(*held, kv_lens=lens)  # an eager graph
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, grads = step()
    for rep in range(3):
        with torch.no_grad():
            for t in held:
                t.mul_(0.9)
            lens[1] = 20 + 37 * rep
        graph.replay()
        torch.cuda.synchronize()
        eo, eg = step()
        assert torch.equal(o, eo)
        assert all(torch.equal(a, b) for a, b in zip(grads, eg))
    assert alive.shape == q.shape
    sq.poll_device_error()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,m", [(300, 200), (1, 3000)])
def test_queries_without_states_may_hold_anything(cuda_ok, d, n, m):
    q, k, v, _ = problem(47, 3, 2, 2, n, m, d)
    q[1] = float("nan")
    q[2] = float("inf")
    mask = torch.ones(3, m, dtype=torch.bool, device="cuda")
    mask[1:] = False
    lens = torch.tensor([m, 0, 0], dtype=torch.int32, device="cuda")
    keep, s = keep_of(3, m, None, mask), d ** -0.5
    bound = bounds(q[:1], k[:1], v[:1], keep[:1], s)[0]
    for kw in (dict(key_mask=mask), dict(kv_lens=lens), dict(key_mask=mask, kv_lens=lens)):
        o, lse = sq.squad_cross_fwd(q, k, v, **kw)
        assert (o[1:] == 0).all() and (lse[1:] == -float("inf")).all()
        assert_within(o[:1], forward(q[:1], k[:1], v[:1], keep[:1], s)[0], bound, "o")


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_outputs_of_any_order_of_axes(cuda_ok, dtype):
    # an output whose tokens are the slowest axis and batch rows the fastest is written; one whose rows overlap is not
    q, k, v, _ = problem(48, 2, 4, 2, 10, 20, 64, dtype)
    want, _ = sq.squad_cross_fwd(q, k, v)
    out = torch.empty(10, 4, 2, 64, device="cuda", dtype=dtype).permute(2, 1, 0, 3)
    assert torch.equal(sq.squad_cross_fwd(q, k, v, out=out)[0], want)
    with pytest.raises(sq.SquadError):
        sq.squad_cross_fwd(q, k, v, out=torch.empty(2048 * 4, device="cuda", dtype=dtype).as_strided(q.shape, (1024, 64, 64, 1)))


@pytest.mark.parametrize("B,h,n,m,d", [(6, 16, 1300, 600, 64), (6, 16, 1300, 600, 128), (7, 2, 90, 6000, 128), (7, 2, 90, 6000, 64)])
def test_lengths_of_every_kind_in_turn(cuda_ok, B, h, n, m, d):
    # many items to an SM whose lengths end inside blocks, at their ends and before the first, and parts of the
    # keys that lie behind a length
    q, k, v, do = problem(49, B, h, h, n, m, d)
    for i in range(3):
        gen = torch.Generator().manual_seed(50 + i)
        lens = torch.randint(0, m + 1, (B,), generator=gen)
        lens[i], lens[i + 1], lens[i + 2] = 0, 128 * (m // 256), 1
        check(q, k, v, do, kv_lens=lens.int().cuda(), backward_too=i == 0)
