"""Cross attention on the GPU against its definition in 64 bits (cross_formula.py, which derives the bounds)."""
import math

import pytest
import torch

import sub_quadratic_two_b200 as sq
from cross_formula import assert_within, backward, bounds, forward, keep_of

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def rows(gen, B, h, n, d, dtype, layout, mul=1.0):
    shape = (B, n, h, d) if layout == "tokens" else (B, h, n, d)
    x = (torch.randn(shape, generator=gen, device="cuda") * mul).to(dtype)
    return x.transpose(1, 2) if layout == "tokens" else x


def problem(seed, B, h, hk, n, m, d, dtype=BF16, layout="heads", mul=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    q, k, v, do = (rows(gen, B, heads, r, d, dtype, layout, s) for heads, r, s in
                   ((h, n, mul), (hk, m, 1.0), (hk, m, 1.0), (h, n, 1.0)))
    return q, k, v, do


def check(q, k, v, do, scale=None, kv_lens=None, key_mask=None, backward_too=True):
    keep = keep_of(k.shape[0], k.shape[2], kv_lens, key_mask)
    s = scale or q.shape[-1] ** -0.5
    o, lse = sq.squad_cross_fwd(q, k, v, scale, kv_lens, key_mask)
    ro, rl, _ = forward(q, k, v, keep, s)
    clean = [torch.where(keep[:, None, :, None], t, torch.zeros((), dtype=t.dtype, device="cuda")) for t in (k, v)]
    bs = bounds(q, *clean, keep, s, do if backward_too else None)
    sq.poll_device_error()
    assert_within(o, ro, bs[0], "o")
    empty = rl == -math.inf
    assert torch.equal(lse == -math.inf, empty)
    assert_within(torch.where(empty, 0.0, lse.double()), torch.where(empty, 0.0, rl), bs[1], "lse")
    if backward_too:
        got = sq.squad_cross_bwd(q, k, v, o, lse, do, scale, kv_lens, key_mask)
        sq.poll_device_error()
        for name, g, r, b in zip(("dq", "dk", "dv"), got, backward(q, *clean, keep, s, do), bs[2:]):
            assert_within(g, r, b, name)
    return o, lse


SHAPES = [  # B, h, hk, n, m, d
    (1, 1, 1, 1, 1, 64), (1, 1, 1, 1, 1, 128), (1, 2, 2, 1, 2, 128), (2, 2, 1, 2, 1, 64), (1, 3, 3, 5, 17, 128),
    (1, 2, 2, 127, 31, 64), (1, 2, 2, 128, 64, 128), (1, 2, 2, 129, 77, 128), (2, 4, 2, 130, 127, 64),
    (1, 2, 2, 255, 128, 128), (1, 2, 1, 256, 129, 128), (2, 2, 2, 257, 255, 64), (1, 2, 2, 300, 256, 128),
    (1, 1, 1, 511, 257, 128), (1, 4, 1, 640, 512, 64), (1, 2, 2, 1000, 226, 128), (3, 6, 2, 333, 385, 64),
    (1, 2, 2, 64, 1111, 128), (1, 8, 8, 2048, 77, 128), (2, 3, 1, 1, 5000, 128), (1, 4, 2, 7, 4097, 64),
]


@pytest.mark.parametrize("layout", ["heads", "tokens"])
@pytest.mark.parametrize("B,h,hk,n,m,d", SHAPES)
def test_bf16_shapes(cuda_ok, B, h, hk, n, m, d, layout):
    check(*problem(n * 31 + m, B, h, hk, n, m, d, BF16, layout))


@pytest.mark.parametrize("B,h,hk,n,m,d", [
    (1, 24, 24, 1, 6000, 128), (1, 3, 3, 1, 27280, 128), (2, 5, 5, 3, 9000, 64), (1, 2, 1, 129, 8200, 128),
    (1, 37, 37, 128, 5000, 64)])
def test_few_queries_over_long_states(cuda_ok, B, h, hk, n, m, d):
    # the keys of a query tile are split over jobs of many blocks each
    q, k, v, do = problem(m + h, B, h, hk, n, m, d)
    for _ in range(3):
        check(q, k, v, do, backward_too=False)


@pytest.mark.parametrize("dtype,h,n,m,d", [(BF16, 40, 1100, 520, 64), (BF16, 100, 300, 300, 128), (BF16, 330, 100, 130, 64)])
@pytest.mark.parametrize("padded", [False, True])
def test_many_items_with_odd_tiles(cuda_ok, dtype, h, n, m, d, padded):
    # query tiles taken in pairs, the last of a head alone, several items per SM
    q, k, v, do = problem(h, 2, h, h, n, m, d)
    lens = torch.tensor([m, m // 3], dtype=torch.int32, device="cuda") if padded else None
    check(q, k, v, do, kv_lens=lens)


@pytest.mark.parametrize("B,h,hk,n,m,d", [
    (1, 1, 1, 1, 1, 32), (1, 2, 2, 3, 2, 64), (2, 2, 1, 63, 65, 96), (1, 2, 2, 64, 64, 128), (1, 2, 2, 65, 63, 160),
    (1, 4, 2, 130, 77, 192), (1, 1, 1, 33, 300, 224), (2, 2, 2, 100, 130, 256), (1, 3, 3, 257, 129, 32),
    (1, 2, 2, 1, 2000, 64), (1, 2, 1, 700, 1, 128),
])
@pytest.mark.parametrize("layout", ["heads", "tokens"])
def test_f32_shapes(cuda_ok, B, h, hk, n, m, d, layout):
    check(*problem(n * 37 + m, B, h, hk, n, m, d, F32, layout))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,m", [(150, 300), (1, 700), (260, 128), (40, 5)])
def test_lengths_with_anything_behind_them(cuda_ok, dtype, d, n, m):
    B = 7
    lens = torch.tensor([m, 0, 1, m - 1, min(m, 128), m + 50, -3], dtype=torch.int32, device="cuda")
    q, k, v, do = problem(m, B, 4, 2, n, m, d, dtype)
    keep = keep_of(B, m, lens)
    for t, bad in ((k, math.nan), (v, math.inf)):  # what lies behind a length must not matter
        t.copy_(torch.where(keep[:, None, :, None], t, torch.full((), bad, dtype=dtype, device="cuda")))
    check(q, k, v, do, kv_lens=lens)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,m", [(150, 300), (1, 900), (300, 130), (129, 33)])
def test_masks_with_holes(cuda_ok, dtype, n, m):
    B, d = 5, 64
    gen = torch.Generator(device="cuda").manual_seed(m)
    mask = torch.rand(B, m, generator=gen, device="cuda") < 0.6
    mask[1] = False                 # nothing left
    mask[2, : min(m, 140)] = False  # the whole first block and a part of the next
    mask[3] = False
    mask[3, m - 1] = True           # one key, the last
    q, k, v, do = problem(m + 1, B, 4, 4, n, m, d, dtype)
    for t, bad in ((k, -math.inf), (v, math.nan)):
        t.copy_(torch.where(mask[:, None, :, None], t, torch.full((), bad, dtype=dtype, device="cuda")))
    o, _ = check(q, k, v, do, key_mask=mask)
    assert (o[1] == 0).all()
    assert torch.equal(o[3], v[3][:, m - 1:].expand_as(o[3]))  # one key left: its value
    check(q, torch.nan_to_num(k, 0, 0, 0), torch.nan_to_num(v, 0, 0, 0), do, key_mask=mask[:1])  # one row for all
    lens = torch.tensor([m, m, m // 2, m, 3], dtype=torch.int32, device="cuda")
    check(q, k, v, do, kv_lens=lens, key_mask=mask)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_scale_and_peaked_rows(cuda_ok, dtype):
    q, k, v, do = problem(5, 1, 2, 2, 200, 300, 64, dtype, mul=12.0)
    check(q, k, v, do)
    check(*problem(6, 1, 2, 2, 200, 300, 64, dtype), scale=0.4)


def test_scores_that_grow_along_the_keys(cuda_ok):
    # the running maximum moves by far at every block, up and down
    q, k, v, do = problem(8, 1, 2, 2, 140, 640, 128)
    ramp = torch.cat([torch.linspace(0.1, 6, 320), torch.linspace(6, 0.1, 320)]).cuda()
    q.abs_()
    k.copy_((k.abs().float() * ramp[None, None, :, None]).to(k.dtype))
    check(q, k, v, do, backward_too=True)


def test_minus_infinite_scores_in_kept_places(cuda_ok):
    # a kept state whose scores are -inf has weight 0; a query that sees only such states has no defined
    # softmax and comes out as an empty row (zeros)
    q, k, v, _ = problem(9, 1, 1, 1, 3, 200, 64)
    q.fill_(1.0)
    k[:, :, 1:, :] = -math.inf
    o, lse = sq.squad_cross_fwd(q, k, v)
    assert torch.equal(o, v[:, :, :1].expand_as(o))
    k.fill_(-math.inf)
    o, lse = sq.squad_cross_fwd(q, k, v)
    assert (o == 0).all() and (lse == -math.inf).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_zero_lengths(cuda_ok, dtype):
    q = torch.randn(2, 2, 5, 64, device="cuda").to(dtype).requires_grad_()
    k, v = (torch.randn(2, 2, 0, 64, device="cuda").to(dtype).requires_grad_() for _ in "kv")
    o = sq.cross_attention(q, k, v)
    assert o.shape == q.shape and (o == 0).all()
    o.sum().backward()
    assert (q.grad == 0).all() and k.grad.shape == k.shape
    k = torch.randn(2, 2, 9, 64, device="cuda").to(dtype).requires_grad_()
    q0 = torch.randn(2, 2, 0, 64, device="cuda").to(dtype).requires_grad_()
    sq.cross_attention(q0, k, k).sum().backward()
    assert (k.grad == 0).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_autograd_layouts_and_broadcast_states(cuda_ok, dtype):
    # one encoding for every clip of the batch, seen through expand: its gradient is the sum
    B, h, n, m, d = 3, 4, 150, 90, 64
    q, k, v, do = problem(11, B, h, 2, n, m, d, dtype, "tokens")
    k1, v1 = k[:1].detach().clone().requires_grad_(), v[:1].detach().clone().requires_grad_()
    ql = q.detach().requires_grad_()
    o = sq.cross_attention(ql, k1.expand(B, -1, -1, -1), v1.expand(B, -1, -1, -1))
    assert o.stride() == q.stride()  # token-major in, token-major out
    o.backward(do)
    kb, vb = k[:1].expand(B, -1, -1, -1), v[:1].expand(B, -1, -1, -1)
    keep, s = keep_of(B, m), d ** -0.5
    _, _, bq, bk, bv = bounds(q, kb, vb, keep, s, do)
    rq, rk, rv = backward(q, kb, vb, keep, s, do)
    assert_within(ql.grad, rq, bq, "dq")
    u = torch.finfo(dtype).eps  # autograd's sum over the batch rounds once per addition
    assert_within(k1.grad, rk.sum(0, keepdim=True), bk.sum(0, keepdim=True) + 2 * u * rk.abs().sum(0, keepdim=True), "dk")
    assert_within(v1.grad, rv.sum(0, keepdim=True), bv.sum(0, keepdim=True) + 2 * u * rv.abs().sum(0, keepdim=True), "dv")
    # an expanded upstream gradient, and leaves that need none
    o = sq.cross_attention(ql, k, v)
    (g,) = torch.autograd.grad(o.sum(), ql)
    (r,) = torch.autograd.grad((sq.cross_attention(ql, k, v) * torch.ones_like(o)).sum(), ql)
    assert torch.equal(g, r)


def test_gradients_against_differences(cuda_ok):
    # the fp32 kernel's gradients against central differences of the 64-bit formula
    q, k, v, do = problem(12, 1, 2, 1, 5, 9, 32, F32)
    keep, s = keep_of(1, 9), 32 ** -0.5
    o, lse = sq.squad_cross_fwd(q, k, v)
    grads = sq.squad_cross_bwd(q, k, v, o, lse, do)
    xs = [t.double() for t in (q, k, v)]
    h = 1e-5
    for t, (x, g) in enumerate(zip(xs, grads)):
        for i in range(0, x.numel(), 7):
            both = []
            for sign in (1, -1):
                y = [z.clone() for z in xs]
                y[t].view(-1)[i] += sign * h
                both.append((forward(*y, keep, s)[0] * do.double()).sum().item())
            num = (both[0] - both[1]) / (2 * h)
            # differences: h^2 times a third derivative (below 1e2 here) and 1e-15 / h; kernel: fp32
            assert abs(num - g.reshape(-1)[i].item()) <= 1e-7 + 2e-5 * max(1.0, abs(num)), (t, i)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_repeats_bitwise_and_writes_only_its_rows(cuda_ok, dtype):
    B, h, n, m, d = 2, 4, 131, 300, 64
    q, k, v, do = problem(13, B, h, 2, n, m, d, dtype)
    lens = torch.tensor([300, 40], dtype=torch.int32, device="cuda")
    big = torch.full((B, h, n + 9, d), 7.0, device="cuda", dtype=dtype)
    o1, l1 = sq.squad_cross_fwd(q, k, v, kv_lens=lens, out=big[:, :, 4:4 + n])
    assert (big[:, :, :4] == 7).all() and (big[:, :, 4 + n:] == 7).all()
    o2, l2 = sq.squad_cross_fwd(q, k, v, kv_lens=lens)
    assert torch.equal(o1, o2) and torch.equal(l1, l2)
    g1 = sq.squad_cross_bwd(q, k, v, o2, l2, do, kv_lens=lens)
    g2 = sq.squad_cross_bwd(q, k, v, o2, l2, do, kv_lens=lens)
    assert all(torch.equal(a, b) for a, b in zip(g1, g2))
    sq.poll_device_error()


def test_streams_graphs_and_two_at_once(cuda_ok):
    B, h, n, m, d = 1, 4, 200, 700, 128
    probs = [problem(20 + i, B, h, h, n if i else 3, m, d) for i in range(2)]
    refs = [sq.squad_cross_fwd(*p[:3])[0].clone() for p in probs]
    grefs = [sq.squad_cross_bwd(*p[:3], *sq.squad_cross_fwd(*p[:3]), p[3]) for p in probs]
    torch.cuda.synchronize()
    # on streams of their own, both in flight
    streams = [torch.cuda.Stream() for _ in probs]
    outs = [None, None]
    for rep in range(5):
        for i, (p, st) in enumerate(zip(probs, streams)):
            outs[i] = sq.squad_cross_fwd(*p[:3], stream=st)[0]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, refs))
    # captured, with one memory pool for both graphs, and replayed in turn with new inputs
    pool, graphs, held = torch.cuda.graph_pool_handle(), [], []
    ins = [[t.clone() for t in p] for p in probs]
    for p in ins:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, pool=pool):
            o, lse = sq.squad_cross_fwd(*p[:3])
            gr = sq.squad_cross_bwd(*p[:3], o, lse, p[3])
        graphs.append(g)
        held.append((o, gr))
    for _ in range(2):
        for i, g in enumerate(graphs):
            for t, src in zip(ins[i], probs[i]):
                t.copy_(src)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(held[i][0], refs[i])
            assert all(torch.equal(a, b) for a, b in zip(held[i][1], grefs[i]))
    sq.poll_device_error()


def test_refusals(cuda_ok):
    q, k, v, do = problem(30, 2, 4, 2, 6, 9, 64)
    o, lse = sq.squad_cross_fwd(q, k, v)
    lens = torch.tensor([9, 9], dtype=torch.int32, device="cuda")
    for bad in (dict(kv_lens=lens.long()), dict(kv_lens=lens[:1]), dict(kv_lens=lens.cpu()),
                dict(key_mask=torch.ones(2, 8, dtype=torch.bool, device="cuda")),
                dict(key_mask=torch.ones(2, 9, device="cuda")), dict(key_mask=torch.ones(2, 9, dtype=torch.bool)),
                dict(key_mask=torch.ones(9, 2, dtype=torch.bool, device="cuda").t()),
                dict(out=torch.empty(2, 4, 6, 32, device="cuda", dtype=BF16)),
                dict(out=torch.empty(2, 4, 6, 64, device="cuda"))):
        with pytest.raises(ValueError):
            sq.squad_cross_fwd(q, k, v, **bad)
    for qq, kk, vv in ((q, k[:1], v[:1]), (q, k, v[:, :, :5]), (q, k[:, :, :, :32], v[:, :, :, :32]), (q[:, :3], k, v),
                       (q, k.float(), v), (q.cpu(), k, v), (q[0], k, v), (q.transpose(2, 3), k, v)):
        with pytest.raises(ValueError):
            sq.squad_cross_fwd(qq, kk, vv)
    with pytest.raises(TypeError):
        sq.squad_cross_fwd(q.half(), k.half(), v.half())
    with pytest.raises(ValueError):
        sq.squad_cross_bwd(q, k, v, o, lse[:1], do)
    with pytest.raises(ValueError):
        sq.squad_cross_bwd(q, k, v, o[:, :, :3], lse, do)
    x = torch.randn(2, 4, 6, 96, device="cuda").to(BF16)
    with pytest.raises(sq.SquadError):
        sq.squad_cross_fwd(x, x, x)  # bf16 heads of 96
    flat = torch.randn(2 * 4 * 6 * 64 + 8, device="cuda").to(BF16)
    with pytest.raises(sq.SquadError):
        sq.squad_cross_fwd(flat[1:1 + q.numel()].view(q.shape), k, v)  # 2 bytes off
    odd = torch.randn(2, 4, 6, 68, device="cuda").to(BF16)[..., :64]
    with pytest.raises(sq.SquadError):
        sq.squad_cross_fwd(odd, k, v)  # rows 136 bytes apart
    with pytest.raises(sq.SquadError):
        sq.squad_cross_fwd(q[:, :, :1].expand(-1, -1, 6, -1), k, v)  # every query the same memory
    sq.poll_device_error()
