"""Rotary positions on the GPU against complex multiplication in 64 bits.

y = a c - b s takes two products and one sum in fp32 from an fp32 table: with e = 2^-24 the products, the
sum and the table's rounding are off by at most 4 e (|a| + |b|), the output's rounding by u |y|, u = eps / 2.
"""
import pytest
import torch

import sub_quadratic_two_b200 as sq
from workloads import random_problem

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def turned(x, grid, axes, pairing, theta=10000.0, offset=(0, 0, 0), inverse=False):
    """(rotated, |a| + |b| of each channel's pair) in fp64."""
    T, H, W = grid
    tok = torch.arange(T * H * W, device=x.device)
    ang = []
    for p, c, first in zip((tok // (H * W), tok // W % H, tok % W), axes, offset):
        i = torch.arange(c // 2, device=x.device, dtype=torch.float64)
        ang.append((p.double() + first)[:, None] * torch.exp(-2 * i / max(c, 1) * torch.log(torch.tensor(theta).double())))
    ang = torch.cat(ang, 1) * (-1 if inverse else 1)
    w = torch.polar(torch.ones_like(ang), ang)
    r, x = sum(axes), x.double()
    out, mag = x.clone(), torch.zeros_like(x)
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if pairing == "adjacent" else (x[..., : r // 2], x[..., r // 2: r])
    z, both = torch.complex(a.contiguous(), b.contiguous()) * w, a.abs() + b.abs()
    if pairing == "adjacent":
        out[..., 0:r:2], out[..., 1:r:2] = z.real, z.imag
        mag[..., 0:r:2], mag[..., 1:r:2] = both, both
    else:
        out[..., : r // 2], out[..., r // 2: r] = z.real, z.imag
        mag[..., : r // 2], mag[..., r // 2: r] = both, both
    return out, mag


def close(y, ref, mag, what=""):
    u = torch.finfo(y.dtype).eps / 2
    err = (y.double() - ref).abs()
    assert (err <= u * ref.abs() * (1 + 2.0 ** -20) + 5 * 2.0 ** -24 * mag).all(), (what, err.max().item())


CASES = [  # B, heads, kv heads, d, grid, axes, pairing
    (1, 1, 1, 8, (1, 1, 1), (4, 2, 2), "adjacent"), (1, 2, 2, 64, (2, 3, 5), None, "adjacent"),
    (2, 8, 4, 128, (3, 7, 9), None, "adjacent"), (1, 3, 1, 96, (2, 5, 11), (32, 32, 32), "adjacent"),
    (1, 9, 8, 128, (1, 22, 40), None, "half"), (2, 2, 2, 64, (5, 4, 3), (16, 24, 24), "half"),
    (1, 4, 2, 128, (2, 4, 4), (20, 6, 6), "adjacent"), (1, 4, 2, 128, (2, 4, 4), (32, 16, 16), "half"),
    (1, 2, 2, 64, (4, 1, 1), (64, 0, 0), "adjacent"), (1, 2, 1, 256, (1, 3, 130), (0, 128, 128), "half"),
    (1, 17, 16, 64, (1, 1, 300), (0, 0, 64), "adjacent"), (1, 2, 2, 1024, (1, 2, 3), (512, 256, 256), "adjacent"),
    (1, 2, 2, 64, (2, 2, 2), (0, 0, 0), "adjacent"),
]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,h,hk,d,grid,axes,pairing", CASES)
def test_forward_and_gradients(cuda_ok, B, h, hk, d, grid, axes, pairing, dtype):
    gen = torch.Generator(device="cuda").manual_seed(d + h)
    n = grid[0] * grid[1] * grid[2]
    rot = sq.rotary_plan(grid, d, axes, pairing=pairing, offset=(7, 0, 2))
    for layout in ("tokens", "heads"):
        xs = [torch.randn((B, n, x, d) if layout == "tokens" else (B, x, n, d), generator=gen, device="cuda").to(dtype)
              for x in (h, hk)]
        xs = [(x.transpose(1, 2) if layout == "tokens" else x).requires_grad_() for x in xs]
        ys = sq.rotary(*xs, rot)
        gs = [torch.randn(y.shape, generator=gen, device="cuda").to(dtype) for y in ys]
        dxs = torch.autograd.grad(ys, xs, gs)
        for x, y, g, dx in zip(xs, ys, gs, dxs):
            assert y.is_contiguous()
            close(y.detach(), *turned(x.detach(), grid, rot.axes, pairing, offset=(7, 0, 2)), "forward")
            close(dx, *turned(g, grid, rot.axes, pairing, offset=(7, 0, 2), inverse=True), "gradient")
            assert dx.shape == x.shape and (n == 1 or x.shape[1] == 1 or dx.stride() == x.stride())


def test_far_positions_and_another_base(cuda_ok):
    grid, off = (2, 3, 4), (1_000_000, 0, 70_000)
    x = torch.randn(1, 2, 24, 64, device="cuda")
    rot = sq.rotary_plan(grid, 64, theta=256.0, offset=off)
    (y,) = sq.squad_rotary([x], rot)
    close(y, *turned(x, grid, rot.axes, "adjacent", 256.0, off))


@pytest.mark.parametrize("pairing", ["adjacent", "half"])
def test_in_place_one_tensor_and_back(cuda_ok, pairing):
    grid = (2, 5, 7)
    x = torch.randn(2, 3, 70, 64, device="cuda")
    rot = sq.rotary_plan(grid, 64, (16, 24, 24), pairing=pairing)
    y, none = sq.rotary(x, None, rot)
    assert none is None
    z = x.clone()
    sq.squad_rotary([z], rot, out=[z])
    assert torch.equal(z, y)
    sq.squad_rotary([z], rot, inverse=True, out=[z])
    # two rotations of fp32: 2 * 5 * 2^-24 * (|a| + |b|), |a| + |b| below 16 here
    assert (z - x).abs().max().item() <= 10 * 2.0 ** -24 * 16


def test_writes_only_its_rows_and_reads_past_none(cuda_ok):
    grid, n = (1, 3, 7), 21
    big = torch.full((2, 4, n + 6, 64), float("nan"), device="cuda", dtype=BF16)
    big[:, :, 3:3 + n] = 1.0
    out = torch.full_like(big, 9.0)
    rot = sq.rotary_plan(grid, 64)
    sq.squad_rotary([big[:, :, 3:3 + n]], rot, out=[out[:, :, 3:3 + n]])
    assert (out[:, :, :3] == 9).all() and (out[:, :, 3 + n:] == 9).all() and torch.isfinite(out).all()


def test_gradient_against_differences(cuda_ok):
    grid, d = (2, 2, 3), 16
    x, g = torch.randn(1, 1, 12, d, device="cuda"), torch.randn(1, 1, 12, d, device="cuda")
    rot = sq.rotary_plan(grid, d, (4, 6, 6))
    xl = x.clone().requires_grad_()
    (dx,) = torch.autograd.grad(sq.rotary(xl, None, rot)[0], xl, g)
    f = lambda z: (turned(z, grid, (4, 6, 6), "adjacent")[0] * g.double()).sum().item()  # noqa: E731
    for i in range(0, x.numel(), 5):
        e = torch.zeros_like(x).double().view(-1)
        e[i] = 1e-3  # linear: differences are exact up to 64-bit rounding
        num = (f(x.double() + e.view_as(x)) - f(x.double() - e.view_as(x))) / 2e-3
        assert abs(num - dx.view(-1)[i].item()) <= 1e-6


def test_streams_and_graphs(cuda_ok):
    grid = (3, 6, 10)
    rot = sq.rotary_plan(grid, 128)
    q, k = (torch.randn(1, 180, h, 128, device="cuda").to(BF16).transpose(1, 2) for h in (8, 2))
    ref = sq.squad_rotary([q, k], rot)
    torch.cuda.synchronize()
    got = sq.squad_rotary([q, k], rot, stream=torch.cuda.Stream())
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, got))
    qs, ks = torch.zeros_like(q), torch.zeros_like(k)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = sq.squad_rotary([qs, ks], rot)
    qs.copy_(q)
    ks.copy_(k)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, out))


def test_attention_with_positions(cuda_ok):
    # attention(..., rotary=) is attention of the turned q and k, gradients included
    grid, tile, d = (2, 8, 8), (1, 4, 4), 64
    inp = random_problem(71, 1, 2, d, grid, tile, dtype=BF16, with_do=True)
    rot = sq.rotary_plan(grid, d)
    tok = [t.cuda().transpose(1, 2).contiguous().transpose(1, 2).requires_grad_() for t in (inp.q, inp.k)]
    v, do = inp.v.cuda().requires_grad_(), inp.do.cuda()
    for call in (lambda q, k, **kw: sq.attention(q, k, v, grid, tile, **kw),
                 lambda q, k, **kw: sq.attention_multi(q, k, v, grid, [(1, 1, 4), tile], **kw)):
        o = call(*tok, rotary=rot)
        grads = torch.autograd.grad(o, tok + [v], do)
        yq, yk = (t.detach().requires_grad_() for t in sq.rotary(*tok, rot))
        o2 = call(yq, yk)
        gq, gk, gv = torch.autograd.grad(o2, (yq, yk, v), do)
        assert torch.equal(o, o2)
        back = sq.squad_rotary([gq, gk], rot, inverse=True)
        for a, b in zip(grads[:2], back):
            # dq of problems over several boxes is summed in hardware order, one bf16 step apart at most
            assert (a.float() - b.float()).abs().max().item() <= 2.0 ** -7 * b.float().abs().max().item()
    with pytest.raises(ValueError):
        sq.attention(*tok, v, grid, tile, rotary=sq.rotary_plan((2, 8, 4), d))
    sq.poll_device_error()


def test_block_of_a_video_transformer(cuda_ok):
    """Rotary positions, grid attention and cross attention in a row, as a layer runs them: forward and gradients."""
    from cross_formula import backward, forward, keep_of
    grid, tile, h, d, m = (2, 4, 8), (1, 4, 4), 2, 64, 77
    n, g = 64, torch.Generator(device="cuda").manual_seed(3)
    mk = lambda r: torch.randn(2, r, h, d, generator=g, device="cuda")  # noqa: E731
    q, k, tk, tv = mk(n), mk(n), mk(m), mk(m)
    v = torch.randn(2, h, n, d, generator=g, device="cuda")
    q, k, tk, tv, v = leaves = [t.requires_grad_() for t in (q, k, tk, tv, v)]
    lens = torch.tensor([77, 20], dtype=torch.int32, device="cuda")
    rot = sq.rotary_plan(grid, d)
    x = sq.attention(q.transpose(1, 2), k.transpose(1, 2), v, grid, tile, rotary=rot)
    y = sq.cross_attention(x, tk.transpose(1, 2), tv.transpose(1, 2), kv_lens=lens)
    do = torch.randn(y.shape, generator=g, device="cuda")
    grads = torch.autograd.grad(y, leaves, do)

    def plain(q, k, tk, tv, v):
        def turn(t):
            return turned_diff(t.transpose(1, 2), grid, rot.axes)
        qr, kr = turn(q), turn(k)
        T, H, W = grid
        tt, th, tw = tile
        win = lambda z: z.reshape(2, h, T // tt, tt, H // th, th, W // tw, tw, d)  # noqa: E731
        loc = lambda z: win(z).permute(0, 1, 2, 4, 6, 3, 5, 7, 8).reshape(2, h, -1, tt * th * tw, d)  # noqa: E731
        att = lambda a, b, c: torch.softmax(a @ b.transpose(-1, -2) / d ** 0.5, -1) @ c  # noqa: E731
        ql, kl, vl = loc(qr), loc(kr), loc(v)
        o1 = att(ql, kl, vl)
        o2 = att(*(z.transpose(2, 3) for z in (ql, kl, o1))).transpose(2, 3)
        o2 = o2.reshape(2, h, T // tt, H // th, W // tw, tt, th, tw, d).permute(0, 1, 2, 5, 3, 6, 4, 7, 8).reshape(2, h, n, d)
        s = o2 @ tk.permute(0, 2, 3, 1) / d ** 0.5
        s = s.masked_fill(~keep_of(2, m, lens)[:, None, None], float("-inf"))
        return torch.softmax(s, -1) @ tv.transpose(1, 2)

    def turned_diff(x, grid, axes):
        T, H, W = grid
        tok = torch.arange(n, device="cuda")
        ang = torch.cat([p.double()[:, None] * 10000.0 ** (-torch.arange(0, c, 2, device="cuda").double() / c)
                         for p, c in zip((tok // (H * W), tok // W % H, tok % W), axes)], 1)
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * ang.cos() - b * ang.sin(), a * ang.sin() + b * ang.cos()], -1).flatten(-2)

    dbl = [t.detach().double().requires_grad_() for t in leaves]
    ref = plain(*dbl)
    # fp32 through four operators of up to 77-term sums: some hundreds of 2^-24 steps of values of order 1
    assert (y.double() - ref).abs().max().item() <= 2e-5
    for name, a, b in zip(("q", "k", "text k", "text v", "v"), grads, torch.autograd.grad(ref, dbl, do.double())):
        assert (a.double() - b).abs().max().item() <= 4e-5 * max(1.0, b.abs().max().item()), name
    sq.poll_device_error()


def test_refusals(cuda_ok):
    rot = sq.rotary_plan((1, 2, 3), 64)
    x = torch.randn(1, 2, 6, 64, device="cuda")
    for bad in ([x[:, :, :5]], [x, x[:, :, :5]], [x.cpu()], [x, x.to(BF16)], [x, x, x], [x.transpose(1, 2)[0]],
                [x.transpose(2, 3)]):
        with pytest.raises(ValueError):
            sq.squad_rotary(bad, rot)
    with pytest.raises(TypeError):
        sq.squad_rotary([x.double()], rot)
    with pytest.raises(ValueError):
        sq.squad_rotary([x], rot, out=[torch.empty(1, 2, 6, 32, device="cuda")])
    with pytest.raises(ValueError):
        sq.squad_rotary([x], sq.rotary_plan((1, 2, 3), 64, device="cpu"))
    with pytest.raises(sq.SquadError):  # 64 - 20 channels to copy do not make whole chunk pairs
        sq.squad_rotary([x.to(BF16)], sq.rotary_plan((1, 2, 3), 64, (8, 6, 6), pairing="half"))
    with pytest.raises(sq.SquadError):
        sq.squad_rotary([x[..., 1:33]], sq.rotary_plan((1, 2, 3), 32))  # 4 bytes off
    with pytest.raises(sq.SquadError):
        sq.squad_rotary([x[..., :32]], sq.rotary_plan((1, 2, 3), 64))  # a table of more channels than d


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d,axes,pairing", [
    (128, (20, 6, 6), "adjacent"), (64, (2, 0, 0), "adjacent"), (64, (0, 0, 0), "adjacent"), (64, (0, 0, 0), "half"),
    (128, (32, 16, 16), "half"), (96, (2, 4, 8), "adjacent")])
def test_copied_channels_are_copied(cuda_ok, dtype, d, axes, pairing):
    # channels past the axes', whatever their neighbours hold: infinities, NaN and signed zeros bit by bit
    grid, n = (2, 3, 5), 30
    rot = sq.rotary_plan(grid, d, axes, pairing=pairing, offset=(3, 0, 1))
    r = sum(axes)
    x = torch.randn(2, 3, n, d, generator=torch.Generator(device="cuda").manual_seed(d + r), device="cuda").to(dtype)
    finite = x.clone()
    odd = torch.tensor([float("inf"), -0.0, float("nan"), 0.0, -float("inf"), -1.0, 0.0], device="cuda").to(dtype)
    x[..., r:] = odd[torch.arange(d - r, device="cuda") % 7]
    for inverse in (False, True):
        (y,) = sq.squad_rotary([x], rot, inverse=inverse)
        bits = torch.int16 if dtype == BF16 else torch.int32
        assert torch.equal(y[..., r:].contiguous().view(bits), x[..., r:].contiguous().view(bits))
        # and they leave the turned channels alone
        assert torch.equal(y[..., :r], sq.squad_rotary([finite], rot, inverse=inverse)[0][..., :r])
