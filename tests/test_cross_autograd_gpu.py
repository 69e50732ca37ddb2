"""Cross attention and rotary positions under what torch's autograd may do around a call: saved tensors kept
elsewhere, derivatives of other kinds, tensors that need none. Bounds as in cross_formula.py."""
import pytest
import torch

import sub_quadratic_two_b200 as sq
from cross_formula import assert_within, backward, bounds, forward, keep_of
from test_cross_gpu import BF16, F32, problem

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("offloaded_first", [False, True])
def test_saved_tensors_kept_on_the_host(cuda_ok, dtype, offloaded_first):
    # what save_on_cpu brings back is dense, whatever lay in the forward: rows of a wide projection lose their gaps
    B, h, n, m, d = 2, 4, 150, 90, 64
    gen = torch.Generator(device="cuda").manual_seed(60)
    wide = torch.randn(B, n, 3, h, d, generator=gen, device="cuda").to(dtype)
    states = torch.randn(B, m, 2, h, d, generator=gen, device="cuda").to(dtype)
    q, k, v = wide[:, :, 1].transpose(1, 2), states[:, :, 0].transpose(1, 2), states[:, :, 1].transpose(1, 2)
    do = torch.randn(B, h, n, d, generator=gen, device="cuda").to(dtype)
    leaves = [t.detach().requires_grad_() for t in (q, k, v)]
    lens = torch.tensor([m, 31], dtype=torch.int32, device="cuda")
    keep, s = keep_of(B, m, lens), d ** -0.5
    bs, want = bounds(q, k, v, keep, s, do), backward(q, k, v, keep, s, do)
    for offloaded in (offloaded_first, not offloaded_first, offloaded_first):
        if offloaded:
            with torch.autograd.graph.save_on_cpu():
                o = sq.cross_attention(*leaves, kv_lens=lens)
        else:
            o = sq.cross_attention(*leaves, kv_lens=lens)
        grads = torch.autograd.grad(o, leaves, do)
        assert_within(o.detach(), forward(q, k, v, keep, s)[0], bs[0], "o")
        for name, g, r, b in zip(("dq", "dk", "dv"), grads, want, bs[2:]):
            assert_within(g, r, b, name)
    sq.poll_device_error()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,m", [(5, 9), (300, 200), (130, 700), (1, 3000)])
def test_queries_without_states_give_no_gradient_whatever_comes_in(cuda_ok, dtype, n, m):
    # dout of a query without states may be infinite or NaN (a loss over padded rows, say), and so may the query
    B, d = 4, 64
    q, k, v, do = problem(61, B, 4, 2, n, m, d, dtype)
    q[1], do[1], do[2], do[3] = float("nan"), float("inf"), float("nan"), -float("inf")
    mask = torch.ones(B, m, dtype=torch.bool, device="cuda")
    mask[1:] = False
    lens = torch.tensor([m, 0, 0, 0], dtype=torch.int32, device="cuda")
    keep, s = keep_of(1, m), d ** -0.5
    bs, want = bounds(q[:1], k[:1], v[:1], keep, s, do[:1])[2:], backward(q[:1], k[:1], v[:1], keep, s, do[:1])
    for kw in (dict(key_mask=mask), dict(kv_lens=lens), dict(key_mask=mask, kv_lens=lens)):
        o, lse = sq.squad_cross_fwd(q, k, v, **kw)
        for name, g, r, b in zip(("dq", "dk", "dv"), sq.squad_cross_bwd(q, k, v, o, lse, do, **kw), want, bs):
            assert (g[1:] == 0).all(), name
            assert_within(g[:1], r, b, name)
    sq.poll_device_error()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,m", [(5, 9), (300, 200), (700, 130), (1, 3000)])
def test_states_that_do_not_count_get_zeros_whatever_comes_in(cuda_ok, dtype, n, m):
    B, d = 2, 64
    q, k, v, do = problem(63, B, 4, 2, n, m, d, dtype)
    do[0, 1, n // 2], q[1, 3, 0] = float("nan"), float("inf")
    mask = torch.rand(B, m, generator=torch.Generator().manual_seed(m)).cuda() < 0.6
    mask[:, 0] = True
    lens = torch.tensor([m - 1, 1], dtype=torch.int32, device="cuda")
    for kw in (dict(key_mask=mask), dict(kv_lens=lens), dict(key_mask=mask, kv_lens=lens)):
        dead = ~keep_of(B, m, kw.get("kv_lens"), kw.get("key_mask"))
        o, lse = sq.squad_cross_fwd(q, k, v, **kw)
        _, dk, dv = sq.squad_cross_bwd(q, k, v, o, lse, do, **kw)
        for g in (dk, dv):
            assert (g.transpose(1, 2)[dead] == 0).all()
    sq.poll_device_error()


def test_forward_mode_is_refused(cuda_ok):
    # a tangent has no formula here: it must not be lost
    grid = (1, 2, 3)
    rot = sq.rotary_plan(grid, 64)
    x, t = torch.randn(1, 2, 6, 64, device="cuda"), torch.randn(1, 2, 6, 64, device="cuda")
    fw = torch.autograd.forward_ad
    with fw.dual_level():
        dual = fw.make_dual(x, t)
        for call in (lambda: sq.cross_attention(dual, x, x), lambda: sq.cross_attention(x, dual, x),
                     lambda: sq.cross_attention(x, x, dual), lambda: sq.rotary(dual, None, rot),
                     lambda: sq.rotary(x, dual, rot), lambda: sq.attention(dual, x, x, grid, (1, 1, 3), rotary=rot),
                     lambda: sq.attention(x, x, dual, grid, (1, 1, 3), rotary=rot)):
            with pytest.raises(RuntimeError):
                call()
            with torch.no_grad(), pytest.raises(RuntimeError):
                call()
        # without tangents a call is as it is outside
        assert torch.equal(sq.cross_attention(x, x, x), sq.squad_cross_fwd(x, x, x)[0])
        y, z = sq.rotary(x, None, rot)
        assert z is None and torch.equal(y, sq.squad_rotary([x], rot)[0])


def test_a_table_that_wants_a_gradient_is_refused(cuda_ok):
    rot = sq.rotary_plan((1, 2, 3), 64)
    x = torch.randn(1, 2, 6, 64, device="cuda")
    learned = sq.Rotary(rot.grid, rot.axes, rot.table.clone().requires_grad_())
    for q in (x, x.clone().requires_grad_()):
        for call in (lambda: sq.rotary(q, None, learned), lambda: sq.rotary(q, q, learned),
                     lambda: sq.attention(q, q, q, (1, 2, 3), (1, 1, 3), rotary=learned),
                     lambda: sq.attention_multi(q, q, q, (1, 2, 3), [(1, 1, 3)], rotary=learned)):
            with pytest.raises(ValueError):
                call()
    with torch.no_grad():
        assert torch.equal(sq.rotary(x, None, learned)[0], sq.rotary(x, None, rot)[0])
    fw = torch.autograd.forward_ad
    with fw.dual_level():
        dual = sq.Rotary(rot.grid, rot.axes, fw.make_dual(rot.table, torch.ones_like(rot.table)))
        with pytest.raises(ValueError):
            sq.rotary(x, None, dual)
        with torch.no_grad(), pytest.raises(ValueError):
            sq.rotary(x, None, dual)


def test_a_scale_that_wants_a_gradient_is_refused(cuda_ok):
    q, k, v, _ = problem(62, 1, 2, 2, 6, 9, 64)
    scale = torch.tensor(0.1, requires_grad=True)
    for t in (q, q.clone().requires_grad_()):
        with pytest.raises(ValueError):
            sq.cross_attention(t, k, v, scale=scale)
    with torch.no_grad():
        assert torch.equal(sq.cross_attention(q, k, v, scale=scale), sq.cross_attention(q, k, v, scale=scale.item()))
