"""Kept calls of cross attention (cross.py) on the CPU, with stand-ins for what needs a device: the descriptor that a
backward launches with is the one of the tensors that it is given."""
import pytest
import torch

import sub_quadratic_two_b200 as sq
from sub_quadratic_two_b200 import cross


@pytest.fixture
def launches(monkeypatch):
    """(descriptor, tensors) of every backward; forwards and backwards compute nothing."""
    seen = []

    def run_fwd(call, q, k, v, kv_lens, key_mask, save, out=None):
        return cross.empty_like_layout(q).zero_(), q.new_zeros(q.shape[:3], dtype=torch.float32)

    def run_bwd(call, q, k, v, o, lse, dout, kv_lens, key_mask):
        seen.append((call.desc, dict(q=q, k=k, v=v, o=o, dout=dout)))
        return torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)

    monkeypatch.setattr(cross, "_calls", {})
    monkeypatch.setattr(cross, "check_strided", lambda *named: None)
    monkeypatch.setattr(cross, "_check_aux", lambda *args: None)
    monkeypatch.setattr(cross, "_run_fwd", run_fwd)
    monkeypatch.setattr(cross, "_run_bwd", run_bwd)
    return seen


def fits(desc, tensors):
    for name, t in tensors.items():
        st = getattr(desc, name)
        assert (st.b, st.h, st.n) == t.stride()[:3], name


@pytest.mark.parametrize("dense_first", [False, True])
def test_saved_tensors_may_come_back_in_another_layout(launches, dense_first):
    # hooks on saved tensors (offloading to the host, say) hand them to the backward as dense copies: rows of a wide
    # projection come back without the gaps between them, and strides of the one must not be used on the other
    wide = torch.randn(2, 6, 3, 4, 64)  # [B, tokens, (q, k, v), heads, d]
    leaves = [wide[:, :, i].transpose(1, 2).detach().requires_grad_() for i in range(3)]

    def step(dense):
        if dense:
            with torch.autograd.graph.saved_tensors_hooks(lambda t: t.detach().clone(memory_format=torch.contiguous_format),
                                                          lambda t: t):
                o = sq.cross_attention(*leaves)
        else:
            o = sq.cross_attention(*leaves)
        torch.autograd.grad(o, leaves, torch.ones_like(o))

    for dense in (dense_first, not dense_first, dense_first):
        step(dense)
    for i, dense in enumerate((dense_first, not dense_first, dense_first)):
        desc, tensors = launches[i]
        assert tensors["q"].is_contiguous() == dense
        fits(desc, tensors)


def test_saved_tensors_of_another_kind_are_not_run_with_a_kept_call(launches):
    # a hook that gives back fewer rows: the kept call's sizes must not be used on them
    q = torch.randn(1, 2, 8, 64, requires_grad=True)
    k, v = torch.randn(1, 2, 9, 64), torch.randn(1, 2, 9, 64)
    o = sq.cross_attention(q, k, v)
    torch.autograd.grad(o, q, torch.ones_like(o))
    with torch.autograd.graph.saved_tensors_hooks(lambda t: t.detach(), lambda t: t[:, :, :5] if t.shape[2] == 9 else t):
        o = sq.cross_attention(q, k, v)
    torch.autograd.grad(o, q, torch.ones_like(o))
    assert [desc.m for desc, _ in launches] == [9, 5]


@pytest.mark.parametrize("which", [0, 1, 2])
def test_forward_mode_tangents_are_refused(launches, which):
    ts = [torch.randn(1, 2, 6, 64) for _ in range(3)]
    fw = torch.autograd.forward_ad
    with fw.dual_level():
        sq.cross_attention(*ts)
        ts[which] = fw.make_dual(ts[which], torch.ones_like(ts[which]))
        with pytest.raises(RuntimeError, match="jvp"):
            sq.cross_attention(*ts)
        with torch.no_grad(), pytest.raises(RuntimeError, match="jvp"):
            sq.cross_attention(*ts)


def test_a_tangent_of_the_incoming_gradient_is_refused(launches):
    q, k, v = (torch.randn(1, 2, 6, 64, requires_grad=True) for _ in range(3))
    fw = torch.autograd.forward_ad
    with fw.dual_level():
        o = sq.cross_attention(q, k, v)
        dout = torch.ones_like(o)
        torch.autograd.grad(o, q, dout, retain_graph=True)
        with pytest.raises(RuntimeError, match="forward-mode"):
            torch.autograd.grad(o, q, fw.make_dual(dout, dout))


def test_a_scale_that_wants_a_gradient_is_refused(launches):
    q, k, v = (torch.randn(1, 2, 6, 64) for _ in range(3))
    scale = torch.tensor(0.1, requires_grad=True)
    for t in (q, q.clone().requires_grad_()):
        with pytest.raises(ValueError, match="constant"):
            sq.cross_attention(t, k, v, scale=scale)
    sq.cross_attention(q, k, v, scale=scale.detach())
    fw = torch.autograd.forward_ad
    with fw.dual_level(), pytest.raises(ValueError, match="constant"):
        sq.cross_attention(q, k, v, scale=fw.make_dual(scale.detach(), torch.tensor(1.0)))
