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
