"""Cross attention calls that take seconds. Bounds as in cross_formula.py."""
import pytest
import torch

import sub_quadratic_two_b200 as sq
from cross_formula import E32, assert_within

pytestmark = pytest.mark.gpu


def test_a_length_that_ends_inside_a_block_after_seconds_of_others(cuda_ok):
    # 32,000 items whose lengths are whole blocks but for the last batch row's: the warp that masks value tiles has
    # nothing to do for more than the 2 s that a wait of one job may last. Queries and states are broadcast, so
    # that all rows of one length come out alike.
    B, h, n, m, d = 80, 100, 1024, 1 << 20, 64
    gen = torch.Generator(device="cuda").manual_seed(70)
    q, k, v = (torch.randn(1, 1, r, d, generator=gen, device="cuda").bfloat16() for r in (n, m, m))
    lens = torch.full((B,), m, dtype=torch.int32)
    lens[-1] = m - 128 * 700 - 37
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    o, lse = sq.squad_cross_fwd(q.expand(B, h, -1, -1), k.expand(B, -1, -1, -1), v.expand(B, -1, -1, -1),
                                kv_lens=lens.cuda())
    end.record()
    torch.cuda.synchronize()
    sq.poll_device_error()
    print(f"{start.elapsed_time(end) / 1e3:.2f} s")
    rows = torch.tensor([0, 127, 128, 700, 1023], device="cuda")
    s = d ** -0.5
    for b, length in ((0, m), (B - 1, int(lens[-1]))):
        assert (o[b] == o[b, 0]).all() and (lse[b] == lse[b, 0]).all()
        z = q[0, 0, rows].double() @ k[0, 0, :length].double().T * s
        p = torch.softmax(z, 1)
        ref = p @ v[0, 0, :length].double()
        E = (d + 4) * E32 * s * (q[0, 0, rows].double().abs() @ k[0, 0, :length].double().abs().T).amax(1, keepdim=True)
        # P to bf16 is off by 2^-8 of itself at most, the m terms of a sum by e each
        x = 2 * E + 2.0 ** -20 + m * E32
        assert_within(o[b, 0, rows], ref, (x + 2.0 ** -8) * (p @ v[0, 0, :length].double().abs()) + 2.0 ** -8 * ref.abs(), "o")
        assert_within(lse[b, 0, rows], torch.logsumexp(z, 1), x[:, 0] + 400 * E32, "lse")
    assert all(torch.equal(o[b], o[0]) for b in range(1, B - 1))
