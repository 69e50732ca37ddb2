"""Cross attention from its definition in 64 bits, and how far a kernel may be from it.

The kernels hold scores, softmax statistics and sums in fp32 and, on bf16, round P and dS to bf16
before the products that read them and each output once. With u = finfo(dtype).eps / 2 for those
roundings (0 for P and dS on fp32) and e = 2^-24 for fp32 steps, element by element:
  scores   |ds_ij| <= E = (d + 4) e s sum_c |q||k| , so P is off by a factor within x = 2 max E + 2^-20
           (exponent, normalising sum of up to m terms: + m e)
  o        (x + u_p + m e) sum_j P |v|  +  u |o|
  dP       (d + 4) e sum_c |dO||v|;  D: sum_c |dO| err_o + d e sum_c |dO||o|
  dS       (x + m e) |dS| + P (err_dP + err_D), then u_p |dS|
  dq, dk   s times the error of dS against |k|, |q|, + (terms) e s sum |dS||k|, + u |dq|
  dv       (x + u_p + n e) sum_i P |dO| + u |dv|
"""
import math

import torch

E32 = 2.0 ** -24


def keep_of(B, m, kv_lens=None, key_mask=None, device="cuda"):
    keep = torch.ones(B, m, dtype=torch.bool, device=device)
    if kv_lens is not None:
        keep &= torch.arange(m, device=device)[None] < kv_lens.to(device)[:, None]
    if key_mask is not None:
        keep &= key_mask.to(device)
    return keep


def forward(q, k, v, keep, scale):
    """o and lse in fp64 ([B, h, n, d], [B, h, n]) and what the bounds need."""
    g = q.shape[1] // k.shape[1]
    rows = keep[:, None, :, None]
    q = q.double()
    k = torch.where(rows, k.double(), 0.0).repeat_interleave(g, 1)
    v = torch.where(rows, v.double(), 0.0).repeat_interleave(g, 1)
    s = torch.einsum("bhnd,bhmd->bhnm", q, k) * scale
    s = s.masked_fill(~keep[:, None, None, :], -math.inf)
    lse = torch.logsumexp(s, -1)
    p = torch.where(keep[:, None, None, :], torch.exp(s - torch.where(lse == -math.inf, 0.0, lse)[..., None]), 0.0)
    return torch.einsum("bhnm,bhmd->bhnd", p, v), lse, (q, k, v, p)


def backward(q, k, v, keep, scale, dout):
    """(dq, dk, dv) in fp64 from the formulas, dk and dv summed over each group of query heads."""
    g = q.shape[1] // k.shape[1]
    o, _, (q, k, v, p) = forward(q, k, v, keep, scale)
    do = dout.double()
    dp = torch.einsum("bhnd,bhmd->bhnm", do, v)
    ds = p * (dp - (do * o).sum(-1, keepdim=True)) * scale
    B, h, m, d = k.shape
    fold = lambda t: t.reshape(B, h // g, g, m, d).sum(2)  # noqa: E731
    return (torch.einsum("bhnm,bhmd->bhnd", ds, k), fold(torch.einsum("bhnm,bhnd->bhmd", ds, q)),
            fold(torch.einsum("bhnm,bhnd->bhmd", p, do)))


def bounds(q, k, v, keep, scale, dout=None):
    """Element-wise bounds on the errors of (o, lse[, dq, dk, dv]), as above."""
    u = torch.finfo(q.dtype).eps / 2
    up = u if q.dtype == torch.bfloat16 else 0.0
    g, B, hk, m, d = q.shape[1] // k.shape[1], *k.shape
    n = q.shape[2]
    o, _, (q, k, v, p) = forward(q, k, v, keep, scale)
    E = (d + 4) * E32 * scale * torch.einsum("bhnd,bhmd->bhnm", q.abs(), k.abs()).amax(-1, keepdim=True)
    x = 2 * E + 2.0 ** -20 + m * E32
    eo = (x + up + m * E32) * torch.einsum("bhnm,bhmd->bhnd", p, v.abs()) + u * o.abs()
    el = x[..., 0] + 4 * E32 * 100
    if dout is None:
        return eo, el
    do = dout.double()
    dp = torch.einsum("bhnd,bhmd->bhnm", do, v)
    ds = p * (dp - (do * o).sum(-1, keepdim=True))
    edp = (d + 4) * E32 * torch.einsum("bhnd,bhmd->bhnm", do.abs(), v.abs())
    ed = (do.abs() * eo).sum(-1, keepdim=True) + d * E32 * (do * o).abs().sum(-1, keepdim=True)
    eds = (x + up) * ds.abs() + p * (edp + ed)
    dq, dk, dv = backward(q, k.reshape(B, hk, g, m, d)[:, :, 0], v.reshape(B, hk, g, m, d)[:, :, 0], keep, scale, dout)
    fold = lambda t: t.reshape(B, hk, g, m, d).sum(2)  # noqa: E731
    edq = scale * torch.einsum("bhnm,bhmd->bhnd", eds + (m + 4) * E32 * ds.abs(), k.abs()) + u * dq.abs()
    edk = scale * fold(torch.einsum("bhnm,bhnd->bhmd", eds + (n * g + 4) * E32 * ds.abs(), q.abs())) + u * dk.abs()
    edv = fold(torch.einsum("bhnm,bhnd->bhmd", (x + up + (n * g + 4) * E32) * p, do.abs())) + u * dv.abs()
    return eo, el, edq, edk, edv


def assert_within(got, ref, bound, what):
    got, ref = got.double(), ref.double()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    over = ((got - ref).abs() - bound - 1e-30).clamp_min(0)
    worst = ((got - ref).abs() / (bound + 1e-30)).max().item()
    assert over.max().item() == 0.0, f"{what}: {worst:.2f} times the bound, |err| {(got - ref).abs().max().item():.3e}"
