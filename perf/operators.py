"""What is measured of the operators around the grid attention: cross attention to an encoder's
states (forward, training step, one pooled query) and the rotary positions of a T x H x W grid
(forward, training step). `own` selects the library's kernels; otherwise `run` computes the plain
torch forms in 32 bits."""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------------- cases

def listed():
    cross = dict(op="cross", B=1, heads=24, kv_heads=24, d=128, dtype="bf16", layout="heads", train=False, lens="",
                 keep=1.0)
    rot = dict(op="rotary", B=1, heads=24, kv_heads=24, d=128, dtype="bf16", pairing="adjacent", train=False, t0=0)
    return [
        # the 27,280-token video grid reading a 512-token prompt: one sampler step of one layer
        dict(cross, name="cross_27280x512", n=27280, m=512),
        # the long video, a guidance pair: a prompt and a much shorter negative prompt in one padded
        # batch, straight from token-major projections
        dict(cross, name="cross_53680x512_pair", B=2, n=53680, m=512, lens="512,126", layout="tokens"),
        # a small latent image with a short caption: latency
        dict(cross, name="cross_2048x77", heads=8, kv_heads=8, n=2048, m=77),
        # one pooling query over every token of a video (the single-token form, split over the keys)
        dict(cross, name="cross_1x27280", n=1, m=27280),
        # resampler-like odd sizes: grouped key heads, d = 64, a mask with holes
        dict(cross, name="cross_gqa_4093x1111", B=2, heads=16, kv_heads=4, d=64, n=4093, m=1111, keep=0.7),
        # fp32, as checks and small models run it
        dict(cross, name="cross_f32_256x77", heads=2, kv_heads=2, d=64, dtype="f32", n=256, m=77),
        # fine-tuning: forward and backward of one layer at the video size
        dict(cross, name="cross_train_27280x512", n=27280, m=512, train=True),
        # fine-tuning on small clips, a padded caption batch (one of them empty: dropped for guidance)
        dict(cross, name="cross_train_2048x226", B=4, heads=8, kv_heads=8, n=2048, m=226, lens="226,61,0,130",
             layout="tokens", train=True),
        dict(cross, name="cross_train_f32_1000x130", heads=4, kv_heads=2, d=96, dtype="f32", n=1000, m=130, train=True),
        # q and k of the 27,280-token grid, token-major projections to the attention's layout
        dict(rot, name="rotary_27280", T=31, H=22, W=40),
        # the same in training, two clips
        dict(rot, name="rotary_train_27280", B=2, T=31, H=22, W=40, train=True),
        # one new latent frame of a stream, fp32, half-split pairs: latency
        dict(rot, name="rotary_frame_f32", heads=8, kv_heads=4, d=64, dtype="f32", pairing="half", T=1, H=22, W=40,
             t0=30),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    if rng.random() < 0.3:
        dtype = rng.choice(["bf16", "bf16", "f32"])
        heads = rng.choice([2, 8, 24] if dtype == "bf16" else [2, 8])
        return dict(op="rotary", B=rng.choice([1, 2]), heads=heads, kv_heads=rng.choice([heads, heads // 2]),
                    d=rng.choice([64, 128]), dtype=dtype, pairing=rng.choice(["adjacent", "half"]),
                    train=rng.random() < 0.4, t0=rng.choice([0, 0, rng.randint(1, 500)]),
                    T=_log_int(rng, 1, 31), H=rng.randint(4, 22), W=rng.randint(4, 40))
    f32 = rng.random() < 0.25
    train = rng.random() < 0.45
    B, heads = rng.choice([1, 2, 3]), rng.choice([2, 8] if f32 else [8, 16, 24])
    n = _log_int(rng, 1, 4096 if f32 else min(53680, (24 if train else 48) * 53680 // (B * heads)))
    most = (1 << 25 if f32 else (330_000_000 if train else 900_000_000)) // (B * heads * n)
    # with one key left everywhere the gradients of q and k are zero, and rounding noise is all there is to
    # compare: a training step has two keys at least in its first batch row
    least = 2 if train else 1
    m = _log_int(rng, least, max(least, min(1024 if f32 else 27280, most)))
    lens, keep = "", 1.0
    kind = rng.random()
    if kind < 0.3:
        lens = ",".join(str(m if train and b == 0 else rng.choice([m, rng.randint(0, m), rng.randint(1, m)]))
                        for b in range(B))
    elif kind < 0.5 and m >= 16:
        keep = round(rng.uniform(0.3, 0.95), 2)
    return dict(op="cross", B=B, heads=heads, kv_heads=rng.choice([heads, heads, heads // 2]),
                d=rng.choice([32, 64, 96, 128] if f32 else [64, 128]), dtype="f32" if f32 else "bf16",
                layout=rng.choice(["heads", "tokens"]), train=train, n=n, m=m, lens=lens, keep=keep)


# ---------------------------------------------------------------------------------- inputs

def _rows(gen, B, h, n, d, dtype, layout):
    """[B, h, n, d], contiguous or a view of token-major [B, n, h, d] memory."""
    shape = (B, h, n, d) if layout == "heads" else (B, n, h, d)
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)
    return x if layout == "heads" else x.transpose(1, 2)


def _axes(d):
    """Channels of time, height and width: height and width take a third each, rounded down to pairs."""
    side = 2 * (d // 6)
    return d - 2 * side, side, side


def _angles(case):
    """[positions of every axis, one after the other][pairs of that axis] as flat 64-bit angles."""
    parts = []
    for size, c, first in zip((case["T"], case["H"], case["W"]), _axes(case["d"]), (case["t0"], 0, 0)):
        freq = 10000.0 ** (-torch.arange(0, c, 2, device="cuda", dtype=torch.float64) / c)
        pos = torch.arange(first, first + size, device="cuda", dtype=torch.float64)
        parts.append((pos[:, None] * freq).reshape(-1))
    return torch.cat(parts)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt, B, h, hk, d = _DT[case["dtype"]], case["B"], case["heads"], case["kv_heads"], case["d"]
    if case["op"] == "rotary":
        n = case["T"] * case["H"] * case["W"]
        s = dict(case=case, q=_rows(gen, B, h, n, d, dt, "tokens"), k=_rows(gen, B, hk, n, d, dt, "tokens"))
        a = _angles(case)
        s["table"] = torch.stack([a.cos(), a.sin()], 1).float().contiguous()  # kept beside the model's weights
        if case["train"]:
            s["dq"], s["dk"] = _rows(gen, B, h, n, d, dt, "heads"), _rows(gen, B, hk, n, d, dt, "heads")
        return s
    n, m = case["n"], case["m"]
    s = dict(case=case, q=_rows(gen, B, h, n, d, dt, case["layout"]), k=_rows(gen, B, hk, m, d, dt, case["layout"]),
             v=_rows(gen, B, hk, m, d, dt, case["layout"]), kv_lens=None, key_mask=None)
    if case["lens"]:
        s["kv_lens"] = torch.tensor([int(x) for x in case["lens"].split(",")], device="cuda", dtype=torch.int32)
    if case["keep"] < 1.0:
        s["key_mask"] = torch.rand((B, m), generator=gen, device="cuda") < case["keep"]
    if case["train"]:
        s["do"] = _rows(gen, B, h, n, d, dt, case["layout"])
    return s


# ---------------------------------------------------------------------------------- one pass

def run(s):
    if own:
        return _run_own(s)
    return _plain_rotary(s) if s["case"]["op"] == "rotary" else _plain_cross(s)


def _run_own(s):
    import sub_quadratic_two_b200 as sq
    case, train = s["case"], s["case"]["train"]
    if case["op"] == "rotary":
        rot = sq.Rotary(grid=(case["T"], case["H"], case["W"]), axes=_axes(case["d"]), table=s["table"],
                        pairing=case["pairing"])
        if not train:
            return sq.rotary(s["q"], s["k"], rot)
        q, k = (s[x].detach().requires_grad_() for x in "qk")
        yq, yk = sq.rotary(q, k, rot)
        return (yq.detach(), yk.detach()) + torch.autograd.grad((yq, yk), (q, k), (s["dq"], s["dk"]))
    opts = dict(kv_lens=s["kv_lens"], key_mask=s["key_mask"])
    if not train:
        return sq.cross_attention(s["q"], s["k"], s["v"], **opts)
    q, k, v = (s[x].detach().requires_grad_() for x in "qkv")
    o = sq.cross_attention(q, k, v, **opts)
    return (o.detach(),) + torch.autograd.grad(o, (q, k, v), s["do"])


def _kept(s):
    """[B, 1, 1, 1, m] truth values of the keys that count, or None."""
    if s["kv_lens"] is not None:
        keep = torch.arange(s["case"]["m"], device="cuda")[None] < s["kv_lens"][:, None]
    elif s["key_mask"] is not None:
        keep = s["key_mask"]
    else:
        return None
    return keep[:, None, None, None, :]


def _plain_cross(s):
    case = s["case"]
    B, h, hk, n, m, d = (case[x] for x in ("B", "heads", "kv_heads", "n", "m", "d"))
    dt, g, scale = _DT[case["dtype"]], h // hk, 1.0 / math.sqrt(d)
    q = s["q"].float().reshape(B, hk, g, n, d)
    k, v = s["k"].float()[:, :, None], s["v"].float()[:, :, None]
    keep = _kept(s)
    if keep is not None:  # what is masked may hold anything
        rows = keep.transpose(-1, -2)
        k, v = torch.where(rows, k, 0.0), torch.where(rows, v, 0.0)
    p = torch.matmul(q, k.transpose(-1, -2)).mul_(scale)
    if keep is not None:
        p.masked_fill_(~keep, -math.inf)
    top = p.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = p.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    p = p.div_(torch.where(total == 0, 1.0, total))
    o = torch.matmul(p, v)
    out = o.reshape(B, h, n, d).to(dt)
    if not case["train"]:
        return out
    do = s["do"].float().reshape(B, hk, g, n, d)
    dv = torch.matmul(p.transpose(-1, -2), do).sum(2)
    dp = torch.matmul(do, v.transpose(-1, -2)).sub_((do * o).sum(-1, keepdim=True))
    ds = dp.mul_(p).mul_(scale)
    dq = torch.matmul(ds, k).reshape(B, h, n, d)
    dk = torch.matmul(ds.transpose(-1, -2), q).sum(2)
    return out, dq.to(dt), dk.to(dt), dv.to(dt)


def _token_angles(case, table):
    """cos and sin [n, pairs] of every token of the grid, in token order, from the flat table."""
    T, H, W = case["T"], case["H"], case["W"]
    pt, ph, pw = (c // 2 for c in _axes(case["d"]))
    a, b = T * pt, T * pt + H * ph
    parts = (table[:a].reshape(T, 1, 1, pt, 2).expand(T, H, W, pt, 2),
             table[a:b].reshape(1, H, 1, ph, 2).expand(T, H, W, ph, 2),
             table[b:].reshape(1, 1, W, pw, 2).expand(T, H, W, pw, 2))
    both = torch.cat(parts, 3).reshape(T * H * W, pt + ph + pw, 2)
    return both[..., 0], both[..., 1]


def _turn(x, cos, sin, pairing, dt):
    x = x.float()
    B, h, n, d = x.shape
    if pairing == "adjacent":
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - b * sin, a * sin + b * cos], -1).reshape(B, h, n, d).to(dt)
    a, b = x[..., : d // 2], x[..., d // 2:]
    return torch.cat([a * cos - b * sin, a * sin + b * cos], -1).to(dt)


def _plain_rotary(s):
    case = s["case"]
    dt = _DT[case["dtype"]]
    cos, sin = _token_angles(case, s["table"])
    out = tuple(_turn(s[x], cos, sin, case["pairing"], dt) for x in "qk")
    if not case["train"]:
        return out
    return out + tuple(_turn(s[x], cos, -sin, case["pairing"], dt) for x in ("dq", "dk"))


# ---------------------------------------------------------------------------------- cost

def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    B, h, hk, d = case["B"], case["heads"], case["kv_heads"], case["d"]
    if case["op"] == "rotary":
        el = B * (h + hk) * case["T"] * case["H"] * case["W"] * d * (2 if case["train"] else 1)
        return {"bytes": 2 * el * e, "flops": 3 * el}
    n, m = case["n"], case["m"]
    if case["lens"]:
        kept = sum(int(x) for x in case["lens"].split(","))
    else:
        kept = B * m * case["keep"]
    flops = 4 * h * n * kept * d
    el = 2 * B * h * n * d + 2 * hk * kept * d
    if case["train"]:  # the output and its gradient once more, dq, dk and dv; five more products
        flops += 10 * h * n * kept * d
        el += 2 * B * h * n * d + 2 * B * hk * m * d
    return {"bytes": int(el * e), "flops": int(flops)}


# ---------------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotary":
        return _exact_rotary(case, s)
    B, h, hk, n, m = (case[x] for x in ("B", "heads", "kv_heads", "n", "m"))
    per, scale, train = h // hk, case["d"] ** -0.5, case["train"]
    outs, dqs = torch.zeros((B, h, n, case["d"]), device="cuda", dtype=torch.float64), None
    if train:
        dqs = torch.zeros_like(outs)
        dks, dvs = (torch.zeros((B, hk, m, case["d"]), device="cuda", dtype=torch.float64) for _ in "kv")
    for b in range(B):
        if s["kv_lens"] is not None:
            rows = torch.arange(int(s["kv_lens"][b]), device="cuda")
        elif s["key_mask"] is not None:
            rows = s["key_mask"][b].nonzero()[:, 0]
        else:
            rows = torch.arange(m, device="cuda")
        if not len(rows):
            continue
        for i in range(h):
            q, k, v = (s["q"][b, i].double(), s["k"][b, i // per][rows].double(), s["v"][b, i // per][rows].double())
            if not train:
                outs[b, i] = torch.exp(q @ k.T * scale - torch.logsumexp(q @ k.T * scale, 1, True)) @ v
                continue
            q, k, v = (x.requires_grad_() for x in (q, k, v))
            o = torch.softmax(torch.einsum("nd,md->nm", q, k) * scale, 1) @ v
            gq, gk, gv = torch.autograd.grad(o, (q, k, v), s["do"][b, i].double())
            outs[b, i], dqs[b, i] = o.detach(), gq
            dks[b, i // per, rows] += gk
            dvs[b, i // per, rows] += gv
    return (outs, dqs, dks, dvs) if train else outs


def _exact_rotary(case, s):
    """The pairs as complex numbers, multiplied by exp(i angle) (its conjugate for the gradients)."""
    T, H, W, d = case["T"], case["H"], case["W"], case["d"]
    tok = torch.arange(T * H * W, device="cuda")
    pos = (case["t0"] + tok // (H * W), tok // W % H, tok % W)
    ang = []
    for p, c in zip(pos, _axes(d)):
        i = torch.arange(c // 2, device="cuda", dtype=torch.float64)
        ang.append(p.double()[:, None] / torch.pow(torch.tensor(10000.0, dtype=torch.float64, device="cuda"), 2 * i / c))
    w = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), torch.cat(ang, 1))

    def turn(x, by):
        x = x.double()
        if case["pairing"] == "adjacent":
            z = torch.view_as_complex(x.reshape(*x.shape[:-1], d // 2, 2).contiguous()) * by
            return torch.view_as_real(z).reshape(x.shape)
        z = torch.complex(x[..., : d // 2].contiguous(), x[..., d // 2:].contiguous()) * by
        return torch.cat([z.real, z.imag], -1)

    out = (turn(s["q"], w), turn(s["k"], w))
    if case["train"]:
        out += (turn(s["dq"], w.conj()), turn(s["dk"], w.conj()))
    return out
