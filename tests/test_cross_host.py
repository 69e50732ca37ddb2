"""Host-side refusals of the cross-attention and rotary entry points (no GPU: nothing is launched)."""
import ctypes

import pytest
import torch

import sub_quadratic_two_b200 as sq
from sub_quadratic_two_b200.cross import SquadCrossDesc
from sub_quadratic_two_b200.positions import SquadRotaryDesc, SquadStrides, default_axes

OK, INVALID, SHAPE, ALIGN, UNSUPPORTED, CUDA, TIMEOUT, WORKSPACE = range(8)
FAKE, MISALIGNED = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10008)


@pytest.fixture(scope="module")
def lib():
    return sq.load_library()


def dense(B, h, n, d):
    return SquadStrides(h * n * d, n * d, d)


def cross_desc(**kw):
    c = dict(B=2, heads=4, kv_heads=2, n=10, m=20, d=64, dtype=sq.SQUAD_BF16, scale=0.0, mask_stride=0)
    over = {k: kw.pop(k) for k in list(kw) if k in ("q", "k", "v", "o", "dout", "dq", "dk", "dv")}
    c.update(kw)
    desc = SquadCrossDesc(*[c[f] for f in ("B", "heads", "kv_heads", "n", "m", "d", "dtype", "scale", "mask_stride")])
    for name in ("q", "o", "dout", "dq"):
        setattr(desc, name, over.get(name, dense(c["B"], c["heads"], c["n"], c["d"])))
    for name in ("k", "v", "dk", "dv"):
        setattr(desc, name, over.get(name, dense(c["B"], c["kv_heads"], c["m"], c["d"])))
    return desc


def fwd(lib, desc, q=FAKE, k=FAKE, v=FAKE, lens=None, mask=None, o=FAKE, lse=None, ws=None, nb=0):
    return lib.squad_cross_fwd(ctypes.byref(desc) if desc else None, q, k, v, lens, mask, o, lse, ws, nb, None)


def bwd(lib, desc, o=FAKE, lse=FAKE, dout=FAKE, dq=FAKE, dk=FAKE, dv=FAKE, ws=FAKE, nb=1 << 30, mask=None):
    return lib.squad_cross_bwd(ctypes.byref(desc), FAKE, FAKE, FAKE, None, mask, o, lse, dout, dq, dk, dv, ws, nb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), SHAPE), (dict(n=0), SHAPE), (dict(m=-1), SHAPE), (dict(kv_heads=3), SHAPE), (dict(kv_heads=0), SHAPE),
    (dict(dtype=5), INVALID), (dict(scale=float("nan")), INVALID), (dict(d=96), UNSUPPORTED),
    (dict(dtype=sq.SQUAD_F32, d=48), UNSUPPORTED), (dict(dtype=sq.SQUAD_F32, d=288), UNSUPPORTED),
    (dict(B=70000, heads=1, kv_heads=1), UNSUPPORTED), (dict(heads=1 << 16, kv_heads=1, n=1 << 15), SHAPE),
    (dict(q=SquadStrides(4 * 10 * 64, 10 * 64, 32)), ALIGN),       # rows overlap
    (dict(q=SquadStrides(4 * 10 * 68, 10 * 68, 68)), ALIGN),       # rows 136 bytes apart
    (dict(k=SquadStrides(-8, 20 * 64, 64)), ALIGN),
    (dict(o=SquadStrides(0, 10 * 64, 64)), ALIGN),                 # an output may not be broadcast
    (dict(o=SquadStrides(4 * 10 * 64, 64, 64)), ALIGN),            # nor may its heads overlap
    (dict(o=SquadStrides(64, 64, 8 * 64)), ALIGN),                 # nor its batch rows
    (dict(o=SquadStrides(3 * 10 * 64, 10 * 64, 64)), ALIGN),
    (dict(q=SquadStrides(4 * 10 * 64, 10 * 64, 0)), ALIGN),
])
def test_descriptor_errors(lib, kw, code):
    assert fwd(lib, cross_desc(**kw)) == code


def test_gradient_strides_are_checked(lib):
    for name in ("dq", "dk", "dv"):
        assert bwd(lib, cross_desc(**{name: SquadStrides(1 << 20, 0, 64)})) == ALIGN
    assert bwd(lib, cross_desc(dout=SquadStrides(1 << 20, 1 << 16, 4))) == ALIGN


def test_pointer_errors(lib):
    d = cross_desc()
    assert fwd(lib, None) == INVALID
    assert fwd(lib, d, q=None) == INVALID and fwd(lib, d, o=None) == INVALID
    assert fwd(lib, d, k=MISALIGNED) == ALIGN and fwd(lib, d, lse=MISALIGNED) == ALIGN
    assert fwd(lib, d, lens=ctypes.c_void_p(0x10002)) == ALIGN
    assert fwd(lib, cross_desc(mask_stride=19), mask=FAKE) == INVALID
    assert bwd(lib, d, lse=None) == INVALID and bwd(lib, d, dv=MISALIGNED) == ALIGN
    assert bwd(lib, d, ws=None) == WORKSPACE and bwd(lib, d, nb=16) == WORKSPACE
    assert bwd(lib, cross_desc(mask_stride=19), mask=FAKE) == INVALID


def test_workspace_size(lib):
    nb = ctypes.c_size_t(0)
    size = lambda which, **kw: (lib.squad_cross_workspace_size(ctypes.byref(cross_desc(**kw)), which, ctypes.byref(nb)),  # noqa: E731
                                nb.value)
    assert size(2)[0] == INVALID and lib.squad_cross_workspace_size(None, 0, ctypes.byref(nb)) == INVALID
    code, b = size(1)
    assert code == OK and b >= 2 * 4 * 10 * 4
    # never more than the tensors themselves by far, over a range of shapes
    for n in (1, 77, 2048, 53680):
        for m in (1, 77, 512, 27280):
            for which in (0, 1):
                code, b = size(which, B=1, heads=24, kv_heads=24, d=128, n=n, m=m)
                assert code == OK and b <= (1 << 20) + 64 * 24 * 128 * 4 * (n + 2 * m)


def rotary(lib, x=FAKE, y=FAKE, heads=2, xs=None, ys=None, table=FAKE, nt=1, **kw):
    c = dict(B=1, d=64, T=2, H=3, W=4, cT=24, cH=20, cW=20, dtype=sq.SQUAD_BF16, pairing=0, inverse=0)
    c.update(kw)
    desc = SquadRotaryDesc(*[c[f] for f, _ in SquadRotaryDesc._fields_])
    s = dense(c["B"], max(heads, 1), 24, c["d"])
    return lib.squad_rotary(ctypes.byref(desc), nt, (ctypes.c_int * 1)(heads), (ctypes.c_void_p * 1)(x),
                            (SquadStrides * 1)(xs or s), (ctypes.c_void_p * 1)(y), (SquadStrides * 1)(ys or s), table, None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=0), SHAPE), (dict(cT=23), SHAPE), (dict(cT=-2), SHAPE), (dict(cT=32), SHAPE), (dict(heads=0), SHAPE),
    (dict(dtype=3), INVALID), (dict(pairing=2), INVALID), (dict(table=None), INVALID), (dict(nt=0), INVALID),
    (dict(nt=3), INVALID), (dict(d=68), UNSUPPORTED), (dict(d=2048), UNSUPPORTED),
    (dict(pairing=1, cT=20), UNSUPPORTED), (dict(B=70000), UNSUPPORTED), (dict(T=1 << 15, H=1 << 10, W=1 << 10), SHAPE),
    (dict(xs=SquadStrides(1, 64, 4)), ALIGN), (dict(ys=SquadStrides(64, 0, 64)), ALIGN),
    (dict(table=ctypes.c_void_p(0x10004)), ALIGN),
])
def test_rotary_errors(lib, kw, code):
    assert rotary(lib, **kw) == code


def test_rotary_pointer_errors(lib):
    assert rotary(lib, x=0x10008) == ALIGN and rotary(lib, y=0x10008) == ALIGN
    assert rotary(lib, x=None) == INVALID and rotary(lib, y=None) == INVALID


def test_rotary_plan_table():
    # every entry of the table is the cos and sin of its axis' position and frequency
    rot = sq.rotary_plan((2, 3, 4), 64, (24, 20, 20), theta=100.0, offset=(5, 0, 1), device="cpu")
    at = 0
    for size, c, first in zip((2, 3, 4), (24, 20, 20), (5, 0, 1)):
        for p in range(size):
            for i in range(c // 2):
                a = torch.tensor((first + p) * 100.0 ** (-2 * i / c), dtype=torch.float64)
                assert abs(rot.table[at, 0].item() - a.cos().item()) <= 2.0 ** -24
                assert abs(rot.table[at, 1].item() - a.sin().item()) <= 2.0 ** -24
                at += 1
    assert at == rot.table.shape[0]
    for d in range(2, 200, 2):
        axes = default_axes(d)
        assert sum(axes) == d and all(c % 2 == 0 and c >= 0 for c in axes)


def test_rotary_plan_refusals():
    t = torch.zeros(2 * 12 + 3 * 10 + 4 * 10, 2)
    sq.Rotary((2, 3, 4), (24, 20, 20), t)
    for bad in (dict(axes=(23, 20, 20)), dict(axes=(24, 20)), dict(grid=(0, 3, 4)), dict(table=t[:-1]),
                dict(table=t.double()), dict(pairing="pairs"), dict(table=t.t().contiguous().t()), dict(axes=(-2, 46, 20))):
        with pytest.raises(ValueError):
            sq.Rotary(**{**dict(grid=(2, 3, 4), axes=(24, 20, 20), table=t), **bad})
    with pytest.raises(ValueError):
        sq.rotary_plan((2, 3, 4), 32, (24, 20, 20), device="cpu")
    with pytest.raises(ValueError):
        sq.rotary_plan((2, 3, 4), 64, offset=(1, 2), device="cpu")
    with pytest.raises(ValueError):
        sq.squad_rotary([torch.zeros(1, 1, 24, 64)], sq.Rotary((2, 3, 4), (24, 20, 20), t))  # host tensors
    with pytest.raises(ValueError):
        sq.cross_attention(*[torch.zeros(1, 1, 4, 64)] * 3)


def test_a_rotary_table_is_a_constant():
    t = torch.zeros(2 * 12 + 3 * 10 + 4 * 10, 2, requires_grad=True)
    x = torch.zeros(1, 1, 24, 64)
    with pytest.raises(ValueError, match="constant"):
        sq.rotary(x, None, sq.Rotary((2, 3, 4), (24, 20, 20), t))
    fw = torch.autograd.forward_ad
    with fw.dual_level(), pytest.raises(ValueError, match="constant"):
        sq.rotary(x, None, sq.Rotary((2, 3, 4), (24, 20, 20), fw.make_dual(t.detach(), torch.ones(t.shape))))


def test_a_stream_of_another_device_is_refused():
    from types import SimpleNamespace
    other = SimpleNamespace(device=torch.device("cuda", 1))
    x = torch.zeros(1, 1, 24, 64)
    with pytest.raises(ValueError, match="stream"):
        sq.squad_cross_fwd(x, x, x, stream=other)
    with pytest.raises(ValueError, match="stream"):
        sq.squad_cross_bwd(x, x, x, x, x[..., 0], x, stream=other)
    t = torch.zeros(2 * 12 + 3 * 10 + 4 * 10, 2)
    with pytest.raises(ValueError, match="stream"):
        sq.squad_rotary([x], sq.Rotary((2, 3, 4), (24, 20, 20), t), stream=other)


def test_rotary_plans_compare_and_are_kept_in_sets():
    a, b = (sq.rotary_plan((1, 2, 3), 64, device="cpu") for _ in range(2))
    assert a == a and a != b and b in [a, b] and {a: 1, b: 2}[b] == 2


def test_outputs_that_begin_at_another_tensor_are_refused(lib):
    # every call here has such an output: nothing is launched
    at = lambda i: ctypes.c_void_p(0x10000 * i)  # noqa: E731
    d = cross_desc()
    for same in (1, 2, 3):
        assert fwd(lib, d, q=at(1), k=at(2), v=at(3), o=at(same)) == INVALID
    names = ("o", "dout", "dq", "dk", "dv")
    for a, b in (("dq", "o"), ("dk", "dout"), ("dv", "dq"), ("dk", "dq"), ("dv", "dk")):
        p = {x: at(4 + i) for i, x in enumerate(names)}
        p[a] = p[b]
        assert bwd(lib, d, lse=at(2), **p) == INVALID
    assert bwd(lib, d, o=at(4), dout=at(5), dq=at(6), dk=FAKE, dv=at(7)) == INVALID  # dk over k

    def two(x, y, ys=None):
        s = dense(1, 2, 24, 64)
        desc = SquadRotaryDesc(1, 64, 2, 3, 4, 24, 20, 20, sq.SQUAD_BF16, 0, 0)
        return lib.squad_rotary(ctypes.byref(desc), 2, (ctypes.c_int * 2)(2, 2), (ctypes.c_void_p * 2)(*x),
                                (SquadStrides * 2)(s, s), (ctypes.c_void_p * 2)(*y), (SquadStrides * 2)(ys or s, s),
                                FAKE, None)

    a, b, c = 0x20000, 0x30000, 0x40000
    assert two((a, b), (b, a)) == INVALID and two((a, b), (c, c)) == INVALID and two((a, a), (a, a)) == INVALID
    assert two((a, b), (a, c), dense(1, 3, 30, 64)) == INVALID  # in place with other strides
