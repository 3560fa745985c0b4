"""rope_rotate and kv_append against the formula in 64 bits."""
import math

import pytest
import torch

from moe_expert_gemv_b200 import qmoe
from tests._attn import HALF_STEP, Case

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


def turned(x, pos, freq, scale, layout):
    """64-bit: pairs as complex numbers, turned."""
    half = freq.numel()
    y = x.double().clone()
    turn = torch.polar(torch.full_like(freq, scale).expand(len(pos), half).contiguous(), torch.outer(pos.double(), freq))[:, None]
    if layout == "half":
        z = torch.complex(y[..., :half], y[..., half:2 * half]) * turn
        y[..., :half], y[..., half:2 * half] = z.real, z.imag
    else:
        z = torch.complex(y[..., 0:2 * half:2], y[..., 1:2 * half:2]) * turn
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = z.real, z.imag
    return y


def close(got, want, x, half, dtype, scale=1.0):
    """Half a step of the result; before that two fp32 products and a sum (3
    2^-24) with a sine and cosine off by at most 2^-21 (2^-23 from rounding the
    reduced angle, up to pi, to fp32; 2 units in the last place from sincosf),
    all relative to scale * (|a| + |b|) <= 2 scale max|x|; fp16's smallest step."""
    tol = HALF_STEP[dtype] * want.abs() + 2.0 ** -20 * 2 * abs(scale) * x.double().abs().amax() + 2.0 ** -25
    d = (got.double() - want).abs()
    assert (d <= tol).all(), "error %.3g times the bound" % (d / tol).max()
    assert torch.equal(got[..., 2 * half:], x[..., 2 * half:])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dim,rot", [(128, 128), (64, 32), (256, 64), (80, 20), (96, 96), (7, 4), (2, 2), (72, 48), (1024, 1024)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_rotate(cuda_dev, layout, dim, rot, dtype):
    x = torch.randn(9, 5, dim, device="cuda").to(dtype)
    pos = torch.tensor([0, 1, 2, 77, 4095, 131071, 1000003, 2 ** 31 - 1, -5], dtype=torch.int32, device="cuda")
    r = qmoe.Rope.make(rot, layout)
    f, _ = qmoe.rope_frequencies(rot)
    y = qmoe.rope_rotate(r, x, pos)
    close(y, turned(x, pos, f.cuda(), 1.0, layout), x, rot // 2, dtype)
    z = x.clone()
    assert qmoe.rope_rotate(r, z, pos, out=z) is z and torch.equal(z, y)
    # strided, and 2-byte aligned only
    wide = torch.zeros(9, 7, dim + 3, dtype=dtype, device="cuda")
    wide[:, 1:6, 1:dim + 1] = x
    out = torch.full((5, 9, dim + 1), 9.0, dtype=dtype, device="cuda")
    qmoe.rope_rotate(r, wide[:, 1:6, 1:dim + 1], pos, out=out.transpose(0, 1)[..., 1:])
    assert torch.equal(out.transpose(0, 1)[..., 1:], y) and (out[..., 0] == 9).all()
    assert qmoe.qmoe_check_status() == 0


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_transpose_is_the_gradient(cuda_dev, layout):
    """<R x, g> = <x, R(-p) g>, and the difference quotient of the (linear) rotation."""
    x, g = (torch.randn(6, 3, 64, device="cuda").half() for _ in range(2))
    pos = torch.arange(6, dtype=torch.int32, device="cuda") * 1000
    r = qmoe.Rope(qmoe.rope_frequencies(48)[0].cuda(), layout, 1.25)
    y, gx = qmoe.rope_rotate(r, x, pos), qmoe.rope_rotate(r, g, -pos)
    f = r.inv_freq
    close(gx, turned(g, -pos, f, 1.25, layout), g, 24, F16, 1.25)
    a, b = (y.double() * g.double()).sum(), (x.double() * gx.double()).sum()
    # each of the 1152 products off by half a step of its rotated factor
    assert (a - b).abs() <= 2 * 2.0 ** -11 * 1.25 * 1.5 * (x.double().norm() * g.double().norm())
    h = torch.zeros_like(x)
    h[2, 1, 5] = 1.0
    d = turned(x.double() + h.double(), pos, f, 1.25, layout) - turned(x, pos, f, 1.25, layout)
    assert ((d * g.double()).sum() - gx[2, 1, 5].double()).abs() <= 2.0 ** -11 * 4


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("layout,dim,rot,page,head_major", [("half", 128, 128, 16, False), ("interleaved", 256, 64, 32, True),
                                                           ("half", 80, 20, 7, False), ("half", 64, 64, 1, True)])
@pytest.mark.parametrize("lens", [[(1, 5), (1, 17), (1, 64)], [(40, 40), (0, 9), (7, 100), (1, 1)]], ids=["decode", "chunks"])
def test_append(cuda_dev, dtype, layout, dim, rot, page, head_major, lens):
    c = Case(lens, 6, 2, dim, page, dtype, head_major=head_major, spare=2)
    T = c.tokens + 2
    f, s = qmoe.rope_frequencies(rot, base=5e5, kind="ramp", factor=8.0, trained=4096, low=1.0, high=32.0)
    r = qmoe.Rope(f.cuda(), layout, s)
    qkv = torch.randn(T, 10 * dim, device="cuda").to(dtype)
    q, k, v = (t.unflatten(1, (-1, dim)) for t in qkv.split([6 * dim, 2 * dim, 2 * dim], 1))
    k0, v0 = c.k.clone(), c.v.clone()
    q_out = torch.full((T, 6, dim), 9.0, dtype=dtype, device="cuda")
    qmoe.kv_append(c.cache, c.batch(), k, v, q=q, rope=r, q_out=q_out)
    assert qmoe.qmoe_check_status() == 0
    pos = torch.cat([torch.arange(kv - n, kv) for n, kv in lens]).cuda()
    n = c.tokens
    close(q_out[:n], turned(q[:n], pos, f.cuda(), s, layout), q[:n], rot // 2, dtype, s)
    assert (q_out[n:] == 9).all()
    kt = turned(k[:n], pos, f.cuda(), s, layout)
    at = 0
    for (m, kv), (pg, sl) in zip(lens, c.slots):
        if m:
            pg, sl = pg[kv - m:], sl[kv - m:]
            close(c.k[pg, sl], kt[at:at + m], k[at:at + m], rot // 2, dtype, s)
            assert torch.equal(c.v[pg, sl], v[at:at + m])
            c.k[pg, sl], c.v[pg, sl] = k0[pg, sl], v0[pg, sl]
        at += m
    # no other slot was written
    assert torch.equal(c.k.view(torch.int16), k0.view(torch.int16)) and torch.equal(c.v.view(torch.int16), v0.view(torch.int16))


def test_append_without_rotation_or_queries(cuda_dev):
    c = Case([(3, 20), (1, 8)], 4, 2, 64, 16)
    k, v = torch.randn(4, 2, 64, device="cuda").half(), torch.randn(4, 2, 64, device="cuda").half()
    assert qmoe.kv_append(c.cache, c.batch(), k, v) is None
    pg, sl = c.slots[0]
    assert torch.equal(c.k[pg[17:], sl[17:]], k[:3]) and torch.equal(c.v[pg[17:], sl[17:]], v[:3])
    r = qmoe.Rope.make(64)
    pos = torch.tensor([9, 9, 9, 9], dtype=torch.int32, device="cuda")
    qmoe.kv_append(c.cache, c.batch(), k, v, rope=r, positions=pos)
    want = qmoe.rope_rotate(r, k, pos)
    assert torch.equal(c.k[pg[17:], sl[17:]], want[:3])
    assert qmoe.qmoe_check_status() == 0


def test_append_bad_places_are_flagged_and_not_stored(cuda_dev):
    c = Case([(2, 40), (3, 1), (1, 16)], 4, 2, 64, 16)
    c.table[0, 2] = -1            # the page of both new tokens of sequence 0
    c.kv_len[2] = 49              # behind the table's 3 pages
    k = torch.randn(6, 2, 64, device="cuda").half()
    k0 = c.k.clone()
    r = qmoe.Rope.make(64)
    q = torch.randn(6, 4, 64, device="cuda").half()
    y = qmoe.kv_append(c.cache, c.batch(), k, k, q=q, rope=r)
    assert qmoe.qmoe_check_status() == qmoe.DEV_BAD_PAGE
    pos = torch.tensor([38, 39, -2, -1, 0, 48], dtype=torch.int32, device="cuda")
    assert torch.equal(y, qmoe.rope_rotate(r, q, pos))   # the queries are turned all the same
    pg, sl = c.slots[1]
    assert torch.equal(c.v[pg, sl][0], k[4])
    c.k[pg, sl] = k0[pg, sl]
    assert torch.equal(c.k.view(torch.int16), k0.view(torch.int16))


def test_python_refusals(cuda_dev):
    c = Case([(1, 5)], 4, 2, 64, 16)
    k = torch.zeros(1, 2, 64, dtype=F16, device="cuda")
    with pytest.raises(ValueError):
        qmoe.kv_append(c.cache, c.batch(), k, k, q=c.q)
    with pytest.raises(ValueError):
        qmoe.kv_append(c.cache, c.batch(), k[:, :1], k)
    with pytest.raises(TypeError):
        qmoe.kv_append(c.cache, c.batch(), k.float(), k)
    with pytest.raises(qmoe.QmoeError):
        qmoe.kv_append(c.cache, c.batch(), k, k, rope=qmoe.Rope.make(66))
    with pytest.raises(TypeError):
        qmoe.rope_rotate(qmoe.Rope.make(64), k, torch.zeros(1, dtype=torch.int64, device="cuda"))


def test_append_many_sequences_in_place(cuda_dev):
    """More sequences than two steps of a warp's search tell apart, some without new tokens; q turned where it lies."""
    g = torch.Generator().manual_seed(2)
    n = torch.randint(0, 3, (1300,), generator=g)
    kv = n + torch.randint(0, 20, (1300,), generator=g)
    n[0] = kv[0] = 0
    c = Case(list(zip(n.tolist(), kv.tolist())), 4, 1, 64, 8, seed=5)
    T = c.tokens
    r = qmoe.Rope.make(64)
    q, k = torch.randn(T, 4, 64, device="cuda").half(), torch.randn(T, 1, 64, device="cuda").half()
    pos = torch.cat([torch.arange(b - a, b) for a, b in c.lens]).int().cuda()
    want_q, want_k = qmoe.rope_rotate(r, q, pos), qmoe.rope_rotate(r, k, pos)
    y = q.clone()
    assert qmoe.kv_append(c.cache, c.batch(), k, k, q=y, rope=r, q_out=y) is y
    assert qmoe.qmoe_check_status() == 0 and torch.equal(y, want_q)
    pg = torch.cat([s[0][b - a:] for (a, b), s in zip(c.lens, c.slots)])
    sl = torch.cat([s[1][b - a:] for (a, b), s in zip(c.lens, c.slots)])
    assert torch.equal(c.k[pg, sl], want_k) and torch.equal(c.v[pg, sl], k)
