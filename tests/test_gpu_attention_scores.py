"""attn_paged's scores over the whole range of the tanh cap, against 64 bits
with a bound that goes by the score and not by the cap."""
import math

import pytest
import torch

from moe_expert_gemv_b200 import qmoe
from tests._attn import HALF_STEP, Case

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


def bound(c, scale, cap, lost):
    """(out, bound of its error), 64-bit, causal.

    The bound, with u half a step of the type: the output's rounding u |o|; the
    weights' u sum p |v|, and `lost` of the row's largest weight for each that
    is too small for the type; a score's error e shifts p and the sum by e
    each: a fp32 dot product of dim terms, its scaling and the exponential's
    argument, (dim + 8) 2^-24 of the sum of |q k| scaled, 2^-21 absolute for
    the exponential, and for a cap 2^-19 of the score: below cap / 2 the
    polynomial's 2^-23 and 8 roundings of 2^-24; above it tanh = 1 - 2 / (1 + E)
    from E = e^2z with 2^-22 of its own and 2^-23 of its argument, which the
    slope 2 E / (1 + E)^2 <= 0.4 takes to 0.8 2^-22, a quotient good to 2^-22 of
    at most 0.54 and two roundings, all of it over tanh >= 0.46; fp32 sums of
    n terms, truncated by the tensor cores: (n + 64) 2^-23 of sum p |v|."""
    u, out, tol, at = HALF_STEP[c.dtype], [], [], 0
    for (n, kv), k, v in zip(c.lens, c.keys, c.values):
        q = c.q[at:at + n].double().transpose(0, 1)
        at += n
        grp = c.heads // c.kv_heads
        k = k.double().repeat_interleave(grp, 1).permute(1, 2, 0)
        v = v.double().repeat_interleave(grp, 1).transpose(0, 1)
        s = q @ k * scale
        e = (c.dim + 8) * 2.0 ** -24 * (q.abs() @ k.abs() * scale).amax(-1, keepdim=True) + 2.0 ** -21
        if cap:
            s = cap * torch.tanh(s / cap)
            e = e + 2.0 ** -19 * s.abs().amax(-1, keepdim=True)
        p = (kv - n + torch.arange(n, device=q.device))[:, None]
        w = torch.softmax(s.masked_fill(torch.arange(kv, device=q.device)[None] > p, -math.inf), -1)
        o, a = w @ v, w @ v.abs()
        t = u * o.abs() + (u + 2 * e + (kv + 64) * 2.0 ** -23) * a + lost * kv * v.abs().amax() * w.amax(-1, keepdim=True) + 2.0 ** -25
        out.append(o.transpose(0, 1))
        tol.append(t.transpose(0, 1))
    return torch.cat(out), torch.cat(tol)


def check(c, got, scale, cap, lost):
    o, tol = bound(c, scale, cap, lost)
    over = (got[:c.tokens].double() - o).abs() / tol
    assert over.max() <= 1, "error %.2f times the bound" % over.max()


# decode, drafts, and rows enough for two row tiles in a unit
LENS = [([(1, 1), (1, 300), (1, 700)], 8, 2, 1), ([(5, 130), (24, 700), (1, 64)], 8, 2, 24), ([(300, 400), (300, 310), (1, 33)], 64, 8, 300)]


@pytest.mark.parametrize("cap", [0.25, 7.0, 50.0, 1e3, 1e5, 1e8, 1e30, 3e38])
@pytest.mark.parametrize("dim,page", [(64, 16), (128, 7), (256, 32)])
@pytest.mark.parametrize("lens,heads,kv_heads,new", LENS, ids=["decode", "drafts", "chunks"])
def test_caps_of_any_size(cuda_dev, lens, heads, kv_heads, new, dim, page, cap):
    c = Case(lens, heads, kv_heads, dim, page, F16, seed=dim)
    scale = dim ** -0.5
    out = qmoe.attn_paged(c.cache, c.batch(new), c.q, softcap=cap)
    assert qmoe.qmoe_check_status() == 0
    check(c, out, scale, cap, 2.0 ** -25)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("dim,page", [(64, 16), (128, 7), (256, 32)])
@pytest.mark.parametrize("lens,heads,kv_heads,new", [([(1, 8192), (1, 4097)], 8, 2, 1), ([(20, 8192), (24, 5000)], 8, 2, 24),
                                                     ([(600, 4300), (600, 700)], 64, 8, 600)], ids=["decode", "drafts", "chunks"])
def test_many_small_weights(cuda_dev, lens, heads, kv_heads, new, dim, page, dtype):
    """64 keys of every 4096 have a score of 25.2 log 2 and the value 0, the others
    score 0 and have the value 1000: their weights, 2^-25.2 of the largest, are
    all of the output, and a weight that is lost is seen.  At most 2^-32 of the
    largest each is: half the smallest fp16 step over the 2^7 that the largest
    is lifted to (it may be up to 2^8 larger, which only helps)."""
    c = Case(lens, heads, kv_heads, dim, page, dtype, seed=1)
    c.q.zero_()
    c.q[..., 0] = 16.0
    for k, v in zip(c.keys, c.values):
        k.zero_()
        v.fill_(1000.0)
        far = torch.arange(k.shape[0], device="cuda") % 4096 < 64
        k[far, :, 0] = 25.2 * math.log(2) / 16
        v[far] = 0.0
    c.write()
    out = qmoe.attn_paged(c.cache, c.batch(new), c.q, scale=1.0)
    assert qmoe.qmoe_check_status() == 0
    check(c, out, 1.0, 0.0, 2.0 ** -32 if dtype == F16 else 0.0)


@pytest.mark.parametrize("window", [1 << 29, (1 << 30) - 1, 1 << 30, (1 << 31) - 1])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("max_new", [1, 40])
def test_the_widest_windows(cuda_dev, window, causal, max_new):
    """As no window, also for rows before their sequence's beginning, which see
    keys where the mask is not causal."""
    c = Case([(6, 2), (3, 1), (4, 0), (5, 300), (1, 1)], 6, 2, 64, 16)
    out, lse = qmoe.attn_paged(c.cache, c.batch(max_new), c.q, window=window, causal=causal, want_lse=True)
    assert qmoe.qmoe_check_status() == 0
    c.check(out, lse, causal=causal)


@pytest.mark.parametrize("cap", [1e-3, 1e-30, 1e-44])
@pytest.mark.parametrize("lens,heads,kv_heads,new", LENS, ids=["decode", "drafts", "chunks"])
def test_caps_far_below_the_scores(cuda_dev, lens, heads, kv_heads, new, cap):
    """Every score is plus or minus the cap, or 0 where the product is 0."""
    c = Case(lens, heads, kv_heads, 128, 16, F16, seed=4)
    for k in c.keys:
        k[::3] = 0
    c.write()
    out = qmoe.attn_paged(c.cache, c.batch(new), c.q, softcap=cap)
    assert qmoe.qmoe_check_status() == 0
    check(c, out, 128 ** -0.5, cap, 2.0 ** -25)
