"""Paged caches, their batches and 64-bit results for the attention tests."""
import math

import torch

from moe_expert_gemv_b200 import qmoe

HALF_STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


class Case:
    """Random sequences (new tokens, cached length) in a shuffled paged cache.
    Slots that no sequence holds, pages that none has and table entries behind
    a sequence's last page are poison: NaN, or a page id outside the cache."""

    def __init__(self, lens, heads, kv_heads, dim, page, dtype=torch.float16, seed=0, head_major=False, spare=0,
                 device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        self.lens, self.heads, self.kv_heads, self.dim, self.page, self.dtype = lens, heads, kv_heads, dim, page, dtype
        pages = [-(-kv // page) for _, kv in lens]
        total = sum(pages) + 2
        ids = torch.randperm(total, generator=g, device=device).to(torch.int32)
        self.table = torch.full((len(lens), max(max(pages), 1)), 1 << 30, dtype=torch.int32, device=device)
        at = 0
        for b, n in enumerate(pages):
            self.table[b, :n] = ids[at:at + n]
            at += n
        shape = (total, kv_heads, page, dim) if head_major else (total, page, kv_heads, dim)
        self.k = torch.full(shape, math.nan, dtype=dtype, device=device)
        self.v = torch.full(shape, math.nan, dtype=dtype, device=device)
        if head_major:
            self.k, self.v = self.k.transpose(1, 2), self.v.transpose(1, 2)
        self.keys, self.values, self.slots = [], [], []
        for b, (_, kv) in enumerate(lens):
            j = torch.arange(kv, device=device)
            self.slots.append((self.table[b].long()[j // page], j % page))
            self.keys.append(torch.randn(kv, kv_heads, dim, generator=g, device=device, dtype=dtype))
            self.values.append(torch.randn(kv, kv_heads, dim, generator=g, device=device, dtype=dtype))
        self.write()
        self.tokens = sum(n for n, _ in lens)
        starts = [0]
        for n, _ in lens:
            starts.append(starts[-1] + n)
        self.q_start = torch.tensor(starts, dtype=torch.int32, device=device)
        self.kv_len = torch.tensor([kv for _, kv in lens], dtype=torch.int32, device=device)
        self.q = 2 * torch.randn(self.tokens + spare, heads, dim, generator=g, device=device, dtype=dtype)
        self.cache = qmoe.KVCache(self.k, self.v)

    def write(self):
        for (pg, sl), k, v in zip(self.slots, self.keys, self.values):
            self.k[pg, sl], self.v[pg, sl] = k, v

    def batch(self, max_new=0):
        return qmoe.KVBatch(self.table, self.q_start, self.kv_len, max_new=max_new)

    def want(self, scale=None, cap=0.0, window=0, causal=True):
        """(out, lse, bound of the error of out), 64-bit.

        The bound, with u half a step of the type: the output's rounding u |o|;
        the weights' rounding u sum p |v| (and 2^-25 for each weight below the
        normal fp16 range); a score's error e (a fp32 dot product of dim
        terms, its scaling and the exponential's argument: (dim + 8) 2^-24 of
        the sum of |q k| scaled, 2^-21 of the cap, 2^-21 absolute for ex2)
        shifts p and the sum by e each; fp32 sums of n terms, truncated by the
        tensor cores: (n + 64) 2^-23 of sum p |v|."""
        scale = self.dim ** -0.5 if scale is None else scale
        u = HALF_STEP[self.dtype]
        out, lse, tol = [], [], []
        at = 0
        for (n, kv), k, v in zip(self.lens, self.keys, self.values):
            q = self.q[at:at + n].double().transpose(0, 1)
            at += n
            grp = self.heads // self.kv_heads
            k = k.double().repeat_interleave(grp, 1).permute(1, 2, 0)
            v = v.double().repeat_interleave(grp, 1).transpose(0, 1)
            s = q @ k * scale
            e = (self.dim + 8) * 2.0 ** -24 * ((q.abs() @ k.abs() * scale).amax(-1, keepdim=True) if kv else 0) + \
                2.0 ** -21 * (1 + cap)
            if cap:
                s = cap * torch.tanh(s / cap)
            p = (kv - n + torch.arange(n, device=q.device))[:, None]
            j = torch.arange(kv, device=q.device)[None]
            see = torch.ones(n, kv, dtype=torch.bool, device=q.device)
            if causal:
                see &= j <= p
            if window:
                see &= j > p - window
            s = s.masked_fill(~see, -math.inf)
            some = see.any(-1)[None, :, None]
            w = torch.where(some, torch.softmax(s, -1), 0.0) if kv else s
            # a masked value does not count, whatever it is
            vis = torch.where(w[..., None] > 0, v[:, None], 0.0) if not torch.isfinite(v).all() else None
            o = w @ v if vis is None else (w[..., None] * vis).sum(2)
            a = w @ v.abs().nan_to_num(0, 0, 0)
            out.append(o.transpose(0, 1))
            lse.append(torch.where(some[..., 0], torch.logsumexp(s, -1), -math.inf).transpose(0, 1)
                       if kv else torch.full((n, self.heads), -math.inf, dtype=torch.float64, device=q.device))
            t = u * o.abs() + (u + 2 * e + (kv + 64) * 2.0 ** -23) * a + \
                (kv * 2.0 ** -25 * v.abs().nan_to_num(0, 0, 0).amax() if kv else 0) + 2.0 ** -25
            tol.append(t.transpose(0, 1))
        return torch.cat(out), torch.cat(lse), torch.cat(tol)

    def check(self, got, lse=None, **kw):
        o, l64, tol = self.want(**kw)
        n = self.tokens
        got = got[:n].double()
        fin = torch.isfinite(o)
        assert torch.equal(fin, torch.isfinite(got)), "finite where the formula is not, or the other way round"
        assert torch.equal(torch.isnan(o), torch.isnan(got)) and torch.equal(o[~fin & ~torch.isnan(o)], got[~fin & ~torch.isnan(o)])
        over = ((got - o).abs() / tol)[fin]
        assert over.numel() == 0 or over.max() <= 1, "error %.2f times the bound" % over.max()
        if lse is not None:
            none = torch.isinf(l64)
            assert torch.equal(none, torch.isinf(lse[:n]) & (lse[:n] < 0))
            # fp32 sums and a score error as above; scores here stay below 64
            assert ((lse[:n].double() - l64).abs()[~none] <= 2.0 ** -14).all()
