"""A decoder's step through the library as a server runs it: quantised
projections, rotation and cache, attention, router and experts, vocabulary
projection, rules on the logits.  Every operator is checked against 64 bits on
the inputs that the one before it gave it, and the step's graph, replayed while
the sequences grow, against the same calls made one by one."""
import numpy as np
import pytest
import torch

import oracle
from moe_expert_gemv_b200 import qmoe, synth
from tests._attn import Case
from tests._util import assert_close, f16_bits
from tests.test_gpu_logits import check as check_logits
from tests.test_gpu_rope import close, turned

pytestmark = pytest.mark.gpu

HIDDEN, HEADS, KV, DIM, ROT, VOCAB, E, I, TOP = 512, 8, 2, 64, 32, 1000, 32, 256, 4
QKV = (HEADS + 2 * KV) * DIM


class Model:
    def __init__(self):
        self.np = {n: synth.dense(i, r, c) for i, (n, r, c) in enumerate(
            [("qkv", QKV, HIDDEN), ("o", HIDDEN, HEADS * DIM), ("vocab", VOCAB, HIDDEN)])}
        shape = dict(qkv=(QKV, HIDDEN), o=(HIDDEN, HEADS * DIM), vocab=(VOCAB, HIDDEN))
        self.w = {n: qmoe.QMatrix.from_numpy(*m, *shape[n], 4) for n, m in self.np.items()}
        self.shape = shape
        self.moe_np = synth.moe_layer(7, 0, E=E, H=HIDDEN, I=I)
        self.moe = qmoe.MoELayer.from_numpy(self.moe_np, E, HIDDEN, I)
        self.rope = qmoe.Rope.make(ROT)


class State:
    """Four sequences' cache, with room to grow, and the step's inputs."""

    def __init__(self, lens, seed):
        room = 8
        self.case = c = Case([(n, kv + room) for n, kv in lens], HEADS, KV, DIM, 16, seed=seed)
        c.lens = lens
        c.keys, c.values = [k[:kv] for k, (_, kv) in zip(c.keys, lens)], [v[:kv] for v, (_, kv) in zip(c.values, lens)]
        c.kv_len.copy_(torch.tensor([kv for _, kv in lens], dtype=torch.int32))
        g = torch.Generator().manual_seed(seed)
        self.x = torch.randn(c.tokens, HIDDEN, generator=g).half().cuda()
        rows = c.tokens
        self.rules = dict(history=torch.randint(0, VOCAB, (rows, 40), generator=g).int().cuda(),
                          history_len=torch.randint(0, 41, (rows,), generator=g).int().cuda(),
                          repetition=(1 + torch.rand(rows, generator=g)).cuda(),
                          frequency=torch.rand(rows, generator=g).cuda(),
                          mask=torch.randint(-(1 << 31), 1 << 31, (1, -(-VOCAB // 32)), generator=g).int().cuda())


def norm(x):
    """The model's norm between its blocks, as PyTorch has it."""
    return torch.nn.functional.layer_norm(x.float(), (HIDDEN,)).half()


def step(m, s, batch, status=None):
    """One layer and the answer; every intermediate result."""
    c, T = s.case, s.x.shape[0]
    r = {"qkv": qmoe.qgemv_affine(m.w["qkv"], s.x, status=status)}
    h = r["qkv"].view(T, HEADS + 2 * KV, DIM)
    r["q"] = qmoe.kv_append(c.cache, batch, h[:, HEADS:HEADS + KV], h[:, HEADS + KV:], q=h[:, :HEADS], rope=m.rope,
                            status=status)
    r["attn"] = qmoe.attn_paged(c.cache, batch, r["q"], status=status)
    r["o"] = qmoe.qgemv_affine(m.w["o"], r["attn"].view(T, HEADS * DIM), status=status)
    r["mid"] = norm(s.x + r["o"])
    r["idx"], r["wt"], _ = qmoe.moe_router_topk(m.moe.router, r["mid"], TOP, status=status)
    r["moe"] = qmoe.moe_prefill_qgemm(m.moe, r["mid"], r["idx"], r["wt"], status=status)
    r["last"] = norm(r["mid"] + r["moe"])
    r["vocab"] = qmoe.qgemv_affine(m.w["vocab"], r["last"], status=status)
    r["logits"] = qmoe.logits_process(r["vocab"], **s.rules, status=status)
    return r


def check_step(m, s, r):
    c, T = s.case, s.x.shape[0]

    def product(name, x, y):
        y64, _ = oracle.qgemv(*m.np[name], *m.shape[name], 4, f16_bits(x))
        assert_close(y.cpu().numpy(), y64, what=name)
    product("qkv", s.x, r["qkv"])
    h = r["qkv"].view(T, HEADS + 2 * KV, DIM)
    pos = torch.cat([torch.arange(kv - n, kv) for n, kv in c.lens]).cuda()
    f = m.rope.inv_freq
    close(r["q"], turned(h[:, :HEADS], pos, f, 1.0, "half"), h[:, :HEADS], ROT // 2, torch.float16)
    at = 0
    for b, (n, kv) in enumerate(c.lens):
        pg, sl = (i[:kv] for i in c.slots[b])
        k, v = c.k[pg, sl], c.v[pg, sl]
        new = h[at:at + n, HEADS:HEADS + KV]
        assert torch.equal(v[kv - n:], h[at:at + n, HEADS + KV:]) and torch.equal(v[:kv - n], c.values[b][:kv - n])
        assert torch.equal(k[:kv - n], c.keys[b][:kv - n])
        if n:
            close(k[kv - n:], turned(new, pos[at:at + n], f, 1.0, "half"), new, ROT // 2, torch.float16)
        c.keys[b], c.values[b] = k, v
        at += n
    c.q = r["q"]
    c.check(r["attn"])
    product("o", r["attn"].reshape(T, HEADS * DIM), r["o"])
    mid = f16_bits(r["mid"])
    _, idx, wt = oracle.router(*m.moe_np["router"], E, HIDDEN, 8, mid, TOP)
    assert np.array_equal(r["idx"].cpu().numpy(), idx)
    y64, _ = oracle.Layer(m.moe_np, E, HIDDEN, I).moe(mid, idx, r["wt"].cpu().numpy().astype(np.float64))
    assert_close(r["moe"].cpu().numpy(), y64, what="experts")
    product("vocab", r["last"], r["vocab"])
    check_logits({"logits": r["vocab"].cpu(), **{k: v.cpu() for k, v in s.rules.items()}}, r["logits"])
    assert torch.isfinite(r["vocab"]).all()


@pytest.mark.parametrize("lens", [[(1, 5), (1, 1), (1, 300), (1, 64)], [(1, 70), (0, 9), (6, 6), (9, 200)]])
def test_step(cuda_dev, lens):
    m, s = Model(), State(lens, 3)
    check_step(m, s, step(m, s, s.case.batch()))
    assert qmoe.qmoe_check_status() == 0


def test_replayed_step(cuda_dev):
    lens = [(1, 40), (1, 15), (1, 1), (1, 127)]
    m, a, b = Model(), State(lens, 5), State(lens, 5)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    warm = State(lens, 6)
    with torch.cuda.stream(side):
        batch = b.case.batch(max_new=1)
        step(m, warm, warm.case.batch(max_new=1))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            got = step(m, b, batch, status)
    torch.cuda.synchronize()
    for i in range(3):
        if i:
            x = torch.randn(len(lens), HIDDEN, generator=torch.Generator().manual_seed(i)).half().cuda()
            for s in (a, b):
                s.x.copy_(x)
                s.case.kv_len += 1
                s.case.lens = [(1, kv + i) for _, kv in lens]
        want = step(m, a, a.case.batch(max_new=1))
        g.replay()
        torch.cuda.synchronize()
        for k in want:
            assert torch.equal(want[k], got[k]), "%s, step %d" % (k, i)
        check_step(m, b, got)
    assert int(status) == 0 and qmoe.qmoe_check_status() == 0


@pytest.mark.parametrize("lens", [[(1, 900), (1, 3)], [(40, 700), (128, 128)]])
def test_without_dependent_launches(cuda_dev, lens):
    """The same bits with and without programmatic dependent launches."""
    rows = torch.randn(300, 60001, device="cuda").half()
    hist = torch.randint(0, 60001, (300, 4000), dtype=torch.int32, device="cuda")
    rules = dict(history=hist, history_len=torch.full((300,), 4000, dtype=torch.int32, device="cuda"),
                 frequency=torch.ones(300, device="cuda"))
    got = []
    for on in (1, 0):
        before = qmoe.qmoe_set_dependent_launch(on)
        try:
            c = State(lens, 8).case
            k = torch.randn(c.tokens, KV, DIM, generator=torch.Generator().manual_seed(1)).half().cuda()
            q = qmoe.kv_append(c.cache, c.batch(), k, k, q=c.q, rope=qmoe.Rope.make(ROT))
            got.append((q, qmoe.attn_paged(c.cache, c.batch(), q), qmoe.logits_process(rows, **rules)))
            torch.cuda.synchronize()
        finally:
            qmoe.qmoe_set_dependent_launch(before)
    assert all(torch.equal(a, b) for a, b in zip(*got)) and qmoe.qmoe_check_status() == 0
