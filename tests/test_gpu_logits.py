"""logits_process against the formula in 64 bits."""
import math

import pytest
import torch

from moe_expert_gemv_b200 import qmoe

pytestmark = pytest.mark.gpu
STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def make(rows, vocab, hist, biases=0, mask=False, dtype=torch.float32, seed=0):
    g = torch.Generator().manual_seed(seed)
    d = dict(logits=(4 * torch.randn(rows, vocab, generator=g)).to(dtype))
    if hist:
        d["history"] = (vocab ** torch.rand(rows, hist, generator=g)).int().clamp_(max=vocab - 1)
        d["history_len"] = torch.randint(0, hist + 1, (rows,), generator=g).int()
        d["history_len"][0] = hist
        d["prompt_len"] = (d["history_len"] * torch.rand(rows, generator=g)).int()
        d["repetition"] = 0.8 + torch.rand(rows, generator=g)
        d["presence"], d["frequency"] = torch.randn(rows, generator=g), torch.randn(rows, generator=g)
    if biases:
        d["bias_ids"] = torch.randint(-1, vocab, (rows, biases), generator=g).int()
        d["bias"] = 3 * torch.randn(rows, biases, generator=g)
    if mask:
        d["mask"] = torch.randint(-(1 << 31), 1 << 31, (rows, -(-vocab // 32)), generator=g).int()
        if rows > 1:
            d["mask"][1] = 0
    return d


def formula(d):
    """64 bits, on the CPU; also the sum of the magnitudes of a value's terms."""
    x = d["logits"].double()
    rows, vocab = x.shape
    big = x.abs()
    if "history" in d:
        for r in range(rows):
            n = max(0, min(int(d["history_len"][r]), d["history"].shape[1]))
            p = int(d["prompt_len"][r]) if "prompt_len" in d else 0
            h = d["history"][r, :n].long()
            ok = (h >= 0) & (h < vocab)
            seen = torch.zeros(vocab, dtype=torch.bool)
            seen[h[ok]] = True
            gen = torch.arange(n) >= p
            cnt = torch.bincount(h[ok & gen], minlength=vocab).double()
            rep = d["repetition"][r].double() if "repetition" in d else 1.0
            x[r] = torch.where(seen, torch.where(x[r] > 0, x[r] / rep, x[r] * rep), x[r])
            f = d["frequency"][r].double() if "frequency" in d else 0.0
            q = d["presence"][r].double() if "presence" in d else 0.0
            x[r] -= f * cnt + q * (cnt > 0)
            big[r] = torch.maximum(big[r], x[r].abs()) + abs(f) * cnt + abs(q) * (cnt > 0)
    if "bias" in d:
        ids = d["bias_ids"].long()
        ok = (ids >= 0) & (ids < vocab)
        x.scatter_add_(1, ids.clamp(0, vocab - 1), d["bias"].double() * ok)
        big.scatter_add_(1, ids.clamp(0, vocab - 1), d["bias"].double().abs() * ok)
    if "mask" in d:
        v = torch.arange(vocab)
        x[((d["mask"].expand(rows, -1)[:, v // 32] >> (v % 32)) & 1) == 0] = -math.inf
    return x, big


def check(d, got):
    want, big = formula(d)
    got = got.double().cpu()
    inf = ~torch.isfinite(want)
    assert torch.equal(want[inf].nan_to_num(1e9), got[inf].nan_to_num(1e9))
    # half a step of the result; up to 2 + 1024 fp32 operations, of which a value meets at most 8 here
    tol = STEP[d["logits"].dtype] * want.abs() + 8 * 2.0 ** -24 * big + 2.0 ** -25
    e = ((got - want).abs() / tol)[~inf]
    assert e.numel() == 0 or e.max() <= 1, "error %.2f times the bound" % e.max()


def run(d, **kw):
    c = {k: v.cuda() for k, v in d.items()}
    y = qmoe.logits_process(c.pop("logits"), **c, **kw)
    assert qmoe.qmoe_check_status() == 0
    return y


@pytest.mark.parametrize("dtype", list(STEP))
@pytest.mark.parametrize("rows,vocab,hist,biases,mask", [
    (1, 32000, 700, 0, False), (3, 50257, 2000, 17, True), (2, 1, 5, 1, True), (5, 31, 40, 3, True), (4, 8192, 1, 0, True),
    (2, 8193, 300, 1, False), (1, 262144, 9000, 300, True), (7, 1001, 0, 20, True), (2, 40000, 0, 0, True), (3, 999, 3000, 0, False),
    (33, 16411, 129, 1000, True), (2, 70001, 0, 0, False)])
def test_all_rules(cuda_dev, dtype, rows, vocab, hist, biases, mask):
    d = make(rows, vocab, hist, min(biases, vocab), mask, dtype, seed=vocab)
    if biases == 1000:   # distinct ids: a value meets few of them
        d["bias_ids"] = torch.stack([torch.randperm(vocab)[:biases] for _ in range(rows)]).int()
    check(d, run(d))


def test_single_rules(cuda_dev):
    full = make(3, 5000, 400, 9, True, seed=5)
    for only in ("repetition", "presence", "frequency", "bias", "mask", "prompt_len", None):
        d = {"logits": full["logits"]}
        if only in ("repetition", "presence", "frequency", "prompt_len"):
            d |= {k: full[k] for k in ("history", "history_len", only)}
            if only == "prompt_len":
                d["frequency"] = full["frequency"]
        elif only == "bias":
            d |= {k: full[k] for k in ("bias", "bias_ids")}
        elif only:
            d[only] = full[only]
        check(d, run(d))


def test_in_place_strided_and_shared_mask(cuda_dev):
    d = make(4, 1003, 300, 5, True, torch.float16)
    d["mask"] = d["mask"][:1].contiguous()
    wide = torch.full((4, 2011), 7.0, dtype=torch.float16)
    wide[:, 3:1006] = d["logits"]
    w = wide.cuda()
    c = {k: v.cuda() for k, v in d.items()}
    c.pop("logits")
    hist = torch.full((4, 401), 5, dtype=torch.int32, device="cuda")
    hist[:, 50:350] = c["history"]
    c["history"] = hist[:, 50:350]
    view = w[:, 3:1006]
    assert qmoe.logits_process(view, out=view, **c) is view
    assert qmoe.qmoe_check_status() == 0
    check(d, view)
    assert (w[:, :3] == 7).all() and (w[:, 1006:] == 7).all()


def test_values_that_are_not_finite(cuda_dev):
    d = make(2, 300, 50, 0, True)
    d["logits"][:, 0::7], d["logits"][:, 1::7], d["logits"][:, 2::7] = math.inf, -math.inf, math.nan
    d["repetition"][:] = 1.3
    got = run(d).cpu()
    want, _ = formula(d)
    # an infinity keeps its sign, a NaN stays one, and a cleared bit is -inf whatever was there
    assert torch.equal(torch.isnan(got), torch.isnan(want)) and torch.equal(torch.isposinf(got), torch.isposinf(want))
    assert torch.equal(torch.isneginf(got), torch.isneginf(want))


def test_the_same_bias_id_many_times_adds_in_order(cuda_dev):
    d = make(1, 100, 0, 1024)
    d["bias_ids"][:] = 42
    d["bias"] = torch.rand(1, 1024)
    y = run(d)
    s = torch.zeros(())
    for b in d["bias"][0]:
        s = s + b
    assert y[0, 42].cpu() == d["logits"][0, 42] + s
    assert torch.equal(y.cpu()[0, :42], d["logits"][0, :42])


def test_bad_ids_are_flagged_and_skipped(cuda_dev):
    for key, ids in (("history", [5, -1, 1000, 3]), ("history", [5, -7, 3, 3]), ("bias_ids", [2, 1000, -1, 2])):
        d = make(1, 1000, 4, 4)
        d["history_len"][:] = 4
        d["prompt_len"][:] = 0
        d[key] = torch.tensor([ids], dtype=torch.int32)
        c = {k: v.cuda() for k, v in d.items()}
        y = qmoe.logits_process(c.pop("logits"), **c)
        assert qmoe.qmoe_check_status() == qmoe.DEV_BAD_TOKEN
        check(d, y)


def test_history_length_is_cut(cuda_dev):
    d = make(2, 500, 60)
    d["history_len"] = torch.tensor([100000, -3], dtype=torch.int32)
    check(d, run(d))


def test_no_rows(cuda_dev):
    assert qmoe.logits_process(torch.empty(0, 50, device="cuda")).shape == (0, 50)


def test_python_refusals(cuda_dev):
    x = torch.zeros(2, 100, device="cuda")
    h = torch.zeros(2, 4, dtype=torch.int32, device="cuda")
    n = torch.zeros(2, dtype=torch.int32, device="cuda")
    for kw in (dict(history=h), dict(repetition=x[:, 0].contiguous()), dict(bias=x[:, :3].contiguous()),
               dict(mask=h[:, :3].contiguous()), dict(history=h.t().contiguous().t(), history_len=n)):
        with pytest.raises(ValueError):
            qmoe.logits_process(x, **kw)
    with pytest.raises(TypeError):
        qmoe.logits_process(x.double())
    with pytest.raises(TypeError):
        qmoe.logits_process(x, history=h, history_len=n.long())
    with pytest.raises(qmoe.QmoeError):
        qmoe.logits_process(x, bias_ids=torch.zeros(2, 1025, dtype=torch.int32, device="cuda"),
                            bias=torch.zeros(2, 1025, device="cuda"))


def test_more_tokens_than_a_table_holds(cuda_dev):
    """Long histories of tokens that all differ, and ones whose hashes fall
    together (the table's parts go by the low 16 bits of 0x9E3779B1 * id)."""
    V = 200000
    part = [i for i in range(V) if ((i * 0x9E3779B1 & 0xFFFF) * 4 >> 16) == 1]
    assert len(part) > 12000
    for ids in (torch.randperm(V)[:60000], torch.tensor(part[:12000]), torch.tensor(part[:12000]).repeat(2)):
        d = make(1, V, len(ids), 5, True, seed=3)
        d["history"], d["history_len"] = ids[None].int(), torch.tensor([len(ids)], dtype=torch.int32)
        d["prompt_len"] = torch.tensor([len(ids) // 3], dtype=torch.int32)
        check(d, run(d))


def test_captured_and_replayed_with_new_rules(cuda_dev):
    d = make(3, 40000, 900, 4, True, torch.bfloat16)
    c = {k: v.cuda() for k, v in d.items()}
    x = c.pop("logits")
    out = torch.empty_like(x)
    qmoe.logits_process(x, out=out, **c)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qmoe.logits_process(x, out=out, **c)
    for seed in (1, 2):
        d = make(3, 40000, 900, 4, True, torch.bfloat16, seed=seed)
        x.copy_(d["logits"])
        for k in c:
            c[k].copy_(d[k])
        g.replay()
        torch.cuda.synchronize()
        check(d, out)
    assert qmoe.qmoe_check_status() == 0


def test_no_history_yet(cuda_dev):
    """A history without columns is none; a row's logits have to be apart from each other."""
    x = torch.randn(3, 70, device="cuda")
    none = torch.empty(3, 0, dtype=torch.int32, device="cuda")
    y = qmoe.logits_process(x, history=none, history_len=torch.zeros(3, dtype=torch.int32, device="cuda"),
                            repetition=torch.full((3,), 2.0, device="cuda"))
    assert torch.equal(y, x)
    for bad in (x[:, :1].expand(3, 70), x.t().contiguous().t()):
        with pytest.raises(ValueError):
            qmoe.logits_process(bad)
        with pytest.raises(ValueError):
            qmoe.logits_process(bad, out=torch.empty_like(x))
    with pytest.raises(ValueError):
        qmoe.logits_process(x, out=x[:, :1].expand(3, 70))
    assert qmoe.qmoe_check_status() == 0


@pytest.mark.parametrize("rows,vocab,hist,dtype,mask", [(8, 262144, 33000, torch.float16, False), (300, 60001, 4000, torch.bfloat16, True),
                                                        (1, 70001, (1 << 20) - 1, torch.float32, True),
                                                        (17, 200003, 22000, torch.float32, False)])
def test_much_work_with_histories(cuda_dev, rows, vocab, hist, dtype, mask):
    """Histories long enough, over rows and vocabulary, to be sorted first."""
    d = make(rows, vocab, hist, biases=5, mask=mask, dtype=dtype, seed=rows)
    g = torch.Generator().manual_seed(1)
    d["history"][torch.rand(d["history"].shape, generator=g) < 0.1] = -1
    if rows > 2:
        d["history_len"][1], d["history_len"][2] = 0, 1
    y = run(d)
    check(d, y)
    assert torch.equal(y, run(d))
    c = d["logits"].cuda()
    x = {k: v.cuda() for k, v in d.items() if k != "logits"}
    assert torch.equal(qmoe.logits_process(c, out=c, **x), y)
    x["history"][0, 0] = vocab
    qmoe.logits_process(c, **x)
    assert qmoe.qmoe_check_status() == qmoe.DEV_BAD_TOKEN


@pytest.mark.parametrize("dtype", list(STEP))
@pytest.mark.parametrize("hist,biases,mask", [(1500, 9, True), (300, 0, False), (0, 30, True), (0, 0, True), (0, 0, False)])
def test_large_slices(cuda_dev, dtype, hist, biases, mask):
    """Rows enough for slices of 16 KB, which begin anywhere within 16 bytes."""
    d = make(48, 60001, hist, biases, mask, dtype, seed=hist + biases)
    y = run(d)
    check(d, y)
    out = torch.full((48, 60007), 7.0, dtype=dtype, device="cuda")
    c = {k: v.cuda() for k, v in d.items()}
    qmoe.logits_process(c.pop("logits"), out=out[:, 3:60004], **c)
    assert torch.equal(out[:, 3:60004], y) and (out[:, :3] == 7).all() and (out[:, 60004:] == 7).all()
