"""The operators between the library's quantised products, as cases that can be measured.

Three operators: `append` (rotary positions of a step's queries and keys, keys and values stored in a paged
cache), `attention` (new tokens over that cache) and `logits` (penalties, biases and a grammar mask on the
vocabulary projection's output).  With `own` false, run() computes them in elementary torch operations; with
`own` true it calls the library.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
#: the most that a drawn attention case may cost (the largest listed one's flops and cache bytes)
MOST_FLOPS, MOST_BYTES = 1.0e12, 2.2e9


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # one user's next token, short context: launch and latency
        dict(name="attn decode 1x900", op="attention", dtype="f16", batch=1, new=1, ctx=900, ragged=False, heads=32, kv_heads=8,
             dim=128, page=16, window=0, cap=0.0, lse=False),
        # a full serving batch's next tokens, contexts of every length up to 4K
        dict(name="attn decode 64x4k ragged", op="attention", dtype="f16", batch=64, new=1, ctx=4096, ragged=True, heads=32, kv_heads=8,
             dim=128, page=16, window=0, cap=0.0, lse=False),
        # two long documents: the cache is all that counts
        dict(name="attn decode 2x100k", op="attention", dtype="bf16", batch=2, new=1, ctx=100003, ragged=False, heads=32, kv_heads=4,
             dim=128, page=64, window=0, cap=0.0, lse=True),
        # 24 draft tokens verified at once in a sliding-window layer with capped scores
        dict(name="attn verify 8x24 window cap", op="attention", dtype="f16", batch=8, new=24, ctx=4096, ragged=True, heads=16,
             kv_heads=8, dim=256, page=32, window=1024, cap=50.0, lse=False),
        # the 128-token prefill chunk at the end of a 4K context
        dict(name="attn chunk 128 over 4k", op="attention", dtype="f16", batch=1, new=128, ctx=4096, ragged=False, heads=32, kv_heads=8,
             dim=128, page=16, window=0, cap=0.0, lse=False),
        # several prompts' long chunks in one call, ragged, bf16
        dict(name="attn prompts 4x2048 over 8k", op="attention", dtype="bf16", batch=4, new=2048, ctx=8192, ragged=True, heads=32,
             kv_heads=8, dim=128, page=64, window=0, cap=0.0, lse=False),
        # one decode step of a small batch
        dict(name="append decode 7", op="append", dtype="f16", batch=7, new=1, ctx=600, ragged=True, heads=32, kv_heads=8, dim=128,
             rot=128, layout="half", factor=1.0, page=16),
        # a 128-token chunk, a quarter of each head rotated in neighbouring pairs
        dict(name="append chunk 128 partial", op="append", dtype="bf16", batch=1, new=128, ctx=1000, ragged=False, heads=16, kv_heads=8,
             dim=256, rot=64, layout="interleaved", factor=1.0, page=32),
        # several prompts at far positions, frequencies scaled for a long context
        dict(name="append prompts 4x2048 scaled", op="append", dtype="f16", batch=4, new=2048, ctx=3001, ragged=True, heads=32,
             kv_heads=8, dim=128, rot=128, layout="half", factor=8.0, page=64),
        # one user's next token
        dict(name="logits 1x32000", op="logits", dtype="f16", rows=1, vocab=32000, history=700, biases=0, mask=False),
        # a serving batch, odd vocabulary, everything on
        dict(name="logits 48x151937 all", op="logits", dtype="f32", rows=48, vocab=151937, history=4096, biases=40, mask=True),
        # the widest batch, the largest vocabulary, long histories
        dict(name="logits 256x262144", op="logits", dtype="bf16", rows=256, vocab=262144, history=12000, biases=0, mask=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "append", "logits"])
    if op == "logits":
        rows = _log(rng, 1, 256)
        return dict(op=op, dtype=rng.choice(["f16", "bf16", "f32"]), rows=rows, vocab=_log(rng, 1000, 262144 if rows <= 128 else 131072),
                    history=_log(rng, 1, 12000), biases=rng.choice([0, 1, 17, 300]), mask=rng.random() < 0.5)
    heads, kv_heads = rng.choice([(32, 8), (16, 8), (8, 8), (32, 4), (28, 4), (12, 1), (16, 2), (6, 2)])
    dim = rng.choice([64, 64, 80, 96, 128, 128, 256])
    page = rng.choice([8, 16, 20, 32, 64, 128])
    dtype = rng.choice(["f16", "bf16"])
    if op == "append":
        batch = _log(rng, 1, 64)
        new = rng.choice([1, _log(rng, 1, max(1, 8192 // batch))])
        return dict(op=op, dtype=dtype, batch=batch, new=new, ctx=new + _log(rng, 1, 1000), ragged=rng.random() < 0.5, heads=heads,
                    kv_heads=kv_heads, dim=dim, rot=rng.choice([dim, dim // 2, 2 * (dim // 8)]), layout=rng.choice(["half", "interleaved"]),
                    factor=rng.choice([1.0, 4.0, 16.0]), page=page)
    while True:
        batch = _log(rng, 1, 64)
        new = rng.choice([1, 1, _log(rng, 2, 40), _log(rng, 2, 2048)])
        c = dict(op=op, dtype=dtype, batch=batch, new=new, ctx=new + _log(rng, 1, 100000) - 1, ragged=rng.random() < 0.6, heads=heads,
                 kv_heads=kv_heads, dim=dim, page=page, window=rng.choice([0, 0, _log(rng, 1, 5000)]), cap=rng.choice([0.0, 0.0, 30.0, 50.0]),
                 lse=rng.random() < 0.4)
        scores = batch * new * heads * c["ctx"]
        if 4.0 * dim * scores <= MOST_FLOPS and 4.0 * batch * c["ctx"] * kv_heads * dim <= MOST_BYTES and scores <= 2.4e9:
            return c


def _lens(case):
    """(new tokens, cached tokens with them) of each sequence: a matter of the case alone."""
    n, new, ctx = case["batch"], case["new"], case["ctx"]
    if not case["ragged"]:
        return [new] * n, [ctx] * n
    part = [((i + 1) * 0.6180339887498949) % 1.0 for i in range(n)]
    q = [max(1, round(new * (0.25 + 0.75 * p))) for p in part]
    return q, [max(a, round(ctx * (1.0 - p))) for a, p in zip(q, part[::-1])]


# ----------------------------------------------------------------- inputs --
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    s = {"case": case}
    if case["op"] == "logits":
        return _prepare_logits(case, s, g, dt)
    q_len, kv_len = _lens(case)
    page, kvh, dim, heads = case["page"], case["kv_heads"], case["dim"], case["heads"]
    pages = [-(-n // page) for n in kv_len]
    most, total = max(pages), sum(pages) + 3
    ids = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(pages), most), -1, dtype=torch.int32, device="cuda")  # what lies behind a sequence's last page
    held = torch.arange(most, device="cuda")[None] < torch.tensor(pages, device="cuda")[:, None]
    table[held] = ids[: sum(pages)]
    s["table"] = table
    s["q_start"] = torch.tensor(np.cumsum([0] + q_len), dtype=torch.int32, device="cuda")
    s["kv_len"] = torch.tensor(kv_len, dtype=torch.int32, device="cuda")
    s["tokens"], s["max_new"], s["max_len"] = sum(q_len), max(q_len), max(kv_len)
    rand = lambda *n: torch.randn(*n, generator=g, device="cuda", dtype=dt)  # noqa: E731
    s["k"], s["v"] = rand(total, page, kvh, dim), rand(total, page, kvh, dim)
    if case["op"] == "append":  # one row of the QKV projection's output for each token
        qkv = rand(s["tokens"], (heads + 2 * kvh) * dim)
        s["q"] = qkv[:, : heads * dim].unflatten(1, (heads, dim))
        s["k_new"] = qkv[:, heads * dim: (heads + kvh) * dim].unflatten(1, (kvh, dim))
        s["v_new"] = qkv[:, (heads + kvh) * dim:].unflatten(1, (kvh, dim))
        # the frequencies, stretched where the wavelength is longer than a part of the trained length
        s["freq"] = _frequencies(case).cuda()
        s["scale"] = 1.0
    else:
        s["q"] = 2 * rand(s["tokens"], heads, dim)
    if own:
        from moe_expert_gemv_b200 import qmoe
        s["cache"] = qmoe.KVCache(s["k"], s["v"])
        s["batch"] = qmoe.KVBatch(s["table"], s["q_start"], s["kv_len"], max_new=s["max_new"])
        if case["op"] == "append":
            s["rope"] = qmoe.Rope(s["freq"], case["layout"], s["scale"])
    return s


def _frequencies(case):
    i = torch.arange(case["rot"] // 2, dtype=torch.float64)
    f = 1e4 ** (-2 * i / case["rot"])
    return torch.where(2 * math.pi / f > 2048, f / case["factor"], f)


def _prepare_logits(case, s, g, dt):
    rows, vocab, most = case["rows"], case["vocab"], case["history"]
    s["logits"] = (4 * torch.randn(rows, vocab, generator=g, device="cuda")).to(dt)
    # a text's tokens: some are far more frequent than others
    u = torch.rand(rows, most, generator=g, device="cuda", dtype=torch.float64)
    s["history"] = (vocab ** u).to(torch.int32).clamp_(max=vocab - 1)
    part = [((i + 1) * 0.6180339887498949) % 1.0 for i in range(rows)]
    n = [max(1, round(most * p)) if rows > 1 else most for p in part]
    s["history_len"] = torch.tensor(n, dtype=torch.int32, device="cuda")
    s["prompt_len"] = torch.tensor([int(a * p) for a, p in zip(n, part[::-1])], dtype=torch.int32, device="cuda")
    knob = lambda lo, hi: lo + (hi - lo) * torch.rand(rows, generator=g, device="cuda")  # noqa: E731
    s["repetition"], s["presence"], s["frequency"] = knob(1.0, 1.4), knob(-0.5, 1.0), knob(0.0, 0.7)
    s["bias_ids"] = s["bias"] = s["mask"] = None
    if case["biases"]:
        at = torch.arange(case["biases"], device="cuda") * (vocab // case["biases"])
        s["bias_ids"] = ((at[None] + torch.randint(0, vocab, (rows, 1), generator=g, device="cuda")) % vocab).to(torch.int32)
        s["bias"] = 5 * torch.randn(rows, case["biases"], generator=g, device="cuda")
    if case["mask"]:  # one bit for each token, the lowest first; half the rows leave little
        bits = torch.randint(-(1 << 31), 1 << 31, (3, rows, -(-vocab // 32)), generator=g, device="cuda").to(torch.int32)
        s["mask"] = torch.where((torch.arange(rows, device="cuda") % 2 == 0)[:, None], bits[0], bits[0] & bits[1] & bits[2])
    return s


# -------------------------------------------------------------- operators --
def run(s):
    case = s["case"]
    if own:
        from moe_expert_gemv_b200 import qmoe
        if case["op"] == "append":
            q = qmoe.kv_append(s["cache"], s["batch"], s["k_new"], s["v_new"], q=s["q"], rope=s["rope"])
            return {"q": q, "k": s["k"], "v": s["v"]}
        if case["op"] == "attention":
            r = qmoe.attn_paged(s["cache"], s["batch"], s["q"], window=case["window"], softcap=case["cap"], want_lse=case["lse"])
            return {"out": r[0], "lse": r[1]} if case["lse"] else {"out": r}
        return {"logits": qmoe.logits_process(
            s["logits"], history=s["history"], history_len=s["history_len"], prompt_len=s["prompt_len"], repetition=s["repetition"],
            presence=s["presence"], frequency=s["frequency"], bias_ids=s["bias_ids"], bias=s["bias"], mask=s["mask"])}
    return {"append": _append, "attention": _attention, "logits": _logits}[case["op"]](s)


def _places(s):
    """Of each new token: its sequence and its position."""
    t = torch.arange(s["tokens"], device="cuda")
    seq = torch.searchsorted(s["q_start"][1:].contiguous(), t.to(torch.int32), right=True)
    return seq, s["kv_len"][seq].long() - s["q_start"][seq + 1].long() + t


def _rotate(x, pos, freq, scale, layout):
    angle = pos.double()[:, None] * freq[None]
    c, sn = (scale * angle.cos()).float()[:, None], (scale * angle.sin()).float()[:, None]
    y, half = x.float(), freq.numel()
    at = (slice(0, half), slice(half, 2 * half)) if layout == "half" else (slice(0, 2 * half, 2), slice(1, 2 * half, 2))
    a, b = y[..., at[0]], y[..., at[1]]
    r = y.clone()
    r[..., at[0]], r[..., at[1]] = a * c - b * sn, a * sn + b * c
    return r.to(x.dtype)


def _append(s):
    case = s["case"]
    seq, pos = _places(s)
    page = s["table"][seq, pos // case["page"]].long()
    s["k"][page, pos % case["page"]] = _rotate(s["k_new"], pos, s["freq"], s["scale"], case["layout"])
    s["v"][page, pos % case["page"]] = s["v_new"]
    return {"q": _rotate(s["q"], pos, s["freq"], s["scale"], case["layout"]), "k": s["k"], "v": s["v"]}


def _attention(s):
    case = s["case"]
    n, kvh, dim, group = len(s["kv_len"]), case["kv_heads"], case["dim"], case["heads"] // case["kv_heads"]
    seq, pos = _places(s)
    row = torch.arange(s["tokens"], device="cuda") - s["q_start"][seq]
    # queries of a sequence side by side: [sequence, kv head, token x head of the group, dim]
    q = torch.zeros(n, s["max_new"], kvh, group, dim, device="cuda")
    q[seq, row] = s["q"].float().unflatten(1, (kvh, group))
    at = torch.full((n, s["max_new"]), -1, device="cuda")
    at[seq, row] = pos
    q = q.transpose(1, 2).reshape(n, kvh, -1, dim)
    pages = s["table"].clamp(min=0).long()
    k = s["k"][pages].flatten(1, 2)[:, : s["max_len"]].float().permute(0, 2, 3, 1)
    x = torch.matmul(q, k) * (1.0 / math.sqrt(dim))
    del k
    if case["cap"]:
        x = case["cap"] * torch.tanh(x / case["cap"])
    j = torch.arange(s["max_len"], device="cuda")
    seen = (j[None, None] <= at[..., None]) & (j[None, None] < s["kv_len"][:, None, None])
    if case["window"]:
        seen &= j[None, None] > at[..., None] - case["window"]
    seen = seen[:, None, :, None].expand(-1, 1, -1, group, -1).reshape(n, 1, -1, s["max_len"])
    x = x.masked_fill_(~seen, -math.inf)
    top = x.amax(-1, keepdim=True).clamp(min=-1e30)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    v = s["v"][pages].flatten(1, 2)[:, : s["max_len"]].float().transpose(1, 2)
    o = torch.matmul(x, v) / total.clamp(min=1e-30)
    o = o.unflatten(2, (-1, group)).transpose(1, 2)[seq, row].flatten(1, 2).to(s["q"].dtype)
    if not case["lse"]:
        return {"out": o}
    lse = (top + total.log()).squeeze(-1).unflatten(2, (-1, group)).transpose(1, 2)[seq, row].flatten(1, 2)
    return {"out": o, "lse": lse}


def _logits(s):
    x = s["logits"].float()
    rows, vocab = x.shape
    i = torch.arange(s["history"].shape[1], device="cuda")[None]
    held = i < s["history_len"][:, None]
    ids = s["history"].long()
    seen = torch.zeros(rows, vocab, device="cuda").scatter_add_(1, ids, held.float()) > 0
    n = torch.zeros(rows, vocab, device="cuda").scatter_add_(1, ids, (held & (i >= s["prompt_len"][:, None])).float())
    rep = s["repetition"][:, None]
    x = torch.where(seen, torch.where(x > 0, x / rep, x * rep), x)
    x = x - s["frequency"][:, None] * n - s["presence"][:, None] * (n > 0)
    if s["bias"] is not None:
        x = x.scatter_add(1, s["bias_ids"].long(), s["bias"])
    if s["mask"] is not None:
        bit = (s["mask"][..., None] >> torch.arange(32, device="cuda", dtype=torch.int32)) & 1
        x = x.masked_fill(bit.flatten(1)[:, :vocab] == 0, -math.inf)
    return {"logits": x.to(s["logits"].dtype)}


# ------------------------------------------------------------------- work --
def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "logits":
        part = [((i + 1) * 0.6180339887498949) % 1.0 for i in range(case["rows"])]
        held = sum(max(1, round(case["history"] * p)) if case["rows"] > 1 else case["history"] for p in part)
        cells = case["rows"] * case["vocab"]
        return {"bytes": 2 * cells * size + (cells / 8 if case["mask"] else 0) + 4 * held + 8 * case["rows"] * case["biases"],
                "flops": cells}
    q_len, kv_len = _lens(case)
    tokens = sum(q_len)
    if case["op"] == "append":
        cells = tokens * (case["heads"] + 2 * case["kv_heads"]) * case["dim"]
        return {"bytes": 2 * cells * size, "flops": 3 * cells}
    pairs = keys = 0
    for n, length in zip(q_len, kv_len):
        window = case["window"] or length
        first = max(0, length - n - window + 1)
        keys += length - first
        p = np.arange(length - n, length)
        pairs += int(np.minimum(p + 1, window).sum())
    return {"bytes": 2 * size * keys * case["kv_heads"] * case["dim"] + 2 * size * tokens * case["heads"] * case["dim"],
            "flops": 4.0 * case["dim"] * case["heads"] * pairs}


# ------------------------------------------------------------------ exact --
def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attention": _exact_attention, "logits": _exact_logits}[case["op"]](case, s)


def _exact_append(case, s):
    out = {"q": s["q"].double(), "k": s["k"].double(), "v": s["v"].double()}
    q_len, kv_len = _lens(case)
    half, at = case["rot"] // 2, 0
    for b, (n, length) in enumerate(zip(q_len, kv_len)):
        pos = torch.arange(length - n, length, device="cuda")
        turn = torch.polar(torch.full((n, half), float(s["scale"]), dtype=torch.float64, device="cuda"),
                           torch.outer(pos.double(), s["freq"]))[:, None]
        rotated = []
        for x in (s["q"], s["k_new"]):
            y = x[at: at + n].double()
            head = y[..., : 2 * half]
            pairs = head.unflatten(-1, (2, half)).transpose(-1, -2) if case["layout"] == "half" else head.unflatten(-1, (half, 2))
            z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
            z = (z.transpose(-1, -2) if case["layout"] == "half" else z).flatten(-2)
            rotated.append(torch.cat([z, y[..., 2 * half:]], -1))
        out["q"][at: at + n] = rotated[0]
        slot = s["table"][b].long()[pos // case["page"]] * case["page"] + pos % case["page"]
        out["k"].flatten(0, 1)[slot] = rotated[1]
        out["v"].flatten(0, 1)[slot] = s["v_new"][at: at + n].double()
        at += n
    return out


def _exact_attention(case, s):
    q_len, kv_len = _lens(case)
    kvh, dim, group = case["kv_heads"], case["dim"], case["heads"] // case["kv_heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    at = 0
    for b, (n, length) in enumerate(zip(q_len, kv_len)):
        slot = torch.arange(length, device="cuda")
        slot = s["table"][b].long()[slot // case["page"]] * case["page"] + slot % case["page"]
        pos = torch.arange(length - n, length, device="cuda")
        lag = pos[:, None] - torch.arange(length, device="cuda")[None]
        hidden = (lag < 0) | (lag >= (case["window"] or length))
        for h in range(kvh):
            k, v = s["k"].flatten(0, 1)[slot, h].double(), s["v"].flatten(0, 1)[slot, h].double()
            for i in range(h * group, (h + 1) * group):
                x = s["q"][at: at + n, i].double() @ k.T / math.sqrt(dim)
                if case["cap"]:
                    x = torch.tanh(x / case["cap"]) * case["cap"]
                x.masked_fill_(hidden, -math.inf)
                lse[at: at + n, i] = torch.logsumexp(x, 1)
                out[at: at + n, i] = torch.softmax(x, 1) @ v
        at += n
    return {"out": out, "lse": lse} if case["lse"] else {"out": out}


def _exact_logits(case, s):
    x = s["logits"].double()
    for r in range(case["rows"]):
        n, p = int(s["history_len"][r]), int(s["prompt_len"][r])
        ids = s["history"][r, :n].long()
        told = torch.unique(ids)
        y = x[r, told]
        x[r, told] = torch.where(y > 0, y / s["repetition"][r].double(), y * s["repetition"][r].double())
        made, times = torch.unique(ids[p:], return_counts=True)
        x[r, made] -= s["frequency"][r].double() * times + s["presence"][r].double()
        if s["bias"] is not None:
            x[r, s["bias_ids"][r].long()] += s["bias"][r].double()
        if s["mask"] is not None:
            word = s["mask"][r].long() & 0xFFFFFFFF
            v = torch.arange(case["vocab"], device="cuda")
            x[r, (word[v // 32] >> (v % 32)) & 1 == 0] = -math.inf
    return {"logits": x}
