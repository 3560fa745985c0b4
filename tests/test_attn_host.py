"""What the attention, rope and logits entry points do on the host: frequency
tables, workspace sizes, and the refusal of bad arguments (checked before any
device is touched, so these calls run without a GPU)."""
import ctypes
import math

import pytest
import torch

from moe_expert_gemv_b200 import qmoe

INVALID, ALIGN, UNSUP, CUDA, WS = -1, -2, -3, -4, -7
PTR = 1 << 20   # an aligned address that a refused call never follows


def test_frequencies():
    R, base, fac, n = 64, 10000.0, 8.0, 2048
    i = torch.arange(R // 2, dtype=torch.float64)
    f = base ** (-2 * i / R)
    got, scale = qmoe.rope_frequencies(R, base)
    assert scale == 1.0 and torch.allclose(got, f, rtol=1e-14)
    assert torch.allclose(qmoe.rope_frequencies(R, base, "linear", fac)[0], f / fac, rtol=1e-14)
    got, _ = qmoe.rope_frequencies(R, base, "base", fac)
    assert got[0] == 1.0 and math.isclose(got[-1], f[-1] / fac, rel_tol=1e-12)
    got, scale = qmoe.rope_frequencies(R, base, "bands", fac, trained=n, low=1.0, high=4.0)
    turns = n * f / (2 * math.pi)
    assert scale == 1.0 and torch.equal(got[turns >= 4], f[turns >= 4])
    assert torch.allclose(got[turns <= 1], f[turns <= 1] / fac, rtol=1e-14)
    mid = (turns > 1) & (turns < 4)
    t = (turns[mid] - 1) / 3
    assert mid.any() and torch.allclose(got[mid], f[mid] * t + f[mid] / fac * (1 - t), rtol=1e-13)
    got, scale = qmoe.rope_frequencies(R, base, "ramp", fac, trained=n, low=1.0, high=32.0)
    at = lambda turns: R * math.log(n / (2 * math.pi * turns)) / (2 * math.log(base))  # noqa: E731
    a, b = math.floor(at(32.0)), math.ceil(at(1.0))
    t = ((i - a) / (b - a)).clamp(0, 1)
    assert math.isclose(scale, 0.1 * math.log(fac) + 1, rel_tol=1e-7)
    assert torch.allclose(got, f * (1 - t) + f / fac * t, rtol=1e-13)
    assert torch.equal(qmoe.rope_frequencies(R, base, "bands", 1.0, trained=n)[0], f) or \
        torch.allclose(qmoe.rope_frequencies(R, base, "bands", 1.0, trained=n)[0], f, rtol=1e-15)


@pytest.mark.parametrize("kw", [dict(rot_dim=0), dict(rot_dim=7), dict(rot_dim=8, base=1.0), dict(rot_dim=8, base=math.nan),
                                dict(rot_dim=8, kind="linear", factor=0.5), dict(rot_dim=2, kind="base", factor=2.0),
                                dict(rot_dim=8, kind="bands", factor=2.0, trained=0),
                                dict(rot_dim=8, kind="ramp", factor=2.0, trained=10, low=4.0, high=4.0),
                                dict(rot_dim=8, kind="ramp", factor=math.nan, trained=10)])
def test_frequencies_refused(kw):
    with pytest.raises(qmoe.QmoeError) as e:
        qmoe.rope_frequencies(**kw)
    assert e.value.code == INVALID


def test_workspace_bytes():
    f = qmoe.lib().attn_paged_workspace_bytes
    assert f(0, 1) == f(264, 1) == f(60, 1) == f(128, 0) == 0
    for dim in (8, 64, 128, 256):
        sizes = [f(dim, r) for r in (1, 16, 17, 40, 64, 65, 1000, 1 << 20)]
        assert sizes[0] > 4096 and sizes == sorted(sizes)   # a workspace for more rows serves fewer


def cache(**kw):
    d = dict(k=PTR, v=PTR, page_stride=16 * 2 * 64, token_stride=2 * 64, head_stride=64, num_pages=4, page_size=16, kv_heads=2,
             head_dim=64, dtype=0)
    return qmoe.CKVCache(**(d | kw))


def batch(**kw):
    return qmoe.CKVBatch(**(dict(page_table=PTR, q_start=PTR, kv_len=PTR, batch=2, max_pages=2, tokens=2, max_new=1) | kw))


BAD_CACHE = [(dict(k=None), INVALID), (dict(v=None), INVALID), (dict(dtype=2), INVALID), (dict(dtype=-1), INVALID),
             (dict(num_pages=0), INVALID), (dict(page_size=0), INVALID), (dict(kv_heads=0), INVALID), (dict(head_dim=0), INVALID),
             (dict(page_stride=-8), INVALID), (dict(head_dim=60), UNSUP), (dict(head_dim=264), UNSUP), (dict(k=PTR + 8), ALIGN),
             (dict(token_stride=132), ALIGN), (dict(head_stride=4), ALIGN), (dict(page_size=1 << 30), UNSUP)]
BAD_BATCH = [(dict(page_table=None), INVALID), (dict(q_start=None), INVALID), (dict(kv_len=None), INVALID), (dict(batch=0), INVALID),
             (dict(max_pages=0), INVALID), (dict(tokens=-1), INVALID), (dict(max_new=-1), INVALID), (dict(kv_len=PTR + 2), ALIGN),
             (dict(tokens=1 << 29), UNSUP)]


def attn(c, b, ws=PTR, nbytes=1 << 30, **kw):
    q = kw.pop("q", PTR)
    d = dict(q=qmoe.CRows(q, kw.pop("qt", 256), kw.pop("qh", 64)), out=qmoe.CRows(kw.pop("out", PTR), 256, 64), lse=None, heads=4,
             window=0, causal=1, scale=0.125, softcap=0.0)
    a = qmoe.CAttn(**(d | kw))
    return qmoe.lib().attn_paged(ctypes.byref(a), ctypes.byref(c), ctypes.byref(b), ws, nbytes, None, None)


def test_attn_refusals():
    for kw, code in BAD_CACHE:
        assert attn(cache(**kw), batch()) == code, kw
    for kw, code in BAD_BATCH:
        assert attn(cache(), batch(**kw)) == code, kw
    for kw, code in [(dict(q=None), INVALID), (dict(out=None), INVALID), (dict(heads=0), INVALID), (dict(heads=3), INVALID),
                     (dict(window=-1), INVALID), (dict(softcap=-1.0), INVALID), (dict(softcap=math.nan), INVALID),
                     (dict(scale=0.0), INVALID), (dict(scale=math.nan), INVALID), (dict(q=PTR + 2), ALIGN), (dict(out=PTR + 8), ALIGN),
                     (dict(qt=252), ALIGN), (dict(qh=68), ALIGN), (dict(lse=PTR + 2), ALIGN), (dict(ws=None), WS), (dict(nbytes=4096), WS),
                     (dict(ws=PTR + 8), ALIGN)]:
        assert attn(cache(), batch(), **kw) == code, kw
    L = qmoe.lib()
    assert L.attn_paged(None, ctypes.byref(cache()), ctypes.byref(batch()), PTR, 1 << 30, None, None) == INVALID


def test_append_and_rotate_refusals():
    L = qmoe.lib()
    rope = lambda **kw: qmoe.CRope(**(dict(inv_freq=PTR, rot_dim=64, layout=0, scale=1.0) | kw))  # noqa: E731
    rows = lambda p=PTR: ctypes.byref(qmoe.CRows(p, 256, 64))  # noqa: E731

    def append(c=None, b=None, r=None, pos=None, q=True, q_out=True, heads=4, k=PTR, v=PTR):
        return L.kv_append(ctypes.byref(c or cache()), ctypes.byref(b or batch()), ctypes.byref(r) if r else None, pos,
                           rows() if q else None, rows() if q_out else None, heads, rows(k), rows(v), None, None)

    for kw, code in BAD_CACHE:
        assert append(cache(**kw), r=rope()) == code, kw
    for kw, code in BAD_BATCH:
        assert append(b=batch(**kw), r=rope()) == code, kw
    bad_rope = [(dict(inv_freq=None), INVALID), (dict(rot_dim=0), INVALID), (dict(rot_dim=3), INVALID), (dict(rot_dim=66), INVALID),
                (dict(layout=2), INVALID), (dict(inv_freq=PTR + 4), ALIGN)]
    for kw, code in bad_rope:
        assert append(r=rope(**kw)) == code, kw
    assert append() == INVALID                                       # queries without a rotation
    assert append(r=rope(), q_out=False) == INVALID
    assert append(r=rope(), q=False) == INVALID and append(r=rope(), q=False, q_out=False) == INVALID   # heads left over
    assert append(r=rope(), heads=0) == INVALID and append(r=rope(), k=None) == INVALID
    assert append(r=rope(), k=PTR + 1) == ALIGN and append(r=rope(), pos=PTR + 2) == ALIGN

    def rotate(r=None, x=PTR, dtype=0, tokens=3, heads=2, dim=64, pos=PTR, out=PTR):
        return L.rope_rotate(ctypes.byref(r or rope()), x, 128, 64, dtype, tokens, heads, dim, pos, out, 128, 64, None, None)

    for kw, code in bad_rope:
        assert rotate(rope(**kw)) == code, kw
    for kw, code in [(dict(x=None), INVALID), (dict(out=None), INVALID), (dict(pos=None), INVALID), (dict(dtype=2), INVALID),
                     (dict(tokens=-1), INVALID), (dict(heads=0), INVALID), (dict(dim=1), INVALID), (dict(dim=1026), UNSUP),
                     (dict(x=PTR + 1), ALIGN), (dict(pos=PTR + 1), ALIGN)]:
        assert rotate(**kw) == code, kw


def test_logits_refusals():
    L = qmoe.lib()
    full = dict(history=PTR, history_len=PTR, prompt_len=PTR, history_stride=8, repetition=PTR, presence=PTR, frequency=PTR,
                bias_ids=PTR, bias=PTR, mask=PTR, mask_stride=4, max_history=8, max_bias=3)

    def call(x=PTR, ist=100, dtype=2, rows=2, vocab=100, out=PTR, ost=100, ws=PTR, nbytes=1 << 30, **kw):
        return L.logits_process(ctypes.byref(qmoe.CLogitRules(**(full | kw))), x, ist, dtype, rows, vocab, out, ost, ws, nbytes, None, None)

    for kw, code in [(dict(x=None), INVALID), (dict(out=None), INVALID), (dict(dtype=3), INVALID), (dict(rows=-1), INVALID),
                     (dict(vocab=0), INVALID), (dict(ist=99), INVALID), (dict(ost=99), INVALID), (dict(history_len=None), INVALID),
                     (dict(history=None), INVALID), (dict(history=None, max_history=0), INVALID), (dict(history_stride=7), INVALID),
                     (dict(mask_stride=3), INVALID), (dict(bias=None), INVALID), (dict(max_bias=-1), INVALID), (dict(rows=65536), UNSUP),
                     (dict(max_bias=1025), UNSUP), (dict(max_history=1 << 20, history_stride=1 << 20), UNSUP), (dict(x=PTR + 2), ALIGN),
                     (dict(mask=PTR + 2), ALIGN), (dict(bias=PTR + 1), ALIGN), (dict(ws=PTR + 8), ALIGN),
                     (dict(max_history=9000, history_stride=9000, ws=None), WS),
                     (dict(max_history=9000, history_stride=9000, nbytes=1000), WS)]:
        assert call(**kw) == code, kw
    assert L.logits_process(None, PTR, 100, 2, 2, 100, PTR, 100, None, 0, None, None) == INVALID
    need = L.logits_process_workspace_bytes
    assert need(0, 100) == need(5, -1) == need(5, 100) == 0 and need(5, 9000) > 5 * 9000 * 4 and need(6, 9000) > need(5, 9000)


def test_struct_sizes_match_the_header(tmp_path):
    """The binding's structures have the layout of the C header's."""
    import os
    import shutil
    import subprocess
    if shutil.which("gcc") is None:
        pytest.skip("no C compiler")
    names = {"qmoe_kv_cache": qmoe.CKVCache, "qmoe_kv_batch": qmoe.CKVBatch, "qmoe_rope": qmoe.CRope, "qmoe_rows": qmoe.CRows,
             "qmoe_attn": qmoe.CAttn, "qmoe_logit_rules": qmoe.CLogitRules}
    src = tmp_path / "sizes.c"
    body = "".join('printf("%%zu\\n", sizeof(%s));' % n +
                   "".join('printf("%%zu\\n", offsetof(%s, %s));' % (n, f[0]) for f in c._fields_) for n, c in names.items())
    src.write_text('#include "qmoe.h"\n#include <stdio.h>\nint main(void) { %s return 0; }\n' % body)
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(root, "include"), str(src), "-o", str(tmp_path / "sizes")], check=True)
    got = list(map(int, subprocess.run([str(tmp_path / "sizes")], stdout=subprocess.PIPE, check=True).stdout.split()))
    want = [x for c in names.values() for x in [ctypes.sizeof(c)] + [getattr(c, f[0]).offset for f in c._fields_]]
    assert got == want


def test_attention_refuses_infinite_factors():
    for kw in (dict(softcap=math.inf), dict(scale=math.inf)):
        assert attn(cache(), batch(), **kw) == INVALID
