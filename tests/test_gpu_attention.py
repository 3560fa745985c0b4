"""attn_paged against the formula in 64 bits: types, head layouts, page sizes,
lengths from none to long ones, masks, poison where nothing may be read."""
import math
import threading

import pytest
import torch

from moe_expert_gemv_b200 import qmoe
from tests._attn import Case

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


def run(c, max_new=0, **kw):
    kw = {("softcap" if k == "cap" else k): v for k, v in kw.items()}
    out, lse = qmoe.attn_paged(c.cache, c.batch(max_new), c.q, want_lse=True, **kw)
    assert qmoe.qmoe_check_status() == 0
    return out, lse


DECODE = [(1, 1), (1, 2), (1, 63), (1, 64), (1, 65), (1, 300), (1, 1111)]
DRAFTS = [(5, 5), (3, 130), (8, 64), (1, 700), (7, 71)]
CHUNKS = [(70, 70), (129, 400), (1, 33), (256, 257), (31, 1000)]


@pytest.mark.parametrize("lens", [DECODE, DRAFTS, CHUNKS], ids=["decode", "drafts", "chunks"])
@pytest.mark.parametrize("heads,kv_heads", [(8, 8), (8, 2), (7, 1), (16, 1), (40, 2)])
@pytest.mark.parametrize("dim,page,dtype", [(64, 16, F16), (128, 16, BF16), (128, 7, F16), (256, 32, F16), (80, 20, BF16),
                                            (8, 1, F16), (104, 256, F16), (192, 64, BF16)])
def test_shapes(cuda_dev, lens, heads, kv_heads, dim, page, dtype):
    c = Case(lens, heads, kv_heads, dim, page, dtype, seed=dim + heads)
    out, lse = run(c, max(n for n, _ in lens))
    c.check(out, lse)


@pytest.mark.parametrize("kw", [dict(window=1), dict(window=17), dict(window=64), dict(window=100000), dict(cap=5.0),
                                dict(cap=50.0, window=100), dict(causal=False), dict(causal=False, window=30),
                                dict(scale=0.3, cap=30.0)], ids=str)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("lens", [DECODE, DRAFTS, CHUNKS], ids=["decode", "drafts", "chunks"])
def test_masks_and_caps(cuda_dev, kw, dim, lens):
    c = Case(lens, 8, 2, dim, 16, seed=3)
    out, lse = run(c, max(n for n, _ in lens), **kw)
    c.check(out, lse, **kw)


@pytest.mark.parametrize("max_new", [1, 6, 300])
def test_empty_sequences_and_rows(cuda_dev, max_new):
    """No new tokens, no cached ones, more new ones than cached ones; rows behind
    the last sequence are left as they were, whatever kernel max_new chooses."""
    c = Case([(0, 0), (1, 1), (0, 90), (4, 0), (6, 2), (0, 5), (1, 40), (0, 0)], 6, 2, 64, 16, spare=3)
    for causal in (True, False):
        out = torch.full(c.q.shape, 7.0, dtype=F16, device="cuda")
        lse = torch.full(c.q.shape[:2], 7.0, device="cuda")
        qmoe.attn_paged(c.cache, c.batch(max_new), c.q, out=out, lse=lse, causal=causal)
        assert qmoe.qmoe_check_status() == 0
        c.check(out, lse, causal=causal)
        assert (out[c.tokens:] == 7).all() and (lse[c.tokens:] == 7).all()


def test_nothing_at_all(cuda_dev):
    c = Case([(0, 0), (0, 10)], 4, 2, 64, 16)
    out, lse = run(c)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)


@pytest.mark.parametrize("max_new", [8, 64, 400])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("dim,page", [(64, 16), (128, 7), (128, 64), (256, 16), (256, 1)])
def test_poison_that_is_masked(cuda_dev, max_new, bad, dim, page):
    """A NaN or infinite key or value reaches the rows that see it and no other."""
    c = Case([(8, 200), (3, 9), (40, 150)], 8, 2, dim, page, BF16)
    for b, j in ((0, 196), (0, 10), (1, 8), (2, 130)):
        c.values[b][j, :, ::3] = bad
    c.write()
    for kw in (dict(), dict(window=60)):
        out, lse = run(c, max_new, **kw)
        c.check(out, lse, **kw)
    c.keys[0][197, 1] = math.nan   # seen by the last tokens only
    c.write()
    out, lse = run(c, max_new)
    first = c.q_start[1].item()
    out = out[:, 4:, 1::3]   # columns without poison in the values
    assert torch.isnan(out[first - 3:first]).all() and not torch.isnan(out[:first - 3]).any()


@pytest.mark.parametrize("dim,lens", [(128, DECODE), (64, CHUNKS), (256, DRAFTS)])
def test_strides(cuda_dev, dim, lens):
    """Cache pages [head][token], queries inside a QKV row, an output with gaps."""
    c = Case(lens, 8, 4, dim, 16, head_major=True)
    wide = torch.full((c.tokens, 13, dim), math.nan, dtype=F16, device="cuda")
    wide[:, 2:10] = c.q
    gap = torch.full((8, c.tokens, dim + 8), 3.0, dtype=F16, device="cuda")
    out = gap.transpose(0, 1)[..., :dim]
    qmoe.attn_paged(c.cache, c.batch(max(n for n, _ in lens)), wide[:, 2:10], out=out)
    assert qmoe.qmoe_check_status() == 0
    c.check(out)
    assert (gap[..., dim:] == 3).all()


@pytest.mark.parametrize("lens", [[(1, 20000)], [(1, 9001), (1, 3)], [(40, 5000)], [(300, 4000)]], ids=str)
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_long_contexts_are_split_and_repeat_bitwise(cuda_dev, lens, dim):
    c = Case(lens, 8, 2, dim, 64, seed=5)
    m = max(n for n, _ in lens)
    out, lse = run(c, m)
    c.check(out, lse)
    for _ in range(4):
        again, lse2 = run(c, m)
        assert torch.equal(out, again) and torch.equal(lse, lse2)


def test_many_sequences(cuda_dev):
    """More sequences than threads in a block."""
    g = torch.Generator().manual_seed(1)
    lens = [(int(n), int(n) + int(k)) for n, k in zip(torch.randint(0, 3, (700,), generator=g),
                                                      torch.randint(0, 90, (700,), generator=g))]
    for max_new in (2, 40):
        c = Case(lens, 4, 2, 64, 16)
        out, lse = run(c, max_new)
        c.check(out, lse)


def test_one_workspace_for_all_shapes(cuda_dev):
    ws = qmoe.attn_workspace(256, 4000)
    for dim, lens in ((64, DECODE), (256, CHUNKS), (128, [(1, 9000)]), (64, CHUNKS), (256, DECODE), (128, DRAFTS)):
        c = Case(lens, 8, 2, dim, 16)
        out, lse = run(c, max(n for n, _ in lens), workspace=ws)
        c.check(out, lse)
        assert not ws[:4096].any()


def test_bad_pages_and_lengths_are_flagged(cuda_dev):
    c = Case([(1, 100), (2, 50)], 4, 2, 64, 16)
    c.table[0, 3] = c.cache.num_pages
    out = qmoe.attn_paged(c.cache, c.batch(2), c.q)
    assert qmoe.qmoe_check_status() == qmoe.DEV_BAD_PAGE
    c.keys[0][48:64] = 0
    c.values[0][48:64] = 0
    c.check(out)
    c = Case([(1, 112)], 4, 2, 64, 16)
    c.kv_len[0] = 100000   # beyond the 7 pages: cut to 112
    out = qmoe.attn_paged(c.cache, c.batch(1), c.q)
    assert qmoe.qmoe_check_status() == qmoe.DEV_BAD_PAGE
    c.check(out)


@pytest.mark.parametrize("lens,dim", [([(1, 700), (1, 3000)], 128), ([(130, 700), (64, 64)], 128), ([(9, 600)], 256)])
def test_captured_graphs_replay_with_new_lengths(cuda_dev, lens, dim):
    """Two graphs of the same shapes, replayed in turn with lengths that change."""
    c = Case(lens, 8, 2, dim, 16)
    b = c.batch(max(n for n, _ in lens))
    graphs = []
    for window in (0, 50):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            out = qmoe.attn_paged(c.cache, b, c.q, window=window)
        graphs.append((g, out, window))
    keys, values = c.keys, c.values
    for cut in (0, 37, 1):
        c.lens = [(n, max(kv - cut, n)) for n, kv in lens]
        c.kv_len.copy_(torch.tensor([kv for _, kv in c.lens], dtype=torch.int32))
        c.keys = [k[:kv] for k, (_, kv) in zip(keys, c.lens)]
        c.values = [v[:kv] for v, (_, kv) in zip(values, c.lens)]
        for g, out, window in graphs:
            g.replay()
            torch.cuda.synchronize()
            c.check(out, window=window)
    assert qmoe.qmoe_check_status() == 0


def test_two_streams_at_once(cuda_dev):
    cases = [Case([(1, 9000)], 8, 2, 128, 16, seed=1), Case([(200, 3000)], 8, 2, 128, 16, seed=2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[], []]
    for _ in range(6):
        for i, (c, s) in enumerate(zip(cases, streams)):
            with torch.cuda.stream(s):
                got[i].append(qmoe.attn_paged(c.cache, c.batch(), c.q))
    torch.cuda.synchronize()
    for c, outs in zip(cases, got):
        for o in outs:
            c.check(o)


def test_offsets_beyond_32_bits(cuda_dev):
    """A cache of more than 2^32 elements whose last pages hold the sequence."""
    page, kvh, dim = 64, 8, 128
    pages = (1 << 32) // (page * kvh * dim) + 40
    c = Case([(1, 1000), (20, 300)], 16, kvh, dim, page)
    k = torch.empty(pages, page, kvh, dim, dtype=F16, device="cuda")
    v = torch.empty(pages, page, kvh, dim, dtype=F16, device="cuda")
    shift = pages - c.cache.num_pages
    k[shift:], v[shift:] = c.k, c.v
    c.table += torch.where(c.table < c.cache.num_pages, shift, 0).to(torch.int32)
    c.cache = qmoe.KVCache(k, v)
    out, lse = run(c, 20)
    c.check(out, lse)


def test_python_refusals(cuda_dev):
    c = Case([(1, 30)], 8, 2, 64, 16)
    b = c.batch()
    with pytest.raises(TypeError):
        qmoe.attn_paged(c.cache, b, c.q.bfloat16())
    with pytest.raises(ValueError):
        qmoe.attn_paged(c.cache, b, c.q[..., :56])
    with pytest.raises(ValueError):
        qmoe.attn_paged(c.cache, b, c.q.transpose(1, 2).contiguous().transpose(1, 2))
    with pytest.raises(qmoe.QmoeError):
        qmoe.attn_paged(c.cache, b, c.q[:, :7])
    with pytest.raises(qmoe.QmoeError) as e:
        qmoe.attn_paged(c.cache, b, c.q, workspace=torch.zeros(4096, dtype=torch.uint8, device="cuda"))
    assert e.value.code == qmoe.ERR_WORKSPACE
    with pytest.raises(qmoe.QmoeError):
        qmoe.attn_paged(c.cache, b, c.q, window=-1)
    with pytest.raises(TypeError):
        qmoe.attn_paged(c.cache, b, c.q.cpu())
    with pytest.raises(ValueError):
        qmoe.KVCache(c.k, c.v[:-1])


# enough rows for two row tiles in a unit
MANY = [(300, 700), (70, 70), (1, 33), (0, 40), (230, 257), (40, 40), (5, 0)]


def many(c):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert c.q.shape[0] * (c.heads // c.kv_heads) // 256 * c.kv_heads >= sms
    return c


@pytest.mark.parametrize("heads,kv_heads", [(64, 8), (62, 2), (64, 1)])
@pytest.mark.parametrize("dim,page,dtype", [(128, 16, BF16), (128, 7, F16), (64, 64, F16), (104, 32, BF16), (80, 1, F16), (8, 16, F16)])
def test_two_row_tiles(cuda_dev, heads, kv_heads, dim, page, dtype):
    c = many(Case(MANY, heads, kv_heads, dim, page, dtype, seed=dim, spare=3))
    out = torch.full(c.q.shape, 7.0, dtype=dtype, device="cuda")
    lse = torch.full(c.q.shape[:2], 7.0, device="cuda")
    run(c, 300, out=out, lse=lse)
    c.check(out, lse)
    assert (out[c.tokens:] == 7).all() and (lse[c.tokens:] == 7).all()
    again = torch.empty_like(out)
    run(c, 300, out=again)
    assert torch.equal(again[:c.tokens], out[:c.tokens])


@pytest.mark.parametrize("kw", [dict(window=1), dict(window=100), dict(cap=5.0), dict(cap=50.0, window=200), dict(causal=False),
                                dict(causal=False, window=30, cap=9.0)], ids=str)
@pytest.mark.parametrize("dim", [64, 128])
def test_two_row_tiles_with_masks_and_caps(cuda_dev, kw, dim):
    c = many(Case(MANY, 64, 8, dim, 16, seed=7))
    out, lse = run(c, 300, **kw)
    c.check(out, lse, **kw)


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("dim,page", [(64, 16), (128, 7), (128, 64)])
def test_two_row_tiles_with_poison(cuda_dev, bad, dim, page):
    c = many(Case([(300, 330), (300, 310), (30, 90)], 64, 8, dim, page, BF16))
    for b, j in ((0, 326), (0, 150), (1, 20), (1, 300), (2, 70)):
        c.values[b][j, :, ::3] = bad
    c.write()
    for kw in (dict(), dict(window=60)):
        out, lse = run(c, 300, **kw)
        c.check(out, lse, **kw)


def test_two_row_tiles_in_a_graph(cuda_dev):
    c = many(Case(MANY[:-1], 64, 8, 128, 16))
    b = c.batch(300)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        out, lse = qmoe.attn_paged(c.cache, b, c.q, want_lse=True)
    keys, values = c.keys, c.values
    for cut in (0, 37):
        c.lens = [(n, max(kv - cut, n)) for n, kv in MANY[:-1]]
        c.kv_len.copy_(torch.tensor([kv for _, kv in c.lens], dtype=torch.int32))
        c.keys = [k[:kv] for k, (_, kv) in zip(keys, c.lens)]
        c.values = [v[:kv] for v, (_, kv) in zip(values, c.lens)]
        g.replay()
        torch.cuda.synchronize()
        c.check(out, lse)
    assert qmoe.qmoe_check_status() == 0


def test_two_threads_on_one_stream(cuda_dev):
    """Calls of two kernels each, with one workspace, from two threads at once."""
    cases = [Case([(60, 4000)], 8, 2, 128, 16, seed=1), Case([(200, 3000)], 8, 2, 128, 16, seed=2)]
    want = [qmoe.attn_paged(c.cache, c.batch(), c.q) for c in cases]
    torch.cuda.synchronize()
    got, errors = [[], []], []

    def work(i):
        try:
            for _ in range(200):
                got[i].append(qmoe.attn_paged(cases[i].cache, cases[i].batch(), cases[i].q))
        except Exception as e:  # shown by the main thread
            errors.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors and qmoe.qmoe_check_status() == 0
    for i, c in enumerate(cases):
        c.check(want[i])
        assert all(torch.equal(o, want[i]) for o in got[i])


@pytest.mark.parametrize("lens,max_new", [([(40, 300), (9, 77)], 40), ([(1, 300), (2, 77)], 1)])
@pytest.mark.parametrize("dim,page", [(8, 16), (128, 7), (64, 1), (256, 5), (64, 16)])
def test_nothing_of_the_last_call_remains(cuda_dev, lens, max_new, dim, page):
    """After a call whose values are infinite, which shared memory may still
    hold, the limits of a call's tiles are cleaned of its own values only."""
    bad = Case(lens, 8, 2, dim, page, seed=3)
    for v in bad.values:
        v.fill_(math.inf)
    bad.write()
    c = Case(lens, 8, 2, dim, page, seed=4)
    first, lse = run(c, max_new)
    c.check(first, lse)
    for _ in range(30):
        qmoe.attn_paged(bad.cache, bad.batch(max_new), bad.q)
        out, _ = run(c, max_new)
        assert torch.equal(out, first)
