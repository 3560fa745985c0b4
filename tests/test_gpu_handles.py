"""The binding's handles for attention: what a batch, a cache and a rotation
hold is what the next call uses."""
import pytest
import torch

from moe_expert_gemv_b200 import qmoe
from tests._attn import Case

pytestmark = pytest.mark.gpu


def test_a_batch_whose_members_are_replaced(cuda_dev):
    """New tensors after the first call, the old ones' memory given to others."""
    c = Case([(1, 500), (3, 200)], 8, 2, 64, 16)
    b = c.batch(max_new=3)
    c.check(qmoe.attn_paged(c.cache, b, c.q))
    k = torch.randn(4, 2, 64, device="cuda").half()
    for cut in (100, 7):
        c.lens = [(n, kv - cut) for n, kv in c.lens]
        c.keys, c.values = ([t[:kv] for t, (_, kv) in zip(ts, c.lens)] for ts in (c.keys, c.values))
        b.kv_len = torch.tensor([kv for _, kv in c.lens], dtype=torch.int32, device="cuda")
        c.check(qmoe.attn_paged(c.cache, b, c.q))
    # the same tokens another way round
    c.lens = [(3, c.lens[0][1]), (1, c.lens[1][1])]
    b.q_start = torch.tensor([0, 3, 4], dtype=torch.int32, device="cuda")
    c.check(qmoe.attn_paged(c.cache, b, c.q))
    b.kv_len -= 1   # in place, and assigned again
    c.lens = [(n, kv - 1) for n, kv in c.lens]
    c.keys, c.values = ([t[:-1] for t in ts] for ts in (c.keys, c.values))
    c.check(qmoe.attn_paged(c.cache, b, c.q))
    # the sequences' pages change hands
    b.page_table = b.page_table.flip(0).contiguous()
    c.keys.reverse(), c.values.reverse()
    b.kv_len = b.kv_len.flip(0).contiguous()
    c.lens = [(n, kv) for (n, _), (_, kv) in zip(c.lens, reversed(c.lens))]
    c.check(qmoe.attn_paged(c.cache, b, c.q))
    qmoe.kv_append(c.cache, b, k, k)
    (n, kv), slots = c.lens[0], c.slots[1]
    assert torch.equal(c.k[slots[0][kv - n:kv], slots[1][kv - n:kv]], k[:n])
    assert qmoe.qmoe_check_status() == 0


def test_another_max_new(cuda_dev):
    """A smaller bound than at the first call asks for no larger workspace, a
    larger one chooses the other kernel."""
    c = Case([(3, 500), (1, 200)], 8, 2, 64, 16)
    b = c.batch(max_new=100)
    small = qmoe.attn_workspace(64, 12)
    c.check(qmoe.attn_paged(c.cache, b, c.q))
    b.max_new = 3
    c.check(qmoe.attn_paged(c.cache, b, c.q, workspace=small))
    b.max_new = 100
    with pytest.raises(qmoe.QmoeError) as e:
        qmoe.attn_paged(c.cache, b, c.q, workspace=small)
    assert e.value.code == qmoe.ERR_WORKSPACE
    assert qmoe.qmoe_check_status() == 0


def test_steps_of_many_sizes_hold_one_struct(cuda_dev):
    c = Case([(40, 500)], 8, 2, 64, 16)
    b = c.batch()
    for n in range(1, 41):
        b._c(n)
    assert b._held[0] == 40 and not any(isinstance(v, (dict, list)) for v in vars(b).values())


def test_refused_replacements(cuda_dev):
    c = Case([(1, 500), (3, 200)], 8, 2, 64, 16)
    b = c.batch()
    for name, bad in (("kv_len", torch.zeros(3, dtype=torch.int32, device="cuda")), ("q_start", b.kv_len), ("page_table", b.page_table[:1]),
                      ("page_table", b.page_table[:, :0])):
        with pytest.raises(ValueError):
            setattr(b, name, bad)
    with pytest.raises(TypeError):
        b.kv_len = b.kv_len.long()
    with pytest.raises(TypeError):
        b.kv_len = b.kv_len.cpu()
    for h, name in ((c.cache, "k"), (c.cache, "v"), (qmoe.Rope.make(64), "inv_freq")):
        with pytest.raises(AttributeError):
            setattr(h, name, torch.empty_like(getattr(h, name)))
    c.check(qmoe.attn_paged(c.cache, b, c.q))


def test_a_history_that_grows(cuda_dev):
    """What the binding keeps between calls stays as small as it is, and a
    stream's workspace is not made anew for every token."""
    x = torch.zeros(2, 300, device="cuda")
    hist = torch.zeros(2, 3000, dtype=torch.int32, device="cuda")
    n = torch.full((2,), 3000, dtype=torch.int32, device="cuda")
    one = torch.ones(2, device="cuda")
    stream, seen = torch.cuda.Stream(), set()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        for w in range(2500, 2700):
            y = qmoe.logits_process(x, history=hist[:, :w], history_len=n, presence=one)
            seen.add(qmoe._logits_ws[x.device.index, stream.cuda_stream].data_ptr())
            qmoe._attn_need(64, w)
        assert len(seen) == 1 and (y[:, 0] == -1).all() and not y[:, 1:].any()
        assert qmoe.qmoe_check_status() == 0
    for f in (qmoe._logits_need, qmoe._attn_need):
        assert f.cache_info().maxsize == 64 >= f.cache_info().currsize
