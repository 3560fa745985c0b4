"""logits_process with the histories at which its two ways of finding a slice's
tokens change: looked through by every slice, or sorted first by 8 ranges of
slices, 12288 tokens at a time, from 7000000 rows x slices x tokens on."""
import pytest
import torch

from moe_expert_gemv_b200 import qmoe
from tests.test_gpu_logits import check, make

pytestmark = pytest.mark.gpu

V = 262144   # 129 slices of 2048 where rows are few


def run(d, offset=0, **kw):
    """As it stands, and with rows that begin `offset` elements behind a 16-byte boundary, in place."""
    c = {k: v.cuda() for k, v in d.items()}
    x = c.pop("logits")
    y = qmoe.logits_process(x, **c, **kw)
    wide = torch.full((x.shape[0], x.shape[1] + 24), 7.0, dtype=x.dtype, device="cuda")
    view = wide[:, offset:offset + x.shape[1]]
    view.copy_(x)
    qmoe.logits_process(view, out=view, **c, **kw)
    assert qmoe.qmoe_check_status() == 0
    assert torch.equal(view, y) and (wide[:, :offset] == 7).all() and (wide[:, offset + x.shape[1]:] == 7).all()
    return y


@pytest.mark.parametrize("rows,hist", [(4, 13565), (4, 13566), (5, 12287), (5, 12288), (5, 12289), (5, 24576), (5, 24577), (3, 36865)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_where_the_way_changes(cuda_dev, rows, hist, dtype):
    d = make(rows, V, hist, biases=3, mask=True, dtype=dtype, seed=hist)
    d["history_len"][:] = hist
    d["history_len"][1] = hist - 1
    check(d, run(d, offset=5))


# where the tokens lie: one range, its neighbours' limits, the first and the last slice
PLACES = {"first slice": (0, 2040), "last slice": (V - 100, V), "one range": (5 * 34816, 6 * 34816), "a range's limit": (34816 - 9, 34816 + 9),
          "the last range": (7 * 34816, V), "one token": (77777, 77778), "everywhere": (0, V)}


@pytest.mark.parametrize("place", list(PLACES))
@pytest.mark.parametrize("offset", [0, 1, 2, 3, 4, 5, 6, 7])
def test_where_the_tokens_lie(cuda_dev, place, offset):
    lo, hi = PLACES[place]
    d = make(5, V, 14000, biases=4, mask=True, dtype=torch.bfloat16, seed=offset)
    g = torch.Generator().manual_seed(offset)
    d["history"] = torch.randint(lo, hi, (5, 14000), generator=g).int()
    d["history"][0, ::7] = -1
    d["history_len"] = torch.tensor([14000, 0, 1, 12288, 13999], dtype=torch.int32)
    d["prompt_len"] = torch.tensor([0, 0, 1, 12288, 20000], dtype=torch.int32)
    d["bias_ids"][:, 0] = lo
    d["frequency"] /= 1000
    check(d, run(d, offset=offset))


@pytest.mark.parametrize("rows", [1, 60])
def test_one_token_a_million_times(cuda_dev, rows):
    """Every count the words hold, unsorted and sorted, is exact."""
    n = (1 << 20) - 1 if rows == 60 else 200000
    d = make(rows, 40000, 4, mask=True)
    d["mask"][:] = -1
    d["history"] = torch.full((rows, n), 39999, dtype=torch.int32)
    d["history_len"] = torch.full((rows,), n, dtype=torch.int32)
    d["prompt_len"] = torch.arange(rows, dtype=torch.int32)
    d["repetition"][:], d["presence"][:], d["frequency"][:] = 1.0, 0.0, 1.0
    c = {k: v.cuda() for k, v in d.items()}
    x = c.pop("logits")
    y = qmoe.logits_process(x, **c)
    assert qmoe.qmoe_check_status() == 0
    assert torch.equal(y[:, :39999], x[:, :39999])
    assert torch.equal(y[:, 39999], x[:, 39999] - (n - c["prompt_len"]).float())
