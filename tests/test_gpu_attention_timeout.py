"""A wait inside the attention kernels that runs out ends the call with a timeout
status, and the workspace serves the next call.

With a limit below 100 us a wait is one look: most CTAs give up while the copy
of their first tile is on its way, some come late enough to find it."""
import pytest
import torch

from moe_expert_gemv_b200 import qmoe
from tests._attn import Case

pytestmark = pytest.mark.gpu

# few rows; many; two row tiles a unit; many without TMA (a decode call has no wait there)
CASES = {"long": ([(1, 20000)], 8, 2, 128, 64), "ragged": ([(1, 3000), (1, 70), (1, 9000)], 8, 4, 64, 16), "wide": ([(2, 60000)], 8, 2, 256, 32),
         "drafts": ([(40, 5000)], 8, 2, 128, 64), "chunks": ([(300, 700), (70, 70), (230, 257), (40, 40)], 64, 8, 64, 16),
         "heads of 256": ([(70, 3000)], 8, 2, 256, 32), "no map": ([(70, 3000), (9, 90)], 8, 2, 128, 7)}


@pytest.mark.parametrize("own", [True, False], ids=["own workspace", "given workspace"])
@pytest.mark.parametrize("name", list(CASES))
def test_a_wait_that_runs_out(cuda_dev, name, own):
    c = Case(*CASES[name])
    b = c.batch(max(n for n, _ in c.lens))
    ws = None if own else qmoe.attn_workspace(256, 1 << 14)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.check(qmoe.attn_paged(c.cache, b, c.q, workspace=ws, status=status))
    gave_up = 0
    for limit in (1, 99_999, 100_000, 50_000_000):
        for _ in range(4):
            before = qmoe.qmoe_set_attn_wait_limit_ns(limit)
            try:
                out = qmoe.attn_paged(c.cache, b, c.q, workspace=ws, status=status)
                flags = int(status)   # the call ended
            finally:
                assert qmoe.qmoe_set_attn_wait_limit_ns(before) == limit
            assert flags in (0, qmoe.DEV_TIMEOUT) and not (flags and limit > 1_000_000)
            gave_up += flags != 0
            if ws is not None:
                assert not ws[:4096].any()
            if not flags:
                c.check(out)
            status.zero_()
            c.check(qmoe.attn_paged(c.cache, b, c.q, workspace=ws, status=status))
            assert int(status) == 0
    assert gave_up > 0
    assert qmoe.qmoe_set_attn_wait_limit_ns(0) == 2_000_000_000 and qmoe.qmoe_check_status() == 0
