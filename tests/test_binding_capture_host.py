"""The binding asks the device of a call's tensors, not the current one, whether
its stream is being captured: a graph's workspace is the graph's own."""
import contextlib

import pytest
import torch

from moe_expert_gemv_b200 import qmoe


@pytest.fixture
def devices(monkeypatch):
    """Two devices, of which 0 is current; `capturing` holds those whose current stream is being captured."""
    state = {"current": 0, "capturing": set()}

    @contextlib.contextmanager
    def device(d):
        before, state["current"] = state["current"], d.index
        yield
        state["current"] = before
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: state["current"], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 100 + i, raising=False)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch._C, "_cuda_isCurrentStreamCapturing", lambda: state["current"] in state["capturing"], raising=False)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: state["current"] in state["capturing"])
    monkeypatch.setattr(qmoe, "attn_workspace", lambda dim, rows, device: torch.zeros(1 << 24, dtype=torch.uint8))
    monkeypatch.setattr(qmoe, "_attn_ws", {})
    return state


@pytest.mark.parametrize("index", [0, 1])
def test_the_graph_has_its_own(devices, index):
    dev = torch.device("cuda", index)
    for other in ({1 - index}, set()):   # a capture elsewhere does not count
        devices["capturing"] = other
        assert qmoe._attn_workspace(64, 4, dev) is qmoe._attn_workspace(64, 4, dev)
    assert list(qmoe._attn_ws) == [(index, 100 + index)]
    devices["capturing"] = {index}
    kept = qmoe._attn_ws[index, 100 + index]
    a, b = qmoe._attn_workspace(64, 4, dev), qmoe._attn_workspace(64, 4, dev)
    assert a is not b and a is not kept and b is not kept
    assert len(qmoe._attn_ws) == 1 and qmoe._attn_ws[index, 100 + index] is kept and devices["current"] == 0
