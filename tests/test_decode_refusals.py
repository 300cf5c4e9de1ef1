"""Refusals of the decode operators' torch layer on the CPU: arguments whose
sizes say more than their memory holds. (Tensors stay on the host; the device
check is put aside, and every call is refused before any entry point.)"""

import pytest
import torch

from quantized_weight_skinny_amd import decode_api as qd

CPU = torch.device("cpu")


@pytest.fixture
def on_host(monkeypatch):
    monkeypatch.setattr(qd, "_on_device", lambda *a: None)


def test_a_workspace_must_be_contiguous(on_host):
    """An expanded tensor has elements that its storage does not, and between
    those of a strided one lie somebody else's."""
    for ws in (torch.empty(1, dtype=torch.uint8).expand(4096), torch.empty(8192, dtype=torch.uint8)[::2],
               torch.empty((64, 64), dtype=torch.uint8)[:, :32], torch.empty((64, 64), dtype=torch.float32).t()):
        with pytest.raises(ValueError, match="contiguous"):
            qd._workspace(1024, ws, CPU)
    ws = torch.empty((16, 64), dtype=torch.float32)
    assert qd._workspace(4096, ws, CPU) == (ws, ws.data_ptr(), 4096)
    assert qd._workspace(0, None, CPU) == (None, None, 0)
    assert qd._workspace(4097, ws, CPU)[0] is not ws       # too small: a new one
