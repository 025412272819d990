"""The stream of a call has to be on its tensors' device: the workspace would be made for another one and the kernel would
run there (no GPU: stand-ins with a device)."""
from types import SimpleNamespace

import pytest
import torch


@pytest.mark.parametrize("mine,theirs", [(0, 1), (1, 0)])
def test_a_stream_of_another_device_is_refused(monkeypatch, mine, theirs):
    from linear_recurrent_sequence_amd import retention as R
    monkeypatch.setattr(torch.cuda, "current_device", lambda: mine)
    t = SimpleNamespace(device=torch.device("cuda", mine))
    made = []
    with pytest.raises(ValueError, match="stream"):
        R._launch(t, SimpleNamespace(device=torch.device("cuda", theirs), cuda_stream=0), None, lambda: made.append(1))
    assert not made
    workspace = object()
    got = R._launch(t, SimpleNamespace(device=torch.device("cuda", mine), cuda_stream=24), workspace, None)
    assert got[1].value == 24 and got[2] is workspace
