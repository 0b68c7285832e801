"""A caller's workspace of windowed attention, as the binding takes it (CPU only: stand-ins for tensors of other devices)."""
import pytest
import torch

import tree_speculative_verification_gdn_gb300 as tv


class Elsewhere:
    """What the binding asks of a tensor, on a device of its own."""

    def __init__(self, device, cuda=True, contiguous=True):
        self.device, self.is_cuda, self.contiguous = f"cuda:{device}" if cuda else "cpu", cuda, contiguous
        self.index = device

    def get_device(self):
        return self.index

    def is_contiguous(self):
        return self.contiguous

    def data_ptr(self):
        return 4096

    def numel(self):
        return 10

    def element_size(self):
        return 4


def test_a_workspace_lies_on_the_current_device():
    room, size = tv._room(Elsewhere(0), 0)
    assert room.value == 4096 and size == 40
    with pytest.raises(ValueError, match="cuda:1"):
        tv._room(Elsewhere(1), 0)
    for wrong in (Elsewhere(0, cuda=False), Elsewhere(0, contiguous=False)):
        with pytest.raises(ValueError):
            tv._room(wrong, 0)


@pytest.mark.parametrize("call", [tv.tv_window_attn_prompt, tv.tv_window_attn_step])
def test_both_calls_look_at_it(call, monkeypatch):
    seen = []

    def look(workspace, device):
        seen.append(device)
        raise ValueError("looked")
    monkeypatch.setattr(tv, "_room", look)
    monkeypatch.setattr(tv, "_current", lambda t, name: 0)
    q, n, bf = torch.zeros(2, 4, 128, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32), torch.bfloat16
    cache, table = torch.zeros(3, 2, 16, 128, dtype=bf), torch.zeros(2, 1, dtype=torch.int32)
    with pytest.raises(ValueError, match="looked"):
        if call is tv.tv_window_attn_step:
            call(q, cache, cache, table, n, q, n, workspace=Elsewhere(1))
        else:
            call(q, cache, cache, table, torch.zeros(3, dtype=torch.int32), n, q, n, workspace=Elsewhere(1))
    assert seen == [0]
