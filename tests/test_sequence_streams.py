"""Streams that a sequence operator cannot run on are refused (no GPU needed:
nothing is entered)."""
import pytest
import torch

from recurrent_state_update_amd.sequence import _on


class Stream:
    def __init__(self, device):
        self.device = torch.device(device)


@pytest.mark.parametrize("stream", [Stream("cuda:1"), Stream("cpu"), "0", object()])
def test_stream_of_another_device(stream):
    """Its handle would be ignored, and its device made the current one."""
    with pytest.raises(ValueError, match="stream of cuda:0"):
        _on(torch.device("cuda:0"), stream)
