"""The stream argument of the layer calls, without a GPU."""
import pytest
import torch


class Stream:
    def __init__(self, index):
        self.device = torch.device("cuda", index)
        self.device_index, self.cuda_stream = index, 0


def test_a_stream_of_another_device_is_refused():
    """It would be set aside: the call would run on its tensors' device, on
    whatever stream is current there."""
    from gated_delta_rule_55_amd import layer

    with pytest.raises(ValueError, match="stream"):
        with layer._on(torch.device("cuda", 0), Stream(1)):
            pass
