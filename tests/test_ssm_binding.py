"""The state-space binding's handling of streams (no GPU needed)."""
import types

import pytest
import torch

from momentum_delta_rule_gb300 import ssm


def test_a_stream_of_another_device_is_refused():
    # the call would switch back to the tensors' device, and to its current stream
    t = types.SimpleNamespace(device=torch.device("cuda", 0))
    other = types.SimpleNamespace(device=torch.device("cuda", 1))
    with pytest.raises(ValueError, match="stream"):
        ssm._on(t, other)
