"""Streams that a call of the 8-bit layer is given."""
import types

import pytest
import torch


def test_a_stream_of_another_device_is_refused():
    """Its tensors' device has no such stream: the call must not run on another one instead."""
    from dense_fp32_matrix_10_gb300 import fp8
    stream = types.SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=0)
    with pytest.raises(ValueError, match="cuda:1"):
        fp8._on(stream, 0)
