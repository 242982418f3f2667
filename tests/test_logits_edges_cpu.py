"""Checks of the logits calls' arguments in Python that need no GPU."""
import types

import pytest

import split_residual_vector_b200 as pkg

torch = pytest.importorskip("torch")


def test_a_stream_of_another_device_is_refused():
    """A call would otherwise run on its tensors' device's own current stream."""
    other = types.SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=0)
    with pytest.raises(AssertionError, match="another device"):
        with pkg._current(torch.device("cuda", 0), other):
            pass
