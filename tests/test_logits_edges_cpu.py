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


def test_scales_have_a_lower_limit():
    """With S = 0 nothing is launched: the scale alone decides."""
    from split_residual_vector_b200 import build as lib_build
    lib_build.build()
    lib = pkg.library()
    rows = [None, 0, 0, 1, 100, 100, 0]
    calls = (lambda c: lib.mimi_rvq_token_logprob(*rows, None, 0, 0, -1, c, *[0], *[None] * 7),
             lambda c: lib.mimi_rvq_token_logprob_grad(*rows, None, 0, 0, -1, c, *[None] * 4, 100, 100,
                                                       *[None] * 5),
             lambda c: lib.mimi_rvq_distill_topk(*rows, None, None, 0, 4, 0, c, *[None] * 3),
             lambda c: lib.mimi_rvq_distill_topk_grad(*rows, None, None, 0, 4, 0, c, *[None] * 2, 100,
                                                      100, *[None] * 3))
    for call in calls:
        for c in (1e-30, 1.0, 1e30):
            assert call(c) == 0
        for c in (9.9e-31, 1e-37, 1e-44, 0.0, -1e-30):
            assert call(c) == -1
