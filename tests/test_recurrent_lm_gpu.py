"""The example that runs layer norm and the gated linear recurrence together:
training on packed sequences learns, and decoding token by token gives the
logits of the whole prompts."""
import importlib.util
import os

import pytest
import torch

from linear_attention_delta_gb300 import kla

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(
    __file__))), "examples", "recurrent_lm.py")


def test_example_learns_and_decodes():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    spec = importlib.util.spec_from_file_location("recurrent_lm", PATH)
    lm = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(lm)
    losses, worst, scale = lm.main(steps=120)
    # chance is ln 32 = 3.47: a nat below it takes the earlier tokens
    assert losses[0] > 3.0 and losses[-1] < 2.4, (losses[0], losses[-1])
    # bf16 activations: a few roundings of 2^-8 of the logits' size
    assert worst <= 8 * 2.0 ** -8 * scale, (worst, scale)
    assert kla.device_status() == 0
