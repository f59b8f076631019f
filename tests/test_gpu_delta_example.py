"""The example layer: training lowers its loss, and serving gives what whole sequences give."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu


def test_example_trains_and_serves():
    path = os.path.join(os.path.dirname(__file__), "..", "examples", "gated_delta.py")
    spec = importlib.util.spec_from_file_location("gated_delta", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    losses, diff = mod.run(steps=16, tokens=400)
    assert all(torch.isfinite(torch.tensor(losses)))
    assert losses[-1] < 0.9 * losses[0]
    # both sides round each stage to bf16 (2^-9 of an element); their roundings differ at o, the gate and the projection
    assert diff < 1e-2
