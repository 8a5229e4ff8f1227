"""The example that runs the gated delta rule and the layer norm together."""

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu


def test_recall_example():
    """Training with the library's gradients learns the task, and answering
    token by token from the prompt's state gives the whole forward's logits:
    both round to bfloat16 (2^-8) at most ten times a block on the way."""
    from complex_valued_state_gb300 import build as cbuild
    from complex_valued_state_gb300 import cssd

    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for gpu tests")
    cbuild.build()
    cssd.load()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "delta_recall.py")
    spec = importlib.util.spec_from_file_location("delta_recall", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    r = ex.run(steps=120, pairs=48, report=lambda *_: None)
    assert r["losses"][-1] < 0.3 * r["losses"][0]
    assert r["right"] > 0.8
    assert r["apart"] < 2 * 10 * 2.0 ** -8
    assert cssd.device_status() == 0
