"""The example that runs the Hessian, the quantization, the feed-forward block and the loss together."""

import importlib.util
import os

import pytest
import torch

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs an MI355X GPU")]

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "repair_gated_block.py")


def test_repair_lowers_the_loss():
    spec = importlib.util.spec_from_file_location("repair_gated_block", PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    before, after = mod.main(d=128, f=320, vocab=1001, top=16, tokens=500, steps=40)
    assert 0.0 < after < 0.8 * before
