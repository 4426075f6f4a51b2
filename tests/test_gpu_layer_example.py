"""examples/norm_linear.py: the layer operators as a program uses them together."""
import importlib.util
import os

import pytest

from conftest import ROOT

pytestmark = pytest.mark.gpu


def test_train_then_serve():
    path = os.path.join(ROOT, "examples", "norm_linear.py")
    spec = importlib.util.spec_from_file_location("norm_linear", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    got = example.main(steps=60)
    assert got["last_loss"] < 0.1 * got["first_loss"]
    # 4-bit weights in 15 steps over about +-3 sigma: 0.4 sigma a step, 0.4 / sqrt(12) = 12 %
    assert got["served_difference"] < 0.2
