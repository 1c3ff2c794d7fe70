"""The vocabulary losses and the ZeRO step together, as examples/train_head.py
uses them: both losses fall, and the ranks' replicas stay equal."""

import importlib.util
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.gpu
def test_train_head_example(abi, cuda):
    spec = importlib.util.spec_from_file_location("train_head", os.path.join(ROOT, "examples", "train_head.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    h = module.run(steps=40, ranks=3)
    assert h["teacher"][-1] < 0.6 * h["teacher"][0], h["teacher"]
    assert h["student"][-1] < 0.6 * h["student"][0], h["student"]
