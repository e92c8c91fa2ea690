"""The example runs, and training lowers its loss."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_adapter_finetune():
    spec = importlib.util.spec_from_file_location("adapter_finetune",
                                                  os.path.join(HERE, "examples", "adapter_finetune.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    losses = module.main(steps=25)
    assert losses[-1] < 0.5 * losses[0]
