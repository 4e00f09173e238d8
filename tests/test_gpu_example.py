"""The operators together: the finetuning example trains (its loss falls well below
the projected layer's) and serves each request's adapter."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("state", ["f32", "fp8"])
def test_finetuning_lowers_the_loss_and_serves(state):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("adapter_finetune",
                                                  os.path.join(ROOT, "examples", "adapter_finetune.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    first, last, (served, want) = m.finetune(steps=60, state=state)
    assert last < 0.5 * first, (first, last)
    # bf16: the projection's rounding, and that of the sum (2^-8 each)
    assert ((served.float() - want).abs() <= 2.0 ** -7 * want.abs() + 2.0 ** -7 * want.abs().max()).all()
