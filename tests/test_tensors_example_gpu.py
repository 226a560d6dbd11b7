"""The example runs as it is written, and learns: with either moment format
its loss falls to less than a quarter (it starts as the distance of two
unrelated models), and the step counts on the device."""

import os
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("moments", [8, 32])
def test_the_example_learns(moments):
    import tensor_list_step
    losses, norm, applied = tensor_list_step.train(moments=moments, steps=150)
    assert applied == 150 and norm == norm
    assert losses[-1] < losses[0] / 4, (losses[0], losses[-1])
