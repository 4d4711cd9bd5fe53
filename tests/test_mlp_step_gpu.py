"""The operators together, as a training step uses them: the example's step
against autograd in 64 bits.

Every tensor that a product reads is rounded to bf16 (2^-8 of its value at
most, in the 2-norm about 2^-9): a gradient passes through at most six such
roundings (A1, Y, P, dY, dZ2, dZ1), so its relative error in the 2-norm stays
below 6 x 2^-8 even if they all pulled one way.  The loss sees A1 and Y.
"""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "mlp_step.py")
    spec = importlib.util.spec_from_file_location("mlp_step", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("sizes", [dict(), dict(T=64, H=72, F=200, V=257, p=0.5), dict(T=1500, H=512, F=520, p=0.0)])
def test_step_against_autograd(cuda_lib, example, sizes):
    import torch
    torch.manual_seed(1)
    errors = example.check(**sizes)
    assert errors.pop("loss") < 2 * 2.0**-8
    assert set(errors) == {"dX", "dW1", "dW2", "dhead", "db1", "db2"}
    for name, err in errors.items():
        assert err < 6 * 2.0**-8, (name, err)
