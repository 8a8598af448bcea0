"""The example layer of experts: a whole training step through the library
against FP32 autograd.

e4m3 keeps 4 significant bits: a value is off by at most 2^-4 of itself, and by
about 2^-4 / sqrt(3) in the mean square of a spread of values; a product of two
such operands by sqrt(2) of that, 5%. Nothing in the step goes through more
than four such products one after the other (W1, W2, and back), which add
in the mean square to 10%; twice that is asked for."""

import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", [(2000, 1024, 1536, 16, 4), (37, 200, 136, 5, 2), (1, 128, 256, 8, 8),
                                   (4096, 512, 640, 4, 1)], ids=str)
def test_training_step_follows_fp32(cuda_device, shape):
    import experts_layer
    T, D, F, E, k = shape
    x, Wr, W1, W2, grad_out = experts_layer.inputs(T, D, F, E)
    got, indices = experts_layer.step(x, Wr, W1, W2, k, grad_out)
    want = experts_layer.reference(x, Wr, W1, W2, indices, grad_out)
    for name in want:
        if name == "Wr" and k == 1:
            # One renormalised weight is 1 whatever the logits: no gradient.
            assert not bool(got[name].any())
            continue
        off = float((got[name].float() - want[name]).norm() / want[name].norm())
        assert off < 0.2, (name, off)
