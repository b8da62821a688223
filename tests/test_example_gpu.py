"""The example runs the low-precision operators together, forward, backward and for one
token.  Its errors against fp32 autograd are those of the operands' rounding: e4m3 keeps
3 bits (a value is off by 2^-4 at most, about 2^-5.8 in the mean square), e2m1 one; two
to four such roundings add up in each result."""

import os
import sys

import pytest

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("fmt,limit", [("mxfp8", 0.08), ("mxfp4", 0.45), ("nvfp4", 0.35)])
def test_training_step_and_one_token(fmt, limit):
    import low_precision_mlp
    errors = low_precision_mlp.run(300, 512, 1000, fmt)
    assert all(e < limit for e in errors.values()), errors
    assert errors["y"] > 1e-3      # (it does compute in low precision)
